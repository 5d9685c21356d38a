"""MI355X (gfx950) hot path of a row-parallel block-scale fp8 linear layer.

Thin ctypes binding over ``libbsgemm.so`` (declared in ``include/bsgemm.h``):
the functions here only check and marshal torch tensors (device pointers,
sizes, the current HIP stream) and raise on a non-OK status.  Every step of
the path runs in the library's HIP kernels; there is no fallback.  If the
library has not been built, importing the functions raises immediately.

  bsgemm_fp8(A, a_scale, B, b_scale, C=None, bands=1, band_stride=0)
  band_reduce(parts, out=None)
  rowq_e4m3(x, q=None, scale=None)
  rowdq_e4m3(q, scale, y=None)
  blockq_e4m3(x, block_rows, q=None, scale=None)
  actq_e4m3(x, q=None, scale=None)
  bprepack_e4m3(B, Bp=None)
  bsgemm_fp8_pb(A, a_scale, Bp, b_scale, C=None, bands=1, band_stride=0)
  mxgemm_fp8(A, a_scale, B, b_scale, C=None, bands=1, band_stride=0)
  band_rowq_e4m3(parts, q=None, scale=None)
  mxq_e4m3(x, q=None, scale=None)
  lora_plan(ids, n_adapters, plan=None)
  lora_shrink(x, A, plan, H=None)
  lora_expand(H, B, plan, base, out=None, scale=None, bands=1, band_stride=0)
  bsgemm_fp8_lora(A, a_scale, B, b_scale, H, lora_B, ids, scale=None, C=None, bands=1,
                  band_stride=0)
  resnorm(y, resid, y_scale=None, post_w=None, gate=None, pre_w=None, alpha=1.0, beta=1.0,
          eps=1e-6, quant=0, resid_out=None, z=None, q=None, q_scale=None)

Tensors: e4m3 codes are uint8 (or torch.float8_e4m3fn, reinterpreted), bf16
values are torch.bfloat16 (or int16/uint16 bit patterns), scales float32.
All tensors must live on the current CUDA (HIP) device and be contiguous.
Every call takes stream=None, the torch.cuda.Stream to enqueue on (None: the
current one); outputs that it allocates belong to that stream.
The C ABI receives raw pointers and cannot see sizes, so every wrapper checks
each operand's shape and each output's element count against the sizes the
call implies before it takes a pointer, and raises ValueError on a mismatch:
a wrong-shaped buffer never reaches a kernel.
"""
import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbsgemm.so")

BS_OK, BS_ERR_INVALID, BS_ERR_UNSUPPORTED, BS_ERR_LAUNCH = 0, 1, 2, 3

# every extern "C" symbol of include/bsgemm.h
EXPORTS = ("bsgemm_fp8", "band_reduce", "rowq_e4m3", "rowdq_e4m3", "blockq_e4m3", "actq_e4m3",
           "mxgemm_fp8", "mxq_e4m3", "bprepack_e4m3", "bsgemm_fp8_pb", "band_rowq_e4m3",
           "lora_plan", "lora_shrink", "lora_expand", "bsgemm_fp8_lora", "resnorm",
           "bs_status_str")

_lib = None


class BSError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {status_str(status)} (status {status})")


def load():
    """Load libbsgemm.so (built in-tree by ``_build.py``); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m block_scaled_fp8_bsgemm_amd._build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    L.bsgemm_fp8.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, i64, vp]
    L.band_reduce.argtypes = [ctypes.POINTER(vp), i32, vp, i64, i64, vp]
    L.rowq_e4m3.argtypes = [vp, vp, vp, i64, i64, vp]
    L.rowdq_e4m3.argtypes = [vp, vp, vp, i64, i64, vp]
    L.blockq_e4m3.argtypes = [vp, vp, vp, i64, i64, i32, vp]
    L.actq_e4m3.argtypes = [vp, vp, vp, i64, i64, vp]
    L.mxgemm_fp8.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, i64, vp]
    L.mxq_e4m3.argtypes = [vp, vp, vp, i64, i64, vp]
    L.bprepack_e4m3.argtypes = [vp, vp, i64, i64, vp]
    L.bsgemm_fp8_pb.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, i64, vp]
    L.band_rowq_e4m3.argtypes = [ctypes.POINTER(vp), i32, vp, vp, i64, i64, vp]
    f32 = ctypes.c_float
    L.lora_plan.argtypes = [vp, vp, i64, i64, vp]
    L.lora_shrink.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, vp]
    L.lora_expand.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, i64, vp]
    L.bsgemm_fp8_lora.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, i64, vp]
    L.resnorm.argtypes = [vp, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, i64, i64, i32, i32, f32, f32, f32, vp]
    for f in EXPORTS[:-1]:
        getattr(L, f).restype = ctypes.c_int
    L.bs_status_str.argtypes = [ctypes.c_int]
    L.bs_status_str.restype = ctypes.c_char_p
    _lib = L
    return L


def status_str(status):
    return load().bs_status_str(int(status)).decode()


def _check(status, what):
    if status != BS_OK:
        raise BSError(status, what)


def _torch():
    import torch
    return torch


def _ptr(t, dtypes, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


def _shape(t, shape, name):
    _need(tuple(t.shape) == tuple(shape), f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _room(t, n, name):
    _need(t.numel() >= n, f"{name}: {t.numel()} elements, the call writes {n}")


def _dims2(t, name):
    _need(t.dim() == 2, f"{name} must be 2-D, got shape {tuple(t.shape)}")
    return t.shape


def _band_elems(M, N, bands, band_stride):
    """elements of C the band epilogue writes (0 when the ABI will reject the
    band arguments anyway)"""
    if bands < 1 or M % bands or band_stride < 0:
        return 0
    band_rows = M // bands
    stride = band_stride if band_stride else band_rows * N
    return (bands - 1) * stride + band_rows * N


def _check_gemm_operands(A, a_scale, B, b_scale, kq, what):
    """A [M,K], B [N,K]; blockscale (kq = 128): a_scale [M,K/128], b_scale
    [N/128,K/128]; mxfp8 (kq = 32): a_scale [M,K/32], b_scale [N,K/32]."""
    M, K = _dims2(A, "A")
    N, K2 = _dims2(B, "B")
    _need(K2 == K, f"{what}: A is [M,{K}] but B is [N,{K2}]")
    _need(K % 128 == 0 and N % 128 == 0, f"{what}: K and N must be multiples of 128 (K={K}, N={N})")
    if kq == 128:
        _shape(a_scale, (M, K // 128), "a_scale")
        _shape(b_scale, (N // 128, K // 128), "b_scale")
    else:
        _shape(a_scale, (M, K // 32), "a_scale")
        _shape(b_scale, (N, K // 32), "b_scale")
    return M, N, K


def _stream(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _empty(stream, shape, dtype, device):
    """An output of the call, allocated for the stream that writes it: the memory that a
    tensor of the current stream has left may still be in use there."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _u8():
    torch = _torch()
    return (torch.uint8, torch.int8, torch.float8_e4m3fn)


def _b16():
    torch = _torch()
    return (torch.bfloat16, torch.int16, torch.uint16)


def _f32():
    return (_torch().float32,)


def bsgemm_fp8(A, a_scale, B, b_scale, C=None, bands=1, band_stride=0, stream=None):
    """C (bf16) = blockscale(A [M,K] e4m3, a_scale [M,K/128]) x blockscale(B [N,K], b_scale [N/128,K/128])^T,
    written as `bands` destination-major row bands (band d at element d*band_stride)."""
    torch = _torch()
    M, N, K = _check_gemm_operands(A, a_scale, B, b_scale, 128, "bsgemm_fp8")
    need = _band_elems(M, N, bands, band_stride)
    if C is None:
        C = _empty(stream, need, dtype=torch.bfloat16, device=A.device)
    _room(C, need, "C")
    st = load().bsgemm_fp8(_ptr(A, _u8(), "A"), _ptr(a_scale, _f32(), "a_scale"),
                           _ptr(B, _u8(), "B"), _ptr(b_scale, _f32(), "b_scale"),
                           _ptr(C, _b16(), "C"), M, N, K, bands, band_stride, _stream(stream))
    _check(st, "bsgemm_fp8")
    return C


def band_reduce(parts, out=None, stream=None):
    """out (bf16 [rows,N]) = bf16(sum_p fp32(parts[p])), parts summed in index order."""
    torch = _torch()
    parts = list(parts)
    _need(len(parts) >= 1, "band_reduce: no parts")
    rows, N = _dims2(parts[0], "parts[0]")
    for i, p in enumerate(parts):
        _shape(p, (rows, N), f"parts[{i}]")
    if out is None:
        out = _empty(stream, (rows, N), dtype=torch.bfloat16, device=parts[0].device)
    _room(out, rows * N, "out")
    ptrs = (ctypes.c_void_p * len(parts))(*[_ptr(p, _b16(), "part") for p in parts])
    st = load().band_reduce(ptrs, len(parts), _ptr(out, _b16(), "out"), rows, N, _stream(stream))
    _check(st, "band_reduce")
    return out


def rowq_e4m3(x, q=None, scale=None, stream=None):
    """(q uint8 [rows,N], scale fp32 [rows]) = per-row e4m3 quantization of bf16 x."""
    torch = _torch()
    rows, N = _dims2(x, "x")
    if q is None:
        q = _empty(stream, (rows, N), dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = _empty(stream, (rows,), dtype=torch.float32, device=x.device)
    _room(q, rows * N, "q")
    _room(scale, rows, "scale")
    st = load().rowq_e4m3(_ptr(x, _b16(), "x"), _ptr(q, _u8(), "q"), _ptr(scale, _f32(), "scale"),
                          rows, N, _stream(stream))
    _check(st, "rowq_e4m3")
    return q, scale


def rowdq_e4m3(q, scale, y=None, stream=None):
    """y (bf16 [rows,N]) = bf16(decode(q) * scale[row])."""
    torch = _torch()
    rows, N = _dims2(q, "q")
    _need(scale.numel() == rows, f"scale: {scale.numel()} elements for {rows} rows")
    if y is None:
        y = _empty(stream, (rows, N), dtype=torch.bfloat16, device=q.device)
    _room(y, rows * N, "y")
    st = load().rowdq_e4m3(_ptr(q, _u8(), "q"), _ptr(scale, _f32(), "scale"), _ptr(y, _b16(), "y"),
                           rows, N, _stream(stream))
    _check(st, "rowdq_e4m3")
    return y


def blockq_e4m3(x, block_rows, q=None, scale=None, stream=None):
    """(q uint8 [rows,cols], scale fp32 [ceil(rows/block_rows), cols/128]) for fp32 x."""
    torch = _torch()
    rows, cols = _dims2(x, "x")
    _need(block_rows in (1, 128), f"blockq_e4m3: block_rows must be 1 or 128, got {block_rows}")
    nscale = ((rows + block_rows - 1) // block_rows) * (cols // 128)
    if q is None:
        q = _empty(stream, (rows, cols), dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = _empty(stream, ((rows + block_rows - 1) // block_rows, cols // 128), dtype=torch.float32,
                       device=x.device)
    _room(q, rows * cols, "q")
    _room(scale, nscale, "scale")
    st = load().blockq_e4m3(_ptr(x, _f32(), "x"), _ptr(q, _u8(), "q"), _ptr(scale, _f32(), "scale"),
                            rows, cols, block_rows, _stream(stream))
    _check(st, "blockq_e4m3")
    return q, scale


def actq_e4m3(x, q=None, scale=None, stream=None):
    """(q uint8 [rows,cols], scale fp32 [rows, cols/128]) = 1x128 e4m3 quantization of bf16 x."""
    torch = _torch()
    rows, cols = _dims2(x, "x")
    if q is None:
        q = _empty(stream, (rows, cols), dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = _empty(stream, (rows, cols // 128), dtype=torch.float32, device=x.device)
    _room(q, rows * cols, "q")
    _room(scale, rows * (cols // 128), "scale")
    st = load().actq_e4m3(_ptr(x, _b16(), "x"), _ptr(q, _u8(), "q"), _ptr(scale, _f32(), "scale"),
                          rows, cols, _stream(stream))
    _check(st, "actq_e4m3")
    return q, scale


def mxgemm_fp8(A, a_scale, B, b_scale, C=None, bands=1, band_stride=0, stream=None):
    """C (bf16) = mx(A [M,K] e4m3, a_scale u8 [M,K/32]) x mx(B [N,K] e4m3, b_scale u8 [N,K/32])^T,
    E8M0 scales per 1x32 block, written as `bands` destination-major row bands."""
    torch = _torch()
    M, N, K = _check_gemm_operands(A, a_scale, B, b_scale, 32, "mxgemm_fp8")
    need = _band_elems(M, N, bands, band_stride)
    if C is None:
        C = _empty(stream, need, dtype=torch.bfloat16, device=A.device)
    _room(C, need, "C")
    st = load().mxgemm_fp8(_ptr(A, _u8(), "A"), _ptr(a_scale, _u8(), "a_scale"),
                           _ptr(B, _u8(), "B"), _ptr(b_scale, _u8(), "b_scale"),
                           _ptr(C, _b16(), "C"), M, N, K, bands, band_stride, _stream(stream))
    _check(st, "mxgemm_fp8")
    return C


def mxq_e4m3(x, q=None, scale=None, stream=None):
    """(q uint8 [rows,cols], scale E8M0 uint8 [rows, cols/32]) = 1x32 mxfp8 quantization of bf16 x."""
    torch = _torch()
    rows, cols = _dims2(x, "x")
    if q is None:
        q = _empty(stream, (rows, cols), dtype=torch.uint8, device=x.device)
    if scale is None:
        scale = _empty(stream, (rows, cols // 32), dtype=torch.uint8, device=x.device)
    _room(q, rows * cols, "q")
    _room(scale, rows * (cols // 32), "scale")
    st = load().mxq_e4m3(_ptr(x, _b16(), "x"), _ptr(q, _u8(), "q"), _ptr(scale, _u8(), "scale"),
                         rows, cols, _stream(stream))
    _check(st, "mxq_e4m3")
    return q, scale


def bprepack_e4m3(B, Bp=None, stream=None):
    """Bp (uint8, N*K bytes) = the weight B [N,K] e4m3 in bsgemm_fp8_pb's operand order."""
    torch = _torch()
    N, K = _dims2(B, "B")
    if Bp is None:
        Bp = _empty(stream, N * K, dtype=torch.uint8, device=B.device)
    _room(Bp, N * K, "Bp")
    st = load().bprepack_e4m3(_ptr(B, _u8(), "B"), _ptr(Bp, _u8(), "Bp"), N, K, _stream(stream))
    _check(st, "bprepack_e4m3")
    return Bp


def bsgemm_fp8_pb(A, a_scale, Bp, b_scale, C=None, bands=1, band_stride=0, stream=None):
    """bsgemm_fp8 with the weight prepacked by bprepack_e4m3 (Bp holds N*K bytes; N is
    taken from b_scale, [N/128, K/128])."""
    torch = _torch()
    M, K = _dims2(A, "A")
    _need(K % 128 == 0, f"bsgemm_fp8_pb: K must be a multiple of 128 (K={K})")
    _need(b_scale.dim() == 2 and b_scale.shape[1] == K // 128,
          f"b_scale: shape {tuple(b_scale.shape)}, expected [N/128, {K // 128}]")
    N = b_scale.shape[0] * 128
    _shape(a_scale, (M, K // 128), "a_scale")
    _need(Bp.numel() == N * K, f"Bp must hold N*K = {N * K} bytes, got {Bp.numel()}")
    need = _band_elems(M, N, bands, band_stride)
    if C is None:
        C = _empty(stream, need, dtype=torch.bfloat16, device=A.device)
    _room(C, need, "C")
    st = load().bsgemm_fp8_pb(_ptr(A, _u8(), "A"), _ptr(a_scale, _f32(), "a_scale"),
                              _ptr(Bp, _u8(), "Bp"), _ptr(b_scale, _f32(), "b_scale"),
                              _ptr(C, _b16(), "C"), M, N, K, bands, band_stride, _stream(stream))
    _check(st, "bsgemm_fp8_pb")
    return C


def band_rowq_e4m3(parts, q=None, scale=None, stream=None):
    """(q uint8 [rows,N], scale fp32 [rows]) = rowq_e4m3(band_reduce(parts)) in one kernel."""
    torch = _torch()
    parts = list(parts)
    _need(len(parts) >= 1, "band_rowq_e4m3: no parts")
    rows, N = _dims2(parts[0], "parts[0]")
    for i, p in enumerate(parts):
        _shape(p, (rows, N), f"parts[{i}]")
    if q is None:
        q = _empty(stream, (rows, N), dtype=torch.uint8, device=parts[0].device)
    if scale is None:
        scale = _empty(stream, (rows,), dtype=torch.float32, device=parts[0].device)
    _room(q, rows * N, "q")
    _room(scale, rows, "scale")
    ptrs = (ctypes.c_void_p * len(parts))(*[_ptr(p, _b16(), "part") for p in parts])
    st = load().band_rowq_e4m3(ptrs, len(parts), _ptr(q, _u8(), "q"), _ptr(scale, _f32(), "scale"),
                               rows, N, _stream(stream))
    _check(st, "band_rowq_e4m3")
    return q, scale


class _Types:
    """The dtypes the calls below take, formed once: such a call costs a few
    microseconds on the host, and a decode step makes many."""

    def __init__(self):
        import torch
        self.torch = torch
        self.u8, self.bytes, self.b16, self.f32 = _u8(), (torch.uint8,), _b16(), _f32()
        self.i32, self.bf, self.resid = (torch.int32,), (torch.bfloat16,), (torch.bfloat16, torch.float32)


_types = None


def _ty():
    global _types
    if _types is None:
        _types = _Types()
    return _types


def _args(what, stream, *args):
    """The pointers of a call's (tensor or None, dtypes, name) arguments, and its
    stream's handle.  The tensors must be on one device, which must be the current
    one, as must a stream that is given: a kernel launched elsewhere would fault
    on their addresses."""
    torch = _ty().torch
    out, dev = [], None
    for t, dtypes, name in args:
        if t is None:
            out.append(None)
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        d = t.get_device()
        if d != dev:
            if d < 0:
                raise ValueError(f"{name} must be a device tensor")
            if dev is not None:
                raise ValueError(f"{what}: tensors on cuda:{dev} and cuda:{d}")
            dev = d
        if t.dtype not in dtypes:
            raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        out.append(t.data_ptr())
    here = torch.cuda.current_device()
    if dev != here:
        raise ValueError(f"{what}: tensors on cuda:{dev}, but the current device is cuda:{here}")
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev)   # current_stream() alone takes 2.7 us
    elif stream.device.index != dev:
        raise ValueError(f"{what}: the stream is on {stream.device}, the tensors on cuda:{dev}")
    else:
        handle = stream.cuda_stream
    return out, handle


def _check_plan(plan, M, L):
    if plan.numel() != L + 2 + M:
        raise ValueError(f"plan: {plan.numel()} elements, expected {L + 2 + M} for {M} rows and {L} adapters")


def _is(t, shape, name):
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _fits(t, n, name):
    if t.numel() < n:
        raise ValueError(f"{name}: {t.numel()} elements, the call writes {n}")


def _matrix(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    return t.shape


def lora_plan(ids, n_adapters, plan=None, stream=None):
    """plan (int32 [n_adapters + 2 + M]) = the rows of ids (int32 [M]) ordered by adapter: group
    starts, then rows (see bsgemm.h); an id outside [0, n_adapters) means no adapter."""
    ty = _ty()
    if not (ids.dim() == 1):
        raise ValueError(f"ids must be 1-D, got shape {tuple(ids.shape)}")
    if not (n_adapters >= 1):
        raise ValueError(f"lora_plan: n_adapters must be at least 1, got {n_adapters}")
    M = ids.shape[0]
    if plan is None:
        plan = _empty(stream, n_adapters + 2 + M, dtype=ty.torch.int32, device=ids.device)
    _check_plan(plan, M, n_adapters)
    p, st = _args("lora_plan", stream, (ids, ty.i32, "ids"), (plan, ty.i32, "plan"))
    _check(load().lora_plan(*p, M, n_adapters, st), "lora_plan")
    return plan


def lora_shrink(x, A, plan, H=None, stream=None):
    """H (fp32 [M,R]) = each row of x (bf16 [M,K]) times its adapter's A (bf16 [n_adapters,R,K])
    transposed, by the plan of lora_plan; zero rows where there is no adapter."""
    ty = _ty()
    M, K = _matrix(x, "x")
    if not (A.dim() == 3 and A.shape[2] == K):
        raise ValueError(f"A: shape {tuple(A.shape)}, expected [n_adapters, R, {K}]")
    L, R, _ = A.shape
    _check_plan(plan, M, L)
    if H is None:
        H = _empty(stream, (M, R), dtype=ty.torch.float32, device=x.device)
    _fits(H, M * R, "H")
    p, st = _args("lora_shrink", stream, (x, ty.bf, "x"), (A, ty.bf, "A"), (plan, ty.i32, "plan"), (H, ty.f32, "H"))
    if M:
        _check(load().lora_shrink(*p, M, K, L, R, st), "lora_shrink")
    return H


def _check_lora(H, B, scale, N, what):
    M, R = _matrix(H, "H")
    if not (B.dim() == 3 and B.shape[2] == R):
        raise ValueError(f"{what}: shape {tuple(B.shape)}, expected [n_adapters, N, {R}]")
    if N is not None:
        if not (B.shape[1] == N):
            raise ValueError(f"{what}: shape {tuple(B.shape)}, expected [n_adapters, {N}, {R}]")
    if scale is not None:
        _is(scale, (B.shape[0],), "scale")
    return M, B.shape[1], B.shape[0], R


def lora_expand(H, B, plan, base, out=None, scale=None, bands=1, band_stride=0, stream=None):
    """out (bf16 bands) = base + scale[a] * (H [M,R] fp32 x B[a]^T), B bf16 [n_adapters,N,R], a each
    row's adapter by the plan; base and out are banded as bsgemm_fp8's C; out=base works in place."""
    ty = _ty()
    M, N, L, R = _check_lora(H, B, scale, None, "B")
    _check_plan(plan, M, L)
    need = _band_elems(M, N, bands, band_stride)
    if not (base.numel() >= need):
        raise ValueError(f"base: {base.numel()} elements, the call reads {need}")
    if out is None:
        out = _empty(stream, need, dtype=ty.torch.bfloat16, device=base.device)
    _fits(out, need, "out")
    p, st = _args("lora_expand", stream, (H, ty.f32, "H"), (B, ty.bf, "B"), (scale, ty.f32, "scale"),
                  (plan, ty.i32, "plan"), (base, ty.bf, "base"), (out, ty.bf, "out"))
    if M:
        _check(load().lora_expand(*p, M, N, L, R, bands, band_stride, st), "lora_expand")
    return out


def bsgemm_fp8_lora(A, a_scale, B, b_scale, H, lora_B, ids, scale=None, C=None, bands=1, band_stride=0,
                    stream=None):
    """bsgemm_fp8 plus scale[a] * (H [M,R] fp32 x lora_B[a]^T) for each row's adapter a = ids[row]
    (lora_B bf16 [n_adapters,N,R]), added in fp32 before the rounding to bf16."""
    ty = _ty()
    M, K = _matrix(A, "A")
    N = _matrix(B, "B")[0]
    if B.shape[1] != K or K % 128 or N % 128:
        raise ValueError(f"bsgemm_fp8_lora: A is [M,{K}], B {tuple(B.shape)}: one K, and K and N multiples of 128")
    _is(a_scale, (M, K // 128), "a_scale")
    _is(b_scale, (N // 128, K // 128), "b_scale")
    Mh, _, L, R = _check_lora(H, lora_B, scale, N, "lora_B")
    if not (Mh == M):
        raise ValueError(f"H: {Mh} rows, A has {M}")
    _is(ids, (M,), "ids")
    need = _band_elems(M, N, bands, band_stride)
    if C is None:
        C = _empty(stream, need, dtype=ty.torch.bfloat16, device=A.device)
    _fits(C, need, "C")
    p, st = _args("bsgemm_fp8_lora", stream, (A, ty.u8, "A"), (a_scale, ty.f32, "a_scale"), (B, ty.u8, "B"),
                  (b_scale, ty.f32, "b_scale"), (H, ty.f32, "H"), (lora_B, ty.bf, "lora_B"), (scale, ty.f32, "scale"),
                  (ids, ty.i32, "ids"), (C, ty.b16, "C"))
    if M:
        _check(load().bsgemm_fp8_lora(*p, M, N, K, L, R, bands, band_stride, st), "bsgemm_fp8_lora")
    return C


def resnorm(y, resid, y_scale=None, post_w=None, gate=None, pre_w=None, alpha=1.0, beta=1.0, eps=1e-6, quant=0,
            resid_out=None, z=None, q=None, q_scale=None, stream=None):
    """(resid_out, z, q, q_scale): h = alpha * resid + beta * gate * norm(y; post_w) as the new residual,
    z = norm(h; pre_w) in bf16, and z's e4m3 codes with 1x128 fp32 (quant=128) or 1x32 E8M0
    (quant=32) scales, in one pass.

    y: bf16 [rows,N], or e4m3 codes with y_scale fp32 [rows] (the fp8 wire).  resid: bf16 or fp32
    [rows,N]; resid_out=resid updates it in place.  post_w, pre_w: bf16 [N] or None (no norm
    after the block; unit weight).  gate: bf16 [N] or [rows,N] or None.  z is written if a
    buffer is given, or (quant=0) always; what is not written is returned as None."""
    ty = _ty()
    torch = ty.torch
    rows, N = _matrix(y, "y")
    _is(resid, (rows, N), "resid")
    if quant not in (0, 32, 128):
        raise ValueError(f"resnorm: quant must be 0, 32 or 128, got {quant}")
    if y_scale is not None and y_scale.numel() != rows:
        raise ValueError(f"y_scale: {y_scale.numel()} elements for {rows} rows")
    if post_w is not None:
        _is(post_w, (N,), "post_w")
    if pre_w is not None:
        _is(pre_w, (N,), "pre_w")
    gate_row = 0
    if gate is not None:
        gate_row = N if gate.dim() == 2 else 0
        _is(gate, (rows, N) if gate_row else (N,), "gate")
    if resid_out is None:
        resid_out = _empty(stream, (rows, N), resid.dtype, resid.device)
    elif resid_out.dtype != resid.dtype:
        raise ValueError(f"resid_out is {resid_out.dtype}, resid is {resid.dtype}")
    n = rows * N
    _fits(resid_out, n, "resid_out")
    if quant:
        if N % quant:
            raise ValueError(f"resnorm: N={N} is not a multiple of quant={quant}")
        if q is None:
            q = _empty(stream, (rows, N), dtype=torch.uint8, device=y.device)
        if q_scale is None:
            q_scale = _empty(stream, (rows, N // quant), dtype=torch.float32 if quant == 128 else torch.uint8,
                             device=y.device)
        _fits(q, n, "q")
        _fits(q_scale, n // quant, "q_scale")
    else:
        if not (q is None and q_scale is None):
            raise ValueError("resnorm: q and q_scale need quant=32 or 128")
        if z is None:
            z = _empty(stream, (rows, N), dtype=torch.bfloat16, device=y.device)
    if z is not None:
        _fits(z, n, "z")
    p, st = _args("resnorm", stream, (y, ty.bf if y_scale is None else ty.u8, "y"), (y_scale, ty.f32, "y_scale"),
                  (resid, ty.resid, "resid"), (post_w, ty.bf, "post_w"), (gate, ty.bf, "gate"), (pre_w, ty.bf, "pre_w"),
                  (resid_out, ty.resid, "resid_out"), (z, ty.bf, "z"), (q, ty.u8, "q"),
                  (q_scale, ty.f32 if quant == 128 else ty.bytes, "q_scale"))
    if rows:
        _check(load().resnorm(*p[:5], gate_row, *p[5:], rows, N, int(resid.dtype is torch.float32), quant, alpha, beta,
                              eps, st), "resnorm")
    return resid_out, z, q, q_scale
