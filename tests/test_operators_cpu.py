"""lora_plan, lora_shrink, lora_expand, bsgemm_fp8_lora and resnorm without a
GPU: the C entry points refuse malformed calls before any launch, and the
binding refuses tensors of the wrong shape, type or device.  Every call here is
refused or has no rows, since the pointers are fake."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
import opsref

INV, UNS, OK = bs.BS_ERR_INVALID, bs.BS_ERR_UNSUPPORTED, bs.BS_OK
P = 0x1000000   # fake, aligned "device" addresses, 16 MiB apart
ADDR = [P * (i + 1) for i in range(12)]
u8, f32, b16, i32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def L():
    return bs.load()


def plan(L, ids=ADDR[0], plan=ADDR[1], M=64, n=8):
    return L.lora_plan(ids, plan, M, n, None)


def test_plan_refusals(L):
    assert plan(L, ids=0) == INV and plan(L, plan=0) == INV and plan(L, ids=0, plan=0, M=0) == INV
    assert plan(L, M=-1) == INV and plan(L, n=0) == INV and plan(L, n=-4) == INV
    assert plan(L, M=1 << 30) == UNS and plan(L, n=4097) == UNS
    assert plan(L, ids=ADDR[0] + 2) == UNS and plan(L, plan=ADDR[1] + 1) == UNS
    assert plan(L, plan=ADDR[0] + 128) == INV and plan(L, plan=ADDR[0] - 8) == INV


def shrink(L, x=ADDR[0], A=ADDR[1], plan=ADDR[2], H=ADDR[3], M=64, K=256, n=8, R=16):
    return L.lora_shrink(x, A, plan, H, M, K, n, R, None)


def test_shrink_refusals(L):
    for k in ("x", "A", "plan", "H"):
        assert shrink(L, **{k: 0}) == INV
    assert shrink(L, M=-1) == INV and shrink(L, K=0) == INV and shrink(L, n=0) == INV and shrink(L, R=0) == INV
    assert shrink(L, K=252) == UNS and shrink(L, R=12) == UNS and shrink(L, R=264) == UNS
    assert shrink(L, K=(1 << 22) + 8) == UNS and shrink(L, M=1 << 30) == UNS and shrink(L, n=4097) == UNS
    for k, i in (("x", 0), ("A", 1), ("H", 3)):
        assert shrink(L, **{k: ADDR[i] + 8}) == UNS
    assert shrink(L, plan=ADDR[2] + 2) == UNS
    assert shrink(L, H=ADDR[0] + 64) == INV and shrink(L, H=ADDR[1]) == INV and shrink(L, H=ADDR[2] + 16) == INV
    assert shrink(L, M=0) == OK


def expand(L, H=ADDR[0], B=ADDR[1], s=ADDR[2], plan=ADDR[3], base=ADDR[4], out=ADDR[5], M=64, N=512, n=8, R=16,
           bands=1, stride=0):
    return L.lora_expand(H, B, s, plan, base, out, M, N, n, R, bands, stride, None)


def test_expand_refusals(L):
    for k in ("H", "B", "plan", "base", "out"):
        assert expand(L, **{k: 0}) == INV
    assert expand(L, N=0) == INV and expand(L, bands=0) == INV and expand(L, stride=-8) == INV
    assert expand(L, N=516) == UNS and expand(L, bands=65, M=65) == UNS and expand(L, bands=3) == UNS
    assert expand(L, bands=2, stride=32 * 512 - 8) == UNS and expand(L, bands=2, stride=32 * 512 + 4) == UNS
    for k, i in (("H", 0), ("B", 1), ("base", 4), ("out", 5)):
        assert expand(L, **{k: ADDR[i] + 8}) == UNS
    assert expand(L, s=ADDR[2] + 2) == UNS
    assert expand(L, out=ADDR[4] + 16) == INV          # neither base itself nor clear of it
    for k in (0, 1, 2, 3):
        assert expand(L, out=ADDR[k]) == INV
    assert expand(L, base=ADDR[4], out=ADDR[4], M=0) == OK and expand(L, s=0, M=0) == OK


def gemm(L, a=ADDR, M=256, N=512, K=256, n=8, R=16, bands=1, stride=0):
    return L.bsgemm_fp8_lora(*a[:9], M, N, K, n, R, bands, stride, None)


def test_gemm_refusals(L):
    def at(i, v):
        return ADDR[:i] + [v] + ADDR[i + 1:]
    for i in (0, 1, 2, 3, 4, 5, 7, 8):
        assert gemm(L, at(i, 0)) == INV, i
    assert gemm(L, M=-1) == INV and gemm(L, N=0) == INV and gemm(L, n=0) == INV and gemm(L, bands=0) == INV
    assert gemm(L, N=520) == UNS and gemm(L, K=264) == UNS and gemm(L, R=20) == UNS and gemm(L, R=512) == UNS
    assert gemm(L, bands=3) == UNS and gemm(L, n=5000) == UNS
    for i in (0, 2, 4, 5, 8):
        assert gemm(L, at(i, ADDR[i] + 8)) == UNS, i
    for i in (0, 1, 2, 3, 4, 5, 6, 7):
        assert gemm(L, at(8, ADDR[i])) == INV, i
    assert gemm(L, M=0) == OK and gemm(L, at(6, 0), M=0) == OK


def norm(L, y=ADDR[0], ys=0, resid=ADDR[1], post=ADDR[2], gate=ADDR[3], grow=0, pre=ADDR[4], out=ADDR[5],
         z=ADDR[6], q=0, qs=0, rows=64, N=512, f32=0, qb=0, alpha=1.0, beta=1.0, eps=1e-6):
    return L.resnorm(y, ys, resid, post, gate, grow, pre, out, z, q, qs, rows, N, f32, qb, alpha, beta, eps, None)


def test_resnorm_refusals(L):
    for k in ("y", "resid", "out"):
        assert norm(L, **{k: 0}) == INV
    assert norm(L, rows=-1) == INV and norm(L, N=0) == INV and norm(L, f32=2) == INV and norm(L, grow=-512) == INV
    for e in (0.0, -1e-6, float("nan"), float("inf")):
        assert norm(L, eps=e) == INV
    assert norm(L, alpha=float("nan")) == INV and norm(L, beta=float("inf")) == INV
    assert norm(L, N=516) == UNS and norm(L, N=16392) == UNS and norm(L, grow=256) == UNS
    q = dict(q=ADDR[7], qs=ADDR[8])
    assert norm(L, qb=64, **q) == UNS and norm(L, qb=128, N=544, **q) == UNS and norm(L, qb=32, N=520, **q) == UNS
    assert norm(L, qb=128) == INV and norm(L, **q) == INV and norm(L, qb=32, q=ADDR[7]) == INV
    for k, i in (("y", 0), ("resid", 1), ("post", 2), ("gate", 3), ("pre", 4), ("out", 5), ("z", 6)):
        assert norm(L, **{k: ADDR[i] + 8}) == UNS, k
    assert norm(L, qb=128, q=ADDR[7], qs=ADDR[8] + 2) == UNS
    assert norm(L, out=ADDR[0]) == INV and norm(L, out=ADDR[1] + 16) == INV and norm(L, z=ADDR[1]) == INV
    assert norm(L, z=ADDR[5] + 16) == INV and norm(L, qb=128, q=ADDR[6], qs=ADDR[8]) == INV
    assert norm(L, qb=128, q=ADDR[7], qs=ADDR[7]) == INV and norm(L, z=ADDR[4]) == INV
    assert norm(L, out=ADDR[1], rows=0) == OK and norm(L, qb=32, rows=0, q=ADDR[7], qs=ADDR[8] + 1) == OK


def t(*shape, dtype=b16):
    return torch.zeros(shape, dtype=dtype)


def refused(match, fn, *a, **kw):
    with pytest.raises((ValueError, TypeError)) as e:
        fn(*a, **kw)
    assert match in str(e.value), str(e.value)


def test_binding_refusals():
    ids, pl = t(64, dtype=i32), t(8 + 2 + 64, dtype=i32)
    x, A, H, B = t(64, 256), t(8, 16, 256), t(64, 16, dtype=f32), t(8, 512, 16)
    base = t(64 * 512)
    refused("1-D", bs.lora_plan, t(8, 8, dtype=i32), 8)
    refused("n_adapters", bs.lora_plan, ids, 0)
    refused("plan:", bs.lora_plan, ids, 8, t(64, dtype=i32))
    refused("device tensor", bs.lora_plan, ids, 8)
    refused("A:", bs.lora_shrink, x, t(8, 16, 128), pl)
    refused("A:", bs.lora_shrink, x, t(128, 256), pl)
    refused("plan:", bs.lora_shrink, x, A, t(64, dtype=i32))
    refused("H:", bs.lora_shrink, x, A, pl, t(64, 8, dtype=f32))
    refused("device tensor", bs.lora_shrink, x, A, pl)
    refused("B:", bs.lora_expand, H, t(8, 512, 32), pl, base)
    refused("plan:", bs.lora_expand, H, B, t(70, dtype=i32), base)
    refused("base:", bs.lora_expand, H, B, pl, t(64 * 511))
    refused("base:", bs.lora_expand, H, B, pl, base, bands=2, band_stride=32 * 512 + 8)
    refused("out:", bs.lora_expand, H, B, pl, base, t(100))
    refused("scale:", bs.lora_expand, H, B, pl, base, scale=t(4, dtype=f32))
    refused("device tensor", bs.lora_expand, H, B, pl, base)
    g = (t(64, 256, dtype=u8), t(64, 2, dtype=f32), t(512, 256, dtype=u8), t(4, 2, dtype=f32))
    refused("a_scale", bs.bsgemm_fp8_lora, g[0], t(64, 3, dtype=f32), *g[2:], H, B, ids)
    refused("b_scale", bs.bsgemm_fp8_lora, *g[:3], t(2, 4, dtype=f32), H, B, ids)
    refused("one K", bs.bsgemm_fp8_lora, *g[:2], t(512, 128, dtype=u8), g[3], H, B, ids)
    refused("multiples", bs.bsgemm_fp8_lora, *g[:2], t(500, 256, dtype=u8), g[3], H, B, ids)
    refused("A must", bs.bsgemm_fp8_lora, g[0].view(-1), *g[1:], H, B, ids)
    refused("H:", bs.bsgemm_fp8_lora, *g, t(32, 16, dtype=f32), B, ids)
    refused("lora_B:", bs.bsgemm_fp8_lora, *g, H, t(8, 256, 16), ids)
    refused("ids:", bs.bsgemm_fp8_lora, *g, H, B, t(63, dtype=i32))
    refused("C:", bs.bsgemm_fp8_lora, *g, H, B, ids, C=t(64 * 512 - 1))
    refused("device tensor", bs.bsgemm_fp8_lora, *g, H, B, ids)
    y = t(64, 512)
    refused("resid:", bs.resnorm, y, t(64, 256))
    refused("quant", bs.resnorm, y, y, quant=64)
    refused("multiple", bs.resnorm, t(4, 136), t(4, 136), quant=32)
    refused("y_scale", bs.resnorm, t(64, 512, dtype=u8), y, y_scale=t(32, dtype=f32))
    refused("post_w", bs.resnorm, y, y, post_w=t(256))
    refused("pre_w", bs.resnorm, y, y, pre_w=t(1, 512))
    refused("gate", bs.resnorm, y, y, gate=t(64, 1))
    refused("gate", bs.resnorm, y, y, gate=t(64))
    refused("resid_out", bs.resnorm, y, y, resid_out=t(64, 512, dtype=f32))
    refused("resid_out", bs.resnorm, y, y, resid_out=t(10, 512))
    refused("q_scale:", bs.resnorm, y, y, quant=128, q_scale=t(64, 3, dtype=f32))
    refused("need quant", bs.resnorm, y, y, q=t(64, 512, dtype=u8))
    refused("z:", bs.resnorm, y, y, z=t(63, 512))
    refused("device tensor", bs.resnorm, y, y)


def test_reference_plan():
    """The reference of the GPU tests on a case worked by hand."""
    ids = np.array([2, -1, 0, 2, 7, 0, 2])
    assert opsref.plan(ids, 3).tolist() == [0, 2, 2, 5, 7, 2, 5, 0, 3, 6, 1, 4]


@pytest.mark.parametrize("block", [32, 128])
def test_reference_quant_check_finds_mistakes(block):
    """check_quant passes the definition's own codes and fails a code one step
    off, a scale two steps of fp32 off and a scale of the wrong power."""
    z = np.random.default_rng(0).standard_normal((8, 256))
    amax = np.abs(z.reshape(8, -1, block)).max(2)
    s = np.float32(amax / 448).astype(float) if block == 128 else 2.0 ** np.ceil(np.log2(amax / 448))
    v = (z.reshape(8, -1, block) / s[..., None]).reshape(z.shape)
    q = torch.from_numpy(v).clamp(-448, 448).float().to(torch.float8_e4m3fn).view(u8).numpy()
    ez = np.full_like(z, 1e-12)
    opsref.check_quant(q, s, z, ez, block)
    off = q.copy()
    off[3, 77] ^= 1
    with pytest.raises(AssertionError, match="codes"):
        opsref.check_quant(off, s, z, ez, block)
    with pytest.raises(AssertionError, match="scales"):
        opsref.check_quant(q, s * (2.0 if block == 32 else 1 + 2.0 ** -22), z, ez, block)
