"""The operators that stand around the fp8 projection, in their plain form and
as the library's calls, over the sizes they are used at.

  plan     lora_plan        rows ordered by the adapter each one uses
  shrink   lora_shrink      H[m] = x[m] . A[id(m)]^T
  expand   lora_expand      out[m] = base[m] + scale[id(m)] (H[m] . B[id(m)]^T)
  gemm     bsgemm_fp8_lora  the blockscale fp8 product and its rows' adapters in one
                            pass: C[m] = dequant(A)[m] . dequant(B)^T + scale (H[m] . B_l^T)
  resnorm  resnorm          norm after a block, gate, scaled residual, norm before the
                            next block, and its e4m3 operand with block scales

The sizes are those of the wo_b projection (N = 7168 with K = 2048 per GPU, the mxfp8
one's N = 5120, chunks of up to 16384 rows, a ragged batch's 20096 / 8 rows) and
generic ones around them.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decode step of a batch of requests, a few adapters loaded
        dict(name="plan decode", op="plan", M=64, L=8, mix="tokens"),
        # a full prefill chunk and a server's worth of adapters
        dict(name="plan chunk", op="plan", M=16384, L=64, mix="requests"),
        # decode: each row its own request, small rank
        dict(name="shrink decode", op="shrink", M=64, K=2048, R=16, L=16, mix="tokens"),
        # prefill chunk: requests of many tokens each, the usual largest rank
        dict(name="shrink chunk", op="shrink", M=16384, K=2048, R=64, L=8, mix="requests"),
        # an odd decode batch, adapters mixed row by row
        dict(name="expand decode", op="expand", M=37, N=7168, R=16, L=32, mix="tokens", bands=1),
        # the mxfp8 layer's output (whose product has no fused form), one chunk in 8 bands
        dict(name="expand chunk", op="expand", M=16384, N=5120, R=32, L=8, mix="requests", bands=8),
        # a small mixed batch: one row tile, adapters mixed row by row
        dict(name="gemm mixed", op="gemm", M=200, N=7168, K=2048, R=16, L=4, mix="tokens", bands=1),
        # the prefill chunk of the benchmark's layer with adapters of rank 64
        dict(name="gemm chunk", op="gemm", M=16384, N=7168, K=2048, R=64, L=8, mix="requests", bands=8),
        # one token: the gathered wire row into the residual and the next operand
        dict(name="resnorm token", op="resnorm", rows=1, N=7168, wire=True, post=True, gate="channel",
             resid="bf16", z=False, quant=128),
        # the gathered chunk, as the layer hands it on (no norm after the block, no gate)
        dict(name="resnorm chunk", op="resnorm", rows=16384, N=7168, wire=True, post=False, gate="none",
             resid="bf16", z=False, quant=128),
        # the mxfp8 layer: bf16 block output, fp32 residual stream, norms on both sides
        dict(name="resnorm mx", op="resnorm", rows=4096, N=5120, wire=False, post=True, gate="channel",
             resid="f32", z=True, quant=32),
        # one band of the ragged batch, gated element by element, bf16 result
        dict(name="resnorm band", op="resnorm", rows=2512, N=7168, wire=False, post=True, gate="full",
             resid="bf16", z=True, quant=0),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["plan", "shrink", "expand", "gemm", "resnorm", "resnorm"])
    mix = rng.choice(["tokens", "requests"])
    if op == "plan":
        return dict(op=op, M=_log(rng, 16, 16384), L=_log(rng, 4, 256), mix=mix)
    if op == "resnorm":
        quant = rng.choice([0, 32, 128])
        return dict(op=op, rows=_log(rng, 1, 16384), N=_log(rng, 128, 7168, quant or 8),
                    wire=rng.random() < 0.5, post=rng.random() < 0.5,
                    gate=rng.choice(["none", "channel", "full"]), resid=rng.choice(["bf16", "f32"]),
                    z=quant == 0 or rng.random() < 0.5, quant=quant)
    M, R = _log(rng, 1, 16384), 8 * rng.randint(1, 16)
    L = _log(rng, 1, max(1, 1024 // R))
    if op == "shrink":
        return dict(op=op, M=M, K=_log(rng, 64, 7168, 8), R=R, L=L, mix=mix)
    bands = rng.choice([1, 1, 2, 4, 8])
    M = max(bands, M // bands * bands)
    if op == "expand":
        return dict(op=op, M=M, N=_log(rng, 64, 7168, 8), R=R, L=L, mix=mix, bands=bands)
    return dict(op=op, M=M, N=_log(rng, 128, 7168, 128), K=_log(rng, 128, 2048, 128), R=min(R, 64), L=L, mix=mix,
                bands=bands)


# ----------------------------------------------------------------- inputs --

def _adapter_ids(M, L, mix, gen):
    """int32 [M]: the adapter of every row, -1 for about one request in eight
    that has none.  "tokens": every row a request of its own; "requests": rows
    of one request lie together, with lengths that vary."""
    if mix == "tokens":
        owner = torch.arange(M, device=DEV)
        n = M
    else:
        n = max(1, min(M, 2 * L))
        cut = torch.randint(0, M, (n - 1,), generator=gen, device=DEV).sort().values
        owner = torch.bucketize(torch.arange(M, device=DEV), cut, right=True)
    ids = torch.randint(0, L, (n,), generator=gen, device=DEV)
    none = torch.rand(n, generator=gen, device=DEV) < 0.125
    none[0] = False
    return torch.where(none, -1, ids)[owner].to(torch.int32)


def _plain_plan(ids, L):
    key = torch.where((ids >= 0) & (ids < L), ids, L).to(torch.int64)
    order = torch.argsort(key, stable=True)
    n = torch.zeros(L + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    start = torch.cat([torch.zeros(1, dtype=torch.int64, device=ids.device), n.cumsum(0)])
    return torch.cat([start, order]).to(torch.int32)


def _codes(x, rows, cols):
    """fp32 x as e4m3 codes (uint8) with one fp32 scale for each rows x cols block."""
    R, C = x.shape
    b = x.view(R // rows, rows, C // cols, cols)
    s = b.abs().amax((1, 3)) / 448.0
    q = (b / s.clamp_min(1e-30)[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(R, C).view(torch.uint8), s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)

    op = case["op"]
    st = dict(case)
    if op == "resnorm":
        rows, N = case["rows"], case["N"]
        y = normal(rows, N, dtype=torch.float32)
        if case["wire"]:
            st["y"], s = _codes(y, 1, N)
            st["y_scale"] = s.view(-1)
        else:
            st["y"], st["y_scale"] = y.to(torch.bfloat16), None
        rt = torch.bfloat16 if case["resid"] == "bf16" else torch.float32
        st["resid"] = normal(rows, N, std=3.0, dtype=rt)
        st["post_w"] = (1.0 + normal(N, std=0.1, dtype=torch.float32)).to(torch.bfloat16) if case["post"] else None
        st["pre_w"] = (1.0 + normal(N, std=0.1, dtype=torch.float32)).to(torch.bfloat16)
        st["gate"] = None if case["gate"] == "none" else normal(N) if case["gate"] == "channel" else normal(rows, N)
        st["alpha"], st["beta"], st["eps"] = 0.75, 0.5, 1e-6
        st["resid_out"] = torch.empty_like(st["resid"])
        st["z_out"] = torch.empty(rows, N, dtype=torch.bfloat16, device=DEV) if case["z"] else None
        quant = case["quant"]
        st["q_out"] = torch.empty(rows, N, dtype=torch.uint8, device=DEV) if quant else None
        st["s_out"] = torch.empty(rows, N // quant, dtype=torch.float32 if quant == 128 else torch.uint8,
                                  device=DEV) if quant else None
        return st
    M, L = case["M"], case["L"]
    st["ids"] = _adapter_ids(M, L, case["mix"], gen)
    if op == "plan":
        st["plan"] = torch.empty(L + 2 + M, dtype=torch.int32, device=DEV)
        return st
    R = case["R"]
    st["plan"] = _plain_plan(st["ids"], L)
    if op == "shrink":
        K = case["K"]
        st["x"] = normal(M, K)
        st["A"] = normal(L, R, K, std=K ** -0.5)
        st["H"] = torch.empty(M, R, dtype=torch.float32, device=DEV)
        return st
    N = case["N"]
    st["H"] = normal(M, R, dtype=torch.float32)
    st["B"] = normal(L, N, R, std=0.05)
    st["scale"] = 0.5 + torch.rand(L, generator=gen, device=DEV)
    st["out"] = torch.empty(M * N, dtype=torch.bfloat16, device=DEV)
    if op == "expand":
        st["base"] = normal(M * N)
        return st
    K = case["K"]
    st["qa"], st["sa"] = _codes(normal(M, K, dtype=torch.float32), 1, 128)
    st["qb"], st["sb"] = _codes(normal(N, K, std=0.02, dtype=torch.float32), 128, 128)
    return st


# ------------------------------------------------------------- plain forms --

def _values(q):
    return q.view(torch.float8_e4m3fn).to(torch.float32)


def _plain_pick(wide, ids, L):
    """wide [M, L, R] -> [M, R], each row's own adapter; 0 for a row without one."""
    has = (ids >= 0) & (ids < L)
    at = torch.where(has, ids, 0).to(torch.int64)
    M, _, R = wide.shape
    h = wide.gather(1, at[:, None, None].expand(M, 1, R))[:, 0]
    return torch.where(has[:, None], h, 0.0)


def _plain_delta(s):
    """scale[id] (H . B[id]^T) for every row, one product over all adapters side by side."""
    L, R = s["L"], s["R"]
    ids = s["ids"].to(torch.int64)
    has = (ids >= 0) & (ids < L)
    at = torch.where(has, ids, 0)
    h = torch.where(has[:, None], s["H"] * s["scale"][at][:, None], 0.0)
    own_block = at[:, None] == torch.arange(L, device=ids.device)
    wide = torch.where(own_block[:, :, None], h[:, None, :], 0.0).reshape(-1, L * R)
    return wide @ s["B"].float().permute(0, 2, 1).reshape(L * R, -1)


def _plain_resnorm(s):
    y = _values(s["y"]) * s["y_scale"][:, None] if s["wire"] else s["y"].float()
    if s["post_w"] is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * s["post_w"].float()
    if s["gate"] is not None:
        y = y * s["gate"].float()
    h = s["alpha"] * s["resid"].float() + s["beta"] * y
    z = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + s["eps"]) * s["pre_w"].float()
    out = {"resid": h.to(s["resid"].dtype)}
    if s["z"]:
        out["z"] = z.to(torch.bfloat16)
    if s["quant"]:
        b = z.view(z.shape[0], -1, s["quant"])
        amax = b.abs().amax(-1)
        if s["quant"] == 128:
            sc = amax / 448.0
            out["scale"] = sc
        else:
            m, e = torch.frexp(amax)   # amax = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
            k = (e - 9 + (m > 0.875).to(e.dtype)).clamp_min(-127)
            k = torch.where(amax == 0, -127, k)
            sc = torch.ldexp(torch.ones_like(amax), k)
            out["scale"] = (k + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
        q = torch.where(sc[..., None] == 0, 0.0, b / sc[..., None])
        out["q"] = q.clamp(-448, 448).to(torch.float8_e4m3fn).view(z.shape)
    return out


def run(state):
    s = state
    op = s["op"]
    if own:
        return _own_run(s, op)
    if op == "plan":
        return _plain_plan(s["ids"], s["L"])
    if op == "shrink":
        wide = s["x"].float() @ s["A"].float().view(-1, s["K"]).t()
        return _plain_pick(wide.view(s["M"], s["L"], s["R"]), s["ids"], s["L"])
    if op == "expand":
        return (s["base"].float().view(s["M"], -1) + _plain_delta(s)).to(torch.bfloat16).view(-1)
    if op == "gemm":
        M, N, K = s["M"], s["N"], s["K"]
        a = (_values(s["qa"]).view(M, K // 128, 128) * s["sa"][:, :, None]).view(M, K)
        b = (_values(s["qb"]).view(N // 128, 128, K // 128, 128) * s["sb"][:, None, :, None]).view(N, K)
        return (a @ b.t() + _plain_delta(s)).to(torch.bfloat16).view(-1)
    return _plain_resnorm(s)


def _own_run(s, op):
    import block_scaled_fp8_bsgemm_amd as bs
    if op == "plan":
        return bs.lora_plan(s["ids"], s["L"], s["plan"])
    if op == "shrink":
        return bs.lora_shrink(s["x"], s["A"], s["plan"], s["H"])
    if op == "expand":
        return bs.lora_expand(s["H"], s["B"], s["plan"], s["base"], s["out"], scale=s["scale"], bands=s["bands"])
    if op == "gemm":
        return bs.bsgemm_fp8_lora(s["qa"], s["sa"], s["qb"], s["sb"], s["H"], s["B"], s["ids"], s["scale"], s["out"],
                                  bands=s["bands"])
    r, z, q, sc = bs.resnorm(s["y"], s["resid"], y_scale=s["y_scale"], post_w=s["post_w"], gate=s["gate"],
                             pre_w=s["pre_w"], alpha=s["alpha"], beta=s["beta"], eps=s["eps"], quant=s["quant"],
                             resid_out=s["resid_out"], z=s["z_out"], q=s["q_out"], q_scale=s["s_out"])
    out = {"resid": r}
    if z is not None:
        out["z"] = z
    if q is not None:
        out["q"] = q.view(torch.float8_e4m3fn)
        out["scale"] = sc if s["quant"] == 128 else sc.view(torch.float8_e8m0fnu)
    return out


# ----------------------------------------------------------- work and exact --

def work(case):
    op = case["op"]
    if op == "plan":
        return dict(bytes=4 * (2 * case["M"] + case["L"] + 2), flops=case["M"])
    if op == "resnorm":
        n, N = case["rows"] * case["N"], case["N"]
        per = (1 if case["wire"] else 2) + 2 * (2 if case["resid"] == "bf16" else 4)
        per += 2 * case["z"] + (1 if case["quant"] else 0) + (2 if case["gate"] == "full" else 0)
        extra = 4 * case["rows"] * case["wire"] + 2 * N * (1 + case["post"] + (case["gate"] == "channel"))
        if case["quant"]:
            extra += n // case["quant"] * (4 if case["quant"] == 128 else 1)
        return dict(bytes=n * per + extra, flops=12 * n)
    M, R = case["M"], case["R"]
    used = min(case["L"], M)
    if op == "shrink":
        K = case["K"]
        return dict(bytes=2 * M * K + 2 * used * R * K + 4 * M * R + 8 * M, flops=2 * M * K * R)
    N = case["N"]
    lora = 4 * M * R + 2 * used * R * N + 4 * M
    if op == "expand":
        return dict(bytes=4 * M * N + lora, flops=2 * M * N * R)
    K = case["K"]
    return dict(bytes=M * K + N * K + 2 * M * N + M * K // 32 + lora, flops=2 * M * N * (K + R))


def _exact_rows(case, s, product):
    """product(rows, a) for each adapter a's rows, put in their places; 0 elsewhere."""
    out = None
    ids = s["ids"].cpu()
    for a in range(case["L"]):
        rows = (ids == a).nonzero()[:, 0].to(DEV)
        if len(rows):
            got = product(rows, a)
            if out is None:
                out = torch.zeros(case["M"], got.shape[1], dtype=torch.float64, device=DEV)
            out[rows] = got
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "plan":
        ids, L = s["ids"].tolist(), case["L"]
        groups = [[m for m, i in enumerate(ids) if i == a] for a in range(L)]
        groups.append([m for m, i in enumerate(ids) if not 0 <= i < L])
        start = [0]
        for g in groups:
            start.append(start[-1] + len(g))
        return torch.tensor(start + sum(groups, []), dtype=torch.int32)
    if op == "shrink":
        h = _exact_rows(case, s, lambda rows, a: s["x"][rows].double() @ s["A"][a].double().t())
        return torch.zeros(case["M"], case["R"], dtype=torch.float64) if h is None else h
    if op in ("expand", "gemm"):
        M, N = case["M"], case["N"]
        d = _exact_rows(case, s, lambda rows, a: s["scale"][a].double() * (
            s["H"][rows].double() @ s["B"][a].double().t()))
        if op == "expand":
            base = s["base"].double().view(M, N)
        else:
            base = torch.zeros(M, N, dtype=torch.float64, device=DEV)
            for kb in range(case["K"] // 128):
                k = slice(128 * kb, 128 * kb + 128)
                p = s["qa"][:, k].view(torch.float8_e4m3fn).double() @ s["qb"][:, k].view(torch.float8_e4m3fn).double().t()
                base += p * s["sa"][:, kb, None].double() * s["sb"][:, kb].double().repeat_interleave(128)
        return (base if d is None else base + d).view(-1)
    y = s["y"].view(torch.float8_e4m3fn).double() * s["y_scale"].double()[:, None] if case["wire"] else s["y"].double()
    if case["post"]:
        y = y / (y.pow(2).sum(1, keepdim=True) / case["N"] + s["eps"]).sqrt() * s["post_w"].double()
    h = s["alpha"] * s["resid"].double()
    h = h + s["beta"] * (y if s["gate"] is None else s["gate"].double() * y)
    z = h / (h.pow(2).sum(1, keepdim=True) / case["N"] + s["eps"]).sqrt() * s["pre_w"].double()
    out = {"resid": h}
    if case["z"]:
        out["z"] = z
    if case["quant"]:
        b = z.view(z.shape[0], -1, case["quant"])
        sc = b.abs().amax(2) / 448.0
        if case["quant"] == 32:
            sc = torch.exp2(torch.log2(sc).ceil())
        out["scale"] = sc
        out["q"] = (b / sc[:, :, None]).view(z.shape)   # before its rounding to e4m3
    return out
