"""GPU parity of the adapter operators (lora_plan, lora_shrink, lora_expand,
bsgemm_fp8_lora) against plain float64 implementations (opsref.py).  Integer
inputs whose sums fp32 holds exactly are compared bit for bit; random ones
within bounds derived from the arithmetic.  Outputs are poisoned first and lie
between guard elements that no call may touch."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
import opsref
import oracle
import synth
from gpuutil import bits16, device, poison_bf16, say, to_dev
from oracle import bounds

pytestmark = pytest.mark.gpu

MIXES = ("tokens", "requests", "one", "none", "wild")


def make_ids(M, L, mix, seed=0):
    """Rows of one request each, runs of rows, all one adapter, none at all, and
    ids of every value that means none."""
    rng = np.random.default_rng(seed)
    if mix == "one":
        return np.full(M, L - 1, np.int32)
    if mix == "none":
        return np.full(M, -1, np.int32)
    if mix == "tokens":
        return rng.integers(-1, L, M).astype(np.int32)
    if mix == "wild":
        bad = np.array([-1, L, L + 1, -2**31, 2**31 - 1, 1 << 20])
        ids = rng.integers(0, L, M)
        return np.where(rng.random(M) < 0.5, rng.choice(bad, M), ids).astype(np.int32)
    cut = np.sort(rng.integers(0, M + 1, max(1, min(2 * L, M))))
    return rng.integers(-1, L, len(cut) + 1)[np.searchsorted(cut, np.arange(M), side="right")].astype(np.int32)


def guarded(n, dtype, fill):
    """A buffer of n elements between 64 guard elements on either side."""
    full = torch.full((n + 128,), fill, dtype=dtype, device=device())
    return full, full[64:64 + n]


def check_guards(full, fill):
    g = torch.cat([full[:64], full[-64:]])
    assert bool((g == fill).all()), "guard elements were written"


def bf(x):
    return to_dev(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


def values(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------- plan --

@pytest.mark.parametrize("M,L", [(0, 3), (1, 1), (1, 300), (63, 4), (64, 8), (65, 64), (1023, 65), (1025, 7),
                                 (16384, 64), (16385, 3), (40001, 129), (20096, 1000)])
def test_plan(M, L):
    for mix in MIXES:
        say(f"lora_plan M={M} L={L} {mix}")
        ids = make_ids(M, L, mix, M + L)
        full, out = guarded(L + 2 + M, torch.int32, -77)
        bs.lora_plan(to_dev(ids), L, out)
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy(), opsref.plan(ids, L)), mix
        check_guards(full, -77)


# ----------------------------------------------------------------- shrink --

def run_shrink(x, A, ids):
    L, R, _ = A.shape
    full, H = guarded(x.shape[0] * R, torch.float32, -3.0)
    H.fill_(float("nan"))
    plan = to_dev(opsref.plan(ids, L))
    bs.lora_shrink(x, A, plan, H.view(-1, R))
    torch.cuda.synchronize()
    check_guards(full, -3.0)
    return H.view(-1, R)


SHRINK = [(1, 256, 1, 8), (1, 7168, 4, 16), (3, 8, 2, 24), (17, 72, 3, 16), (64, 2048, 16, 16), (65, 2040, 70, 64),
          (200, 520, 5, 128), (257, 1000, 2, 256), (1000, 136, 9, 40), (2100, 512, 3, 64), (4500, 200, 5, 72)]


@pytest.mark.parametrize("M,K,L,R", SHRINK)
def test_shrink_exact_integers(M, K, L, R):
    """Integers up to 4: every partial sum is below 2^24, so H is exact in any order."""
    rng = np.random.default_rng(M)
    x, A = rng.integers(-4, 5, (M, K)), rng.integers(-4, 5, (L, R, K))
    for mix in MIXES:
        say(f"lora_shrink exact M={M} K={K} L={L} R={R} {mix}")
        ids = make_ids(M, L, mix, M)
        H = run_shrink(bf(x), bf(A), ids)
        want, _ = opsref.shrink(x.astype(float), A.astype(float), ids)
        assert np.array_equal(values(H), want), mix


@pytest.mark.parametrize("M,K,L,R", [(64, 2048, 16, 16), (300, 7168, 4, 64), (2100, 2048, 4, 64)])
def test_shrink_random(M, K, L, R):
    say(f"lora_shrink random M={M} K={K} L={L} R={R}")
    rng = np.random.default_rng(M)
    x, A = bf(rng.standard_normal((M, K))), bf(rng.standard_normal((L, R, K)) * K ** -0.5)
    ids = make_ids(M, L, "tokens", 1)
    H = run_shrink(x, A, ids)
    want, bound = opsref.shrink(values(x), values(A), ids)
    err = np.abs(values(H) - want)
    say(f"  relL2 {np.linalg.norm(err) / np.linalg.norm(want):.2e}, largest share of the bound "
        f"{np.max(err / np.maximum(bound, 1e-300)):.3f}")
    assert np.all(err <= bound)
    again = run_shrink(x, A, ids)
    assert torch.equal(H.view(torch.int32), again.view(torch.int32))


def test_shrink_adapters_past_32_bits():
    """An adapter stack of more than 2^32 bytes, its last adapter used."""
    L, R, K = 513, 256, 16400
    say("lora_shrink beyond 2^32 bytes of adapters")
    A = torch.zeros((L, R, K), dtype=torch.bfloat16, device=device())
    rng = np.random.default_rng(0)
    last = rng.integers(-3, 4, (2, R, K))
    A[0], A[L - 1] = bf(last[0]), bf(last[1])
    x = rng.integers(-3, 4, (20, K))
    ids = np.where(np.arange(20) % 3 == 0, 0, L - 1).astype(np.int32)
    H = run_shrink(bf(x), A, ids)
    want = np.where((ids == 0)[:, None], x @ last[0].T, x @ last[1].T)
    assert np.array_equal(values(H), want)


def test_shrink_ignores_what_a_plan_may_not_say():
    """Starts and rows outside the batch, as in a buffer that no lora_plan wrote,
    lead to no access outside it: rows in range are written, the guards stand."""
    say("lora_shrink with a plan out of range")
    M, K, L, R = 40, 64, 3, 16
    x, A = bf(np.ones((M, K))), bf(np.ones((L, R, K)))
    pl = opsref.plan(make_ids(M, L, "tokens"), L)
    pl[1] = -5
    pl[2] = 2**31 - 1
    pl[L + 2:] = np.where(np.arange(M) % 2, 2**30, pl[L + 2:])
    full, H = guarded(M * R, torch.float32, -3.0)
    bs.lora_shrink(x, A, to_dev(pl), H.view(M, R))
    torch.cuda.synchronize()
    check_guards(full, -3.0)


# ----------------------------------------------------------------- expand --

def band_index(M, N, bands, stride):
    """Element of C for each (m, n), [M, N]."""
    rows = M // bands
    s = stride or rows * N
    m = np.arange(M)
    return ((m // rows) * s + (m % rows) * N)[:, None] + np.arange(N)[None, :]


def run_expand(H, B, ids, base, scale=None, bands=1, stride=0, inplace=False):
    """out's values [M, N] for base values [M, N]; gaps and guards checked."""
    M, N = base.shape
    L = B.shape[0]
    at = band_index(M, N, bands, stride)
    n = int(at.max()) + 1
    flat = torch.full((n,), 5.0, dtype=torch.bfloat16, device=device())
    idx = to_dev(at.reshape(-1))
    flat[idx] = base.reshape(-1)
    full, out = guarded(n, torch.bfloat16, -3.0)
    if inplace:
        out.copy_(flat)
    plan = to_dev(opsref.plan(ids, L))
    bs.lora_expand(H, B, plan, out if inplace else flat, out, scale=scale, bands=bands, band_stride=stride)
    torch.cuda.synchronize()
    check_guards(full, -3.0)
    gaps = np.ones(n, bool)
    gaps[at.reshape(-1)] = False
    if gaps.any():
        assert bool((out[to_dev(gaps)] == (5.0 if inplace else -3.0)).all()), "elements between bands were written"
    return out[idx].view(M, N)


EXPAND = [(1, 8, 1, 8, 1, 0), (1, 7168, 3, 16, 1, 0), (37, 1000, 32, 16, 1, 0), (48, 264, 5, 40, 4, 12 * 264 + 64),
          (64, 512, 70, 64, 8, 0), (300, 136, 4, 128, 3, 100 * 136 + 8), (90, 512, 2, 256, 1, 0),
          (2100, 520, 3, 64, 7, 0), (4500, 72, 5, 24, 1, 0), (1000, 2312, 4, 24, 8, 125 * 2312 + 8),
          (300, 7168, 3, 128, 1, 0), (290, 7688, 2, 256, 2, 145 * 7688 + 8), (2400, 7176, 3, 40, 1, 0)]


@pytest.mark.parametrize("M,N,L,R,bands,stride", EXPAND)
def test_expand_exact_integers(M, N, L, R, bands, stride):
    """H up to 2^12 needs both of its bf16 parts, B and base are small, scales are
    powers of two: every sum is exact in fp32 and out is its bf16 rounding."""
    rng = np.random.default_rng(M + N)
    H, B = rng.integers(-4096, 4097, (M, R)), rng.integers(-2, 3, (L, N, R))
    base = rng.integers(-200, 201, (M, N))
    scale = 2.0 ** rng.integers(-2, 3, L)
    for mix in MIXES:
        for inplace in (False, True):
            say(f"lora_expand exact M={M} N={N} L={L} R={R} bands={bands} {mix} inplace={inplace}")
            ids = make_ids(M, L, mix, N)
            d, _ = opsref.delta(H.astype(float), B.astype(float), scale, ids)
            Hd = to_dev(H.astype(np.float32))
            Hd[to_dev((ids < 0) | (ids >= L))] = float("nan")   # not to be read
            got = run_expand(Hd, bf(B), ids, bf(base), to_dev(scale.astype(np.float32)), bands, stride, inplace)
            assert np.array_equal(values(got), bounds.bf16_rne_f64(base + d)), mix


@pytest.mark.parametrize("M,N,L,R,scaled", [(37, 7168, 8, 16, True), (600, 1000, 3, 64, False)])
def test_expand_random(M, N, L, R, scaled):
    """Within the bf16 interval of base + delta, delta off by its derived bound and
    the final fp32 addition by u."""
    say(f"lora_expand random M={M} N={N} L={L} R={R}")
    rng = np.random.default_rng(N)
    H, B = to_dev(rng.standard_normal((M, R)).astype(np.float32)), bf(rng.standard_normal((L, N, R)) * 0.05)
    base = bf(rng.standard_normal((M, N)))
    scale = to_dev((0.5 + rng.random(L)).astype(np.float32)) if scaled else None
    ids = make_ids(M, L, "requests", 2)
    d, bound = opsref.delta(values(H), values(B), None if scale is None else values(scale), ids)
    want = values(base) + d
    got = run_expand(H, B, ids, base, scale)
    ok, used = bounds.within(bits16(got), want, bound + opsref.U * np.abs(want))
    say(f"  largest share of the interval {used.max():.3f}")
    assert ok.all()
    none = (ids < 0) | (ids >= L)
    assert torch.equal(got[to_dev(none)].view(torch.int16), base[to_dev(none)].view(torch.int16))


# ------------------------------------------------------ GEMM with adapters --

def gemm_operands(M, N, K, seed, ints):
    if ints:   # codes of small integers, unit scales: exact sums
        rng = np.random.default_rng(seed)
        code = torch.arange(-4, 5).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        qa, qb = code[rng.integers(0, 9, (M, K))], code[rng.integers(0, 9, (N, K))]
        return qa, np.ones((M, K // 128), np.float32), qb, np.ones((N // 128, K // 128), np.float32)
    A, B = synth.operand_fp32(M, N, K, seed=seed, heavy=M >= 200)
    return (*oracle.quant_blocks(A, 1, 128), *oracle.quant_blocks(B, 128, 128))


def run_gemm(ops, H, B, ids, scale, bands, stride, L):
    M, N = ops[0].shape[0], ops[2].shape[0]
    at = band_index(M, N, bands, stride)
    n = int(at.max()) + 1
    full, C = guarded(n, torch.bfloat16, -3.0)
    Hd = to_dev(H.astype(np.float32))
    Hd[to_dev((ids < 0) | (ids >= L))] = float("nan")
    bs.bsgemm_fp8_lora(*ops, Hd, B, to_dev(ids), scale, C, bands=bands, band_stride=stride)
    torch.cuda.synchronize()
    check_guards(full, -3.0)
    gaps = np.ones(n, bool)
    gaps[at.reshape(-1)] = False
    if gaps.any():
        assert bool((C[to_dev(gaps)] == -3.0).all()), "elements between bands were written"
    return C[to_dev(at.reshape(-1))].view(M, N)


GEMM = [(1, 128, 128, 1, 8, 1, 0), (1, 7168, 2048, 16, 16, 1, 0), (15, 384, 640, 20, 40, 5, 3 * 384 + 8),
        (17, 256, 896, 2, 64, 1, 0), (33, 1152, 512, 40, 24, 3, 0), (64, 640, 384, 64, 72, 8, 0),
        (65, 512, 256, 3, 128, 13, 5 * 512 + 16), (256, 768, 1024, 5, 16, 2, 0), (257, 768, 1024, 5, 16, 1, 0), (16, 128, 256, 3, 16, 1, 0), (200, 384, 256, 4, 16, 4, 50 * 384 + 64),
        (300, 640, 384, 70, 64, 3, 0), (513, 512, 1152, 5, 128, 1, 0), (1040, 1280, 512, 2, 40, 8, 0),
        (520, 1024, 384, 3, 48, 4, 0), (264, 1024, 128, 3, 16, 1, 0), (1000, 1024, 256, 9, 72, 5, 0),
        (700, 2176, 640, 70, 32, 7, 100 * 2176 + 8), (1537, 1280, 896, 4, 8, 1, 0), (2050, 2304, 128, 3, 16, 1, 0), (2100, 2304, 384, 4, 72, 7, 0),
        (2600, 5120, 256, 6, 24, 8, 0), (2056, 2304, 512, 9, 256, 8, 257 * 2304 + 8)]


@pytest.mark.parametrize("M,N,K,L,R,bands,stride", GEMM)
def test_gemm_exact_integers(M, N, K, L, R, bands, stride):
    qa, sa, qb, sb = gemm_operands(M, N, K, M, True)
    rng = np.random.default_rng(M)
    H, B = rng.integers(-1024, 1025, (M, R)), rng.integers(-2, 3, (L, N, R))
    scale = 2.0 ** rng.integers(-2, 3, L)
    v = opsref.e4m3_values()
    acc = (v[qa].astype(np.float32) @ v[qb].astype(np.float32).T).astype(float)   # sums below 2^24: exact
    ops = tuple(to_dev(a) for a in (qa, sa, qb, sb))
    plain = bs.bsgemm_fp8(*ops).view(M, N)
    Bd, sd = bf(B), to_dev(scale.astype(np.float32))
    for mix in MIXES:
        say(f"bsgemm_fp8_lora exact M={M} N={N} K={K} L={L} R={R} bands={bands} {mix}")
        ids = make_ids(M, L, mix, N)
        got = run_gemm(ops, H, Bd, ids, sd, bands, stride, L)
        d, _ = opsref.delta(H.astype(float), B.astype(float), scale, ids)
        assert np.array_equal(values(got), bounds.bf16_rne_f64(acc + d)), mix
        none = to_dev((ids < 0) | (ids >= L))
        assert torch.equal(got[none].view(torch.int16), plain[none].view(torch.int16))


@pytest.mark.parametrize("M,N,K,L,R", [(5, 384, 1152, 4, 48), (200, 512, 256, 4, 16), (700, 1024, 640, 3, 64), (1300, 1280, 512, 8, 32),
                                         (2300, 2304, 640, 3, 136)])
def test_gemm_random(M, N, K, L, R):
    """Inside the fp8 product's interval, widened by the low-rank product's bound and
    2R fp32 additions onto the accumulator."""
    say(f"bsgemm_fp8_lora random M={M} N={N} K={K} L={L} R={R}")
    qa, sa, qb, sb = gemm_operands(M, N, K, 3, False)
    rng = np.random.default_rng(5)
    H = rng.standard_normal((M, R)).astype(np.float32)
    B = bf(rng.standard_normal((L, N, R)) * 0.05)
    scale = (0.5 + rng.random(L)).astype(np.float32)
    ids = make_ids(M, L, "tokens", 4)
    ops = tuple(to_dev(a) for a in (qa, sa, qb, sb))
    got = run_gemm(ops, H, B, ids, to_dev(scale), 1, 0, L)
    acc, _ = oracle.bsgemm(qa, sa, qb, sb)
    d, bound = opsref.delta(H.astype(float), values(B), scale, ids)
    own = bounds.BsgemmBound(qa, sa, qb, sb).rows(0, M)
    want = acc.astype(float) + d
    tol = own + bound + 4 * opsref.U * R * (np.abs(acc) + own)
    ok, used = bounds.within(bits16(got), want, tol)
    say(f"  largest share of the interval {used.max():.3f}")
    assert ok.all()
    plain = bs.bsgemm_fp8(*ops).view(M, N)
    none = to_dev((ids < 0) | (ids >= L))
    assert torch.equal(got[none].view(torch.int16), plain[none].view(torch.int16))
    again = run_gemm(ops, H, B, ids, to_dev(scale), 1, 0, L)
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))


def test_gemm_full_size_against_its_parts():
    """The benchmark's chunk (M=16384, N=7168, K=2048, 8 bands) against bsgemm_fp8 in
    fp32 bounds: rows without an adapter bit for bit, the others within one bf16
    rounding of bsgemm_fp8's own (rounded) output plus the float64 delta."""
    M, N, K, L, R = 16384, synth.HIDDEN, synth.K_SHARD, 8, 64
    say("bsgemm_fp8_lora full size")
    g = torch.Generator(device=device()).manual_seed(0)
    x = torch.randn((M, K), generator=g, device=device())
    w = torch.randn((N, K), generator=g, device=device()) * 0.02
    qa, sa = bs.blockq_e4m3(x, 1)
    qb, sb = bs.blockq_e4m3(w, 128)
    H = torch.randn((M, R), generator=g, device=device())
    B = (torch.randn((L, N, R), generator=g, device=device()) * 0.05).to(torch.bfloat16)
    scale = torch.rand(L, generator=g, device=device()) + 0.5
    ids = make_ids(M, L, "requests", 3)
    plain = bs.bsgemm_fp8(qa, sa, qb, sb, bands=8).view(M, N)
    C = poison_bf16(torch.empty(M * N, dtype=torch.bfloat16, device=device()))
    bs.bsgemm_fp8_lora(qa, sa, qb, sb, H, B, to_dev(ids), scale, C, bands=8)
    torch.cuda.synchronize()
    C = C.view(M, N)
    for a in range(-1, L):
        rows = to_dev(np.flatnonzero(ids == a))
        if not len(rows):
            continue
        if a < 0:
            assert torch.equal(C[rows].view(torch.int16), plain[rows].view(torch.int16))
            continue
        p, c = plain[rows].double(), C[rows].double()
        d = scale[a].double() * (H[rows].double() @ B[a].double().t())
        S = scale[a].double() * (H[rows].double().abs() @ B[a].double().abs().t())
        # half a bf16 step (2^-9 of the value at most, counted as 2^-8) of each rounding,
        # and opsref.delta's bound with the 2R additions onto the accumulator
        tol = 2.0 ** -8 * (p.abs() + c.abs()) + (2.0 ** -17 + 4 * opsref.U * R) * (S + p.abs()) + 1e-30
        assert bool(((c - p - d).abs() <= tol).all()), a


# ------------------------------------------------------------ rows apart --

@pytest.mark.parametrize("M,N,K", [(50, 256, 256), (700, 512, 256), (1100, 1152, 256), (2300, 2304, 384)])
def test_what_is_not_finite_stays_in_its_rows(M, N, K):
    """One adapter's weights are NaN and infinite, one row's input is NaN, and rows of no
    adapter hold NaN in H: those rows come out non-finite, every other one as it does without."""
    say(f"not finite: M={M} N={N} K={K}")
    L, R = 5, 40
    rng = np.random.default_rng(M)
    ids = rng.integers(-1, L, M).astype(np.int32)
    x, A = bf(rng.standard_normal((M, K))), bf(rng.standard_normal((L, R, K)))
    B = bf(rng.standard_normal((L, N, R)))
    ops = tuple(to_dev(a) for a in gemm_operands(M, N, K, 1, False))
    base = bf(rng.standard_normal((M, N))).view(-1)
    di = to_dev(ids)
    plan = bs.lora_plan(di, L)

    def run(x, A, B, H=None):
        h = bs.lora_shrink(x, A, plan) if H is None else H
        return h, bs.lora_expand(h, B, plan, base).view(M, N), bs.bsgemm_fp8_lora(*ops, h, B, di).view(M, N)
    want = run(x, A, B)
    bad_row = int(np.flatnonzero(ids == 1)[0])
    x2, A2, B2 = x.clone(), A.clone(), B.clone()
    x2[bad_row, 3] = float("nan")
    A2[3, 2, 5] = float("inf")
    B2[4, :, 0] = float("nan")
    got = run(x2, A2, B2)
    H3 = want[0].clone()
    H3[di < 0] = float("nan")
    again = run(x, A, B, H3)
    torch.cuda.synchronize()
    hit = (ids == 3) | (np.arange(M) == bad_row)
    for k, (g, w) in enumerate(zip(got, want)):
        bad = hit | ((ids == 4) if k else False)
        ok = to_dev(~bad)
        assert torch.equal(g[ok].view(torch.uint8), w[ok].view(torch.uint8)), k
        assert not bool(torch.isfinite(g[to_dev(bad)]).all(1).any()), k
    for g, w in list(zip(again, want))[1:]:
        assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))
