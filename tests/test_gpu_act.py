"""GPU parity of bsgemm_fp8_act against plain float64 (ffnref.py).  Products of small
integers with powers of two as scales are exact in fp32, so there the whole error is the
epilogue's; random ones lie within the fp8 product's interval, carried through the
epilogue.  Outputs are poisoned first and lie between guard elements."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
import ffnref
import opsref
import oracle
import synth
from gpuutil import bits16, device, say, to_dev
from oracle import bounds
from test_gpu_lora import band_index, bf, check_guards, guarded, values

pytestmark = pytest.mark.gpu


def operands(M, rows, K, seed, ints, spread=2):
    rng = np.random.default_rng(seed)
    if ints:   # codes of small integers; scales that differ from block to block
        code = torch.arange(-4, 5).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        qa, qb = code[rng.integers(0, 9, (M, K))], code[rng.integers(0, 9, (rows, K))]
        sa = 2.0 ** rng.integers(-spread, spread + 1, (M, K // 128))
        sb = 2.0 ** rng.integers(-spread, spread + 1, (rows // 128, K // 128))
        return qa, sa.astype(np.float32), qb, sb.astype(np.float32)
    A, B = synth.operand_fp32(M, rows, K, seed=seed, heavy=M >= 200)
    return (*oracle.quant_blocks(A, 1, 128), *oracle.quant_blocks(B * 3, 128, 128))


def exact_acc(ops):
    qa, sa, qb, sb = ops
    v = opsref.e4m3_values()
    a = (v[qa] * np.repeat(sa.astype(float), 128, 1)).astype(np.float32)
    b = ffnref.dequant(qb, sb).astype(np.float32)
    return (a @ b.T).astype(float)   # sums below 2^24 steps of the smallest product: exact


def run(ops, N, act="none", gated=False, bias=None, resid=None, alpha=1.0, beta=1.0, bands=1, stride=0, inplace=False):
    M = ops[0].shape[0]
    at = band_index(M, N, bands, stride)
    n = int(at.max()) + 1
    full, C = guarded(n, torch.bfloat16, -3.0)
    idx = to_dev(at.reshape(-1))
    flat = None
    if resid is not None:
        flat = torch.full((n,), 5.0, dtype=torch.bfloat16, device=device())
        flat[idx] = resid.reshape(-1)
        if inplace:
            C.copy_(flat)
            flat = C
    bs.bsgemm_fp8_act(*ops, bias=bias, act=act, gated=gated, resid=flat, alpha=alpha, beta=beta, C=C, bands=bands,
                      band_stride=stride)
    torch.cuda.synchronize()
    check_guards(full, -3.0)
    gaps = np.ones(n, bool)
    gaps[at.reshape(-1)] = False
    if gaps.any():
        assert bool((C[to_dev(gaps)] == (5.0 if inplace and resid is not None else -3.0)).all()), "gaps were written"
    return C[idx].view(M, N)


# M, N, K, bands, stride: every kernel, whole and ragged tiles
SHAPES = [(1, 128, 128, 1, 0), (1, 2048, 1792, 1, 0), (3, 384, 2048, 3, 0), (16, 640, 384, 2, 8 * 640 + 8),
          (17, 256, 1152, 1, 0), (32, 384, 256, 4, 0), (33, 1152, 512, 3, 0), (64, 640, 2048, 8, 0),
          (65, 512, 256, 13, 5 * 512 + 16), (200, 384, 256, 4, 50 * 384 + 64), (257, 768, 1024, 1, 0),
          (513, 512, 1152, 1, 0), (700, 2176, 640, 7, 100 * 2176 + 8), (1537, 2304, 896, 1, 0), (2050, 2304, 128, 1, 0),
          (2100, 2304, 384, 7, 0), (2600, 2560, 256, 8, 0), (2056, 2304, 512, 8, 257 * 2304 + 8), (2304, 2560, 512, 9, 0),
          (128, 256, 7168, 2, 0), (100, 7168, 256, 1, 0), (40, 7168, 128, 1, 0), (16, 7296, 256, 1, 0),
          (300, 128, 8320, 3, 0), (70, 2304, 8192, 1, 0),
          (50, 66048, 128, 5, 0)]


@pytest.mark.parametrize("M,N,K,bands,stride", SHAPES)
def test_plain_is_bsgemm_fp8(M, N, K, bands, stride):
    """Without bias, activation and residual: bsgemm_fp8's result bit for bit, whatever
    kernel the sizes choose."""
    say(f"bsgemm_fp8_act plain M={M} N={N} K={K} bands={bands}")
    ops = tuple(to_dev(a) for a in operands(M, N, K, M, False))
    got = run(ops, N, bands=bands, stride=stride)
    want = bs.bsgemm_fp8(*ops).view(M, N)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("M,N,K,bands,stride", SHAPES)
def test_exact_integers(M, N, K, bands, stride):
    """Accumulators, bias, residual and their sums are exact in fp32: the bf16 rounding of
    the formula, bit for bit (none and relu, not gated)."""
    host = operands(M, N, K, M + 1, True)
    ops = tuple(to_dev(a) for a in host)
    acc = exact_acc(host)
    rng = np.random.default_rng(M)
    bias, resid = rng.integers(-64, 65, N) / 4.0, rng.integers(-200, 201, (M, N)).astype(float)
    for act in ("none", "relu"):
        for b, r, inplace in ((True, True, False), (True, True, True), (False, True, True), (True, False, False)):
            say(f"bsgemm_fp8_act exact M={M} N={N} K={K} bands={bands} {act} bias={b} resid={r} inplace={inplace}")
            got = run(ops, N, act, bias=bf(bias) if b else None, resid=bf(resid) if r else None, alpha=0.5, beta=2.0,
                      bands=bands, stride=stride, inplace=inplace)
            want, _ = ffnref.epilogue(acc, 0.0, bias if b else None, act, False, resid if r else None, 0.5, 2.0)
            assert np.array_equal(values(got), bounds.bf16_rne_f64(want)), (act, b, r, inplace)


@pytest.mark.parametrize("M,N,K,bands,stride", SHAPES)
def test_gated_exact_sums(M, N, K, bands, stride):
    """Gated, with exact accumulators: within the epilogue's own bound (the gate's product
    rounds)."""
    host = operands(M, 2 * N, K, M + 2, True)
    ops = tuple(to_dev(a) for a in host)
    acc = exact_acc(host)
    rng = np.random.default_rng(M)
    bias, resid = rng.integers(-64, 65, 2 * N) / 4.0, rng.integers(-200, 201, (M, N)).astype(float)
    for act, b, r, inplace in (("none", False, False, False), ("relu", True, True, True), ("none", True, True, False)):
        say(f"bsgemm_fp8_act gated M={M} N={N} K={K} bands={bands} {act} bias={b} resid={r}")
        got = run(ops, N, act, True, bias=bf(bias) if b else None, resid=bf(resid) if r else None, alpha=2.0, beta=0.25,
                  bands=bands, stride=stride, inplace=inplace)
        want, tol = ffnref.epilogue(acc, np.zeros_like(acc), bias if b else None, act, True, resid if r else None, 2.0, 0.25)
        ok, used = bounds.within(bits16(got), want, tol)
        assert ok.all(), (act, b, r, float(used.max()))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K", [(9, 256, 384), (70, 256, 384), (2100, 2304, 128)])
def test_activations(act, gated, M, N, K):
    """Exact accumulators over the activations' whole range, up to +-100 and next to 0."""
    say(f"bsgemm_fp8_act {act} gated={gated} M={M}")
    rows = 2 * N if gated else N
    qa, sa, qb, sb = operands(M, rows, K, 5, True, spread=1)
    sa = (sa * 2.0 ** np.resize(np.arange(-9, 1), (M, 1))).astype(np.float32)   # one power of two to a row
    host = (qa, sa, qb, sb)
    acc = exact_acc(host)
    got = run(tuple(to_dev(a) for a in host), N, act, gated)
    want, tol = ffnref.epilogue(acc, np.zeros_like(acc), None, act, gated, None, 1.0, 1.0)
    ok, used = bounds.within(bits16(got), want, tol)
    say(f"  t from {acc.min():.1f} to {acc.max():.1f}; largest share of the interval {used.max():.3f}")
    assert ok.all()


@pytest.mark.parametrize("M,N,K,act,gated", [(5, 384, 1152, "silu", True), (40, 256, 2048, "gelu", False),
                                             (200, 512, 256, "gelu_tanh", False), (300, 512, 640, "silu", True),
                                             (2300, 2304, 640, "silu", True), (2300, 2304, 512, "gelu", False)])
def test_random(M, N, K, act, gated):
    say(f"bsgemm_fp8_act random M={M} N={N} K={K} {act} gated={gated}")
    rows = 2 * N if gated else N
    host = operands(M, rows, K, 7, False)
    ops = tuple(to_dev(a) for a in host)
    rng = np.random.default_rng(M)
    bias, resid = bf(rng.standard_normal(rows)), bf(rng.standard_normal((M, N)))
    got = run(ops, N, act, gated, bias, resid, 0.75, 1.25)
    acc, _ = oracle.bsgemm(*host)
    own = bounds.BsgemmBound(*host).rows(0, M)
    want, tol = ffnref.epilogue(acc.astype(float), own, values(bias), act, gated, values(resid), 0.75, 1.25)
    ok, used = bounds.within(bits16(got), want, tol)
    say(f"  largest share of the interval {used.max():.3f}")
    assert ok.all()
    again = run(ops, N, act, gated, bias, resid, 0.75, 1.25)
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("gated", [False, True])
def test_row_is_the_same_in_every_batch(gated):
    """A row's result by itself and in batches of every kernel's sizes."""
    say(f"bsgemm_fp8_act batches gated={gated}")
    N, K = 2304, 640
    rows = 2 * N if gated else N
    qa, sa, qb, sb = (to_dev(a) for a in operands(2100, rows, K, 9, False))
    resid = torch.randn((2100, N), device=device()).to(torch.bfloat16)
    ref = None
    for M in (2100, 700, 64, 20, 16, 1):
        got = bs.bsgemm_fp8_act(qa[:M].contiguous(), sa[:M].contiguous(), qb, sb, act="silu", gated=gated,
                                resid=resid[:M].contiguous()).view(M, N)
        ref = got if ref is None else ref
        assert torch.equal(got.view(torch.int16), ref[:M].view(torch.int16)), M


@pytest.mark.parametrize("M,N,K", [(1, 256, 256), (70, 256, 256), (2100, 2304, 256)])
def test_not_finite(M, N, K):
    """NaN and infinities in the bias and the residual follow the formulas, and reach
    their own elements only; a NaN row of A reaches its own row only."""
    say(f"bsgemm_fp8_act not finite M={M}")
    host = operands(M, N, K, 3, True)
    ops = tuple(to_dev(a) for a in host)
    bias = torch.zeros(N, dtype=torch.bfloat16, device=device())
    bias[5], bias[6], bias[7] = float("nan"), float("inf"), float("-inf")
    resid = torch.zeros((M, N), dtype=torch.bfloat16, device=device())
    resid[M - 1, 9] = float("nan")
    for act, want in (("none", "nan inf -inf"), ("relu", "nan inf 0.0"), ("silu", "nan inf nan"), ("gelu", "nan inf nan"),
                      ("gelu_tanh", "nan inf nan")):
        got = run(ops, N, act, bias=bias, resid=resid)
        assert all(" ".join(str(float(v)) for v in got[m, 5:8]) == want for m in (0, M // 2, M - 1)), act
        bad = ~torch.isfinite(got)
        assert bool(bad[M - 1, 9]) and not bool(bad[:, 10:].any()) and not bool(bad[:, :5].any())
    A = ops[0].clone()
    A[M // 2] = 0x7F
    got = run((A, *ops[1:]), N, "silu")
    plain = run(ops, N, "silu")
    keep = torch.arange(M, device=device()) != M // 2
    assert bool(torch.isnan(got[M // 2]).all()) and torch.equal(got[keep].view(torch.int16), plain[keep].view(torch.int16))


def test_weight_past_32_bits():
    """Gate and up rows more than 2^31 bytes apart, and more than 2^32 in all, at every
    kernel's batch."""
    N, K = 4096, 1 << 20
    say("bsgemm_fp8_act beyond 2^32 bytes of weight")
    B = torch.zeros((2 * N, K), dtype=torch.uint8, device=device())
    B[:, :128] = 0x38                        # 1.0 in the first block
    B[:, K - 128:] = 0x40                    # 2.0 in the last one
    sb = torch.ones((2 * N // 128, K // 128), dtype=torch.float32, device=device())
    sb[:, -1] = torch.arange(2 * N // 128, device=device()) % 8 + 1
    A = torch.zeros((2100, K), dtype=torch.uint8, device=device())
    A[:, :128] = 0x38
    A[:, K - 128:] = 0x38
    sa = torch.ones((2100, K // 128), dtype=torch.float32, device=device())
    t = (128 + 256 * sb[:, -1]).double().repeat_interleave(128)
    want = (t[:N] * t[N:]).to(torch.float32).to(torch.bfloat16)
    for M in (1, 64, 65, 2100):
        got = bs.bsgemm_fp8_act(A[:M], sa[:M], B, sb, gated=True).view(M, N)
        assert bool((got == want).all()), M
        got = bs.bsgemm_fp8_act(A[:M], sa[:M], B, sb).view(M, 2 * N)
        assert bool((got == t.to(torch.bfloat16)).all()), M


def test_millions_of_columns():
    """More columns than the few-rows kernel's grid holds, and just fewer."""
    say("bsgemm_fp8_act millions of columns")
    for N in ((1 << 25) - 256, 1 << 25):
        K = 128
        B = torch.zeros((N, K), dtype=torch.uint8, device=device())
        B[:, 5] = 0x38
        B[N - 1, 5] = 0x40
        sb = (torch.arange(N // 128, device=device()) % 4 + 1).to(torch.float32).view(-1, 1)
        A = torch.zeros((3, K), dtype=torch.uint8, device=device())
        A[:, 5] = torch.tensor([0x38, 0x40, 0xB8], dtype=torch.uint8, device=device())   # 1, 2, -1
        sa = torch.ones((3, 1), dtype=torch.float32, device=device())
        want = sb.view(-1).repeat_interleave(128)
        want[N - 1] *= 2
        C = bs.bsgemm_fp8_act(A, sa, B, sb, act="relu").view(3, N)
        assert bool((C[0] == want).all()) and bool((C[1] == 2 * want).all()) and bool((C[2] == 0).all())
        half = N // 2
        C = bs.bsgemm_fp8_act(A, sa, B, sb, gated=True).view(3, half)
        assert bool((C[0] == want[:half] * want[half:]).all())


def test_rows_of_millions_of_columns():
    """Whole tiles whose rows lie 2^25 elements apart, and the ragged ones below them."""
    M, N, K = 300, 1 << 25, 128
    A = torch.zeros((M, K), dtype=torch.uint8, device=device())
    A[:, 5] = (torch.arange(M, device=device()) % 8).float().to(torch.float8_e4m3fn).view(torch.uint8)
    B = torch.zeros((N, K), dtype=torch.uint8, device=device())
    B[:, 5] = 0x38
    sa = torch.ones((M, 1), dtype=torch.float32, device=device())
    sb = (torch.arange(N // 128, device=device()) % 4 + 1).to(torch.float32).view(-1, 1)
    cols = sb.view(-1).repeat_interleave(128).bfloat16()
    for what in ("bsgemm_fp8", "bsgemm_fp8_act", "gated"):
        say(f"300 rows of 2^25 columns: {what}")
        if what == "bsgemm_fp8":
            C = bs.bsgemm_fp8(A, sa, B, sb).view(M, N)
        else:
            C = bs.bsgemm_fp8_act(A, sa, B, sb, act="relu", gated=what == "gated").view(M, -1)
        want = cols if what != "gated" else cols[: N // 2] * cols[N // 2:]
        for m in (0, 1, 7, 100, 135, 142, 143, 144, 200, 255, 256, 299):
            v = m % 8
            assert bool((C[m] == want * (v * v if what == "gated" else v)).all()), (what, m)
        del C


@pytest.mark.parametrize("gated", [False, True])
def test_offsets_past_32_bits(gated):
    """A past 2^31 bytes and C past 2^31 elements, in place on the residual."""
    say(f"bsgemm_fp8_act 2^24 rows gated={gated}")
    M, N, K = (1 << 24) + 77, 128, 128
    row = torch.arange(M, device=device()) % 16
    A = torch.zeros((M, K), dtype=torch.uint8, device=device())
    A[:, 3] = row.float().to(torch.float8_e4m3fn).view(torch.uint8)
    sa = torch.ones((M, 1), dtype=torch.float32, device=device())
    rows = 256 if gated else 128
    B = torch.zeros((rows, K), dtype=torch.uint8, device=device())
    B[:, 3] = 0x38
    sb = torch.ones((rows // 128, 1), dtype=torch.float32, device=device())
    C = (torch.arange(M, device=device()) % 5).bfloat16().repeat_interleave(N)
    bs.bsgemm_fp8_act(A, sa, B, sb, act="none", gated=gated, resid=C, alpha=2.0, C=C)
    want = (row * row if gated else row) + 2 * (torch.arange(M, device=device()) % 5)
    assert bool((C.view(M, N) == want.bfloat16()[:, None]).all())
