"""GPU parity of moe_route and moe_fp8 against plain float64 (ffnref.py)."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
import ffnref
from gpuutil import bits16, device, say, to_dev
from oracle import bounds
from test_gpu_lora import bf, check_guards, guarded, values

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


# ------------------------------------------------------------------ route --

def run_route(logits, topk, **kw):
    M = logits.shape[0]
    fi, ids = guarded(M * topk, torch.int32, -77)
    fw, w = guarded(M * topk, torch.float32, -3.0)
    bs.moe_route(logits, topk, ids=ids, weights=w, **kw)
    torch.cuda.synchronize()
    check_guards(fi, -77)
    check_guards(fw, -3.0)
    return ids.view(M, topk), w.view(M, topk)


def check_route(logits, topk, bias=None, **kw):
    """ids equal; weights to the fp32 rounding of fp64 scores, which fp64 itself has to 2^-48."""
    ids, w = run_route(logits, topk, bias=None if bias is None else to_dev(bias.astype(np.float32)), **kw)
    want_ids, want = ffnref.route(values(logits), topk, bias=None if bias is None else bias.astype(np.float32).astype(float),
                                  **kw)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    got = values(w)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    with np.errstate(invalid="ignore"):
        off = np.abs(got - want) > ffnref.U * 1.001 * np.abs(want) + 2.0 ** -150
    assert not np.any(off & ~np.isnan(want))


ROUTE = [(1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (3, 60, 4, 1, 1), (5, 64, 64, 1, 1), (64, 65, 6, 5, 2), (7, 128, 1, 64, 3),
         (100, 37, 5, 37, 9), (33, 1000, 8, 8, 8), (9, 1024, 33, 16, 2), (130, 512, 8, 2, 1), (1001, 384, 8, 12, 4),
         (6, 6, 6, 3, 1)]


@pytest.mark.parametrize("M,E,topk,groups,keep", ROUTE)
def test_route(M, E, topk, groups, keep):
    rng = np.random.default_rng(M + E)
    for score in ("softmax", "sigmoid"):
        for dtype in (torch.float32, torch.bfloat16):
            for biased in (False, True):
                say(f"moe_route M={M} E={E} topk={topk} groups={groups}/{keep} {score} {dtype} bias={biased}")
                # bf16 logits: many equal ones
                x = to_dev((rng.standard_normal((M, E)) * 2).astype(np.float32)).to(dtype)
                bias = rng.standard_normal(E) * 0.2 if biased else None
                check_route(x, topk, bias, score=score, groups=groups, topk_groups=keep, renorm=biased, scale=2.5)
                if groups > 1:
                    check_route(x, topk, bias, score=score, groups=groups, topk_groups=keep, group_top=1)


@pytest.mark.parametrize("E,groups", [(8, 1), (64, 4), (200, 8)])
def test_route_ties_and_masks(E, groups):
    """Equal logits, logits and biases of -infinity and NaN, rows with too few experts or
    none, the largest finite values, signed zeros."""
    say(f"moe_route masks E={E} groups={groups}")
    rng = np.random.default_rng(E)
    x = rng.integers(-2, 3, (40, E)).astype(np.float32)
    x[1] = 0.0
    x[2, ::2] = -0.0
    x[3] = -INF
    x[4] = -INF
    x[4, E - 1] = -3.0
    x[5, : E - 2] = -INF
    x[6, ::3] = NAN
    x[7] = NAN
    x[8] = np.finfo(np.float32).max
    x[9] = -np.finfo(np.float32).max
    x[10, 3] = np.finfo(np.float32).max
    x[11, 1] = -np.finfo(np.float32).max
    x[12] = -200.0 + np.arange(E) / 16
    x[13] = 40.0 + np.arange(E) / 64          # sigmoids that are 1 in fp64
    x[14, : E // 2] = -INF
    masked = np.where(rng.random(E) < 0.3, -INF, 0.25 * rng.integers(-2, 3, E))
    masked[1] = NAN
    for score in ("softmax", "sigmoid"):
        for bias in (None, masked, np.full(E, -INF)):
            for renorm in (True, False):
                check_route(to_dev(x), 5, bias, score=score, groups=groups, topk_groups=min(groups, 3), renorm=renorm)


def test_route_infinite_logit():
    """+infinity is chosen first; its softmax weights are NaN, as the formula's."""
    x = np.zeros((2, 16), np.float32)
    x[0, 5] = INF
    say("moe_route +infinity")
    ids, w = run_route(to_dev(x), 3)
    assert ids.tolist() == [[5, 0, 1], [0, 1, 2]] and bool(torch.isnan(w[0]).all()) and bool((w[1] == w[1, 0]).all())
    ids, w = run_route(to_dev(x), 3, score="sigmoid", renorm=False)
    assert ids.tolist() == [[5, 0, 1], [0, 1, 2]] and w[0].tolist() == [1.0, 0.5, 0.5]


def test_route_no_rows_and_many():
    say("moe_route 0 and 300001 rows")
    ids, w = bs.moe_route(torch.empty((0, 64), device=device()), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    g = torch.Generator(device=device()).manual_seed(0)
    x = torch.randn((300001, 16), generator=g, device=device())
    ids, w = run_route(x, 3)
    want = x.argsort(dim=1, descending=True, stable=True)[:, :3]
    assert torch.equal(ids.long(), want)
    s = torch.softmax(x.double(), 1).gather(1, want)
    assert bool(((w.double() - s / s.sum(1, keepdim=True)).abs() <= 2.0 ** -23).all())


def test_route_more_rows_than_a_launch_holds():
    say("moe_route 2^25 + 5 rows")
    M = (1 << 25) + 5
    x = torch.zeros((M, 2), dtype=torch.bfloat16, device=device())
    x[:, 1] = (torch.arange(M, device=device()) % 3 - 1).bfloat16()
    ids, w = run_route(x, 1)
    assert bool((ids[:, 0] == (x[:, 1] > 0)).all()) and bool((w == 1).all())


# ---------------------------------------------------------------- experts --

def make(M, E, topk, D, I, seed=0, mix="distinct", heavy=False):
    rng = np.random.default_rng(seed)
    x = bf(rng.standard_normal((M, D)))
    n = {"distinct": E, "shared": 4 * E}.get(mix, E)
    if mix == "one":
        ids = np.full((M, topk), -1)
        ids[:, 0] = E - 1
    elif mix == "none":
        ids = rng.choice([-1, E, E + 7, 2**31 - 1, -2**31], (M, topk))
    elif mix == "repeats":
        ids = rng.integers(0, min(E, 3), (M, topk))
    else:
        ids = np.stack([rng.permutation(max(n, topk))[:topk] for _ in range(M)])
    w = rng.random((M, topk)).astype(np.float32) - 0.2

    def codes(*shape):   # every finite code
        c = rng.integers(0, 256, shape).astype(np.uint8)
        c[(c & 0x7F) == 0x7F] = 0x38
        return c
    W13, W2 = codes(E, 2 * I, D), codes(E, D, I)
    s13 = ((0.5 + rng.random((E, 2 * I // 128, D // 128))) / 100 * D ** -0.5).astype(np.float32)
    s2 = ((0.5 + rng.random((E, D // 128, I // 128))) / 100 * I ** -0.5).astype(np.float32)
    base = bf(rng.standard_normal((M, D)))
    return x, ids.astype(np.int32), w, W13, s13, W2, s2, base


def run_moe(x, ids, w, W13, s13, W2, s2, base=None, act="silu", inplace=False):
    M, D = x.shape
    topk, (E, _, I) = ids.shape[1], W2.shape
    full, out = guarded(M * D, torch.bfloat16, -3.0)
    fw, ws = guarded(bs.moe_fp8_workspace(M, topk, E, I), torch.uint8, 0xEE)
    ws.fill_(0xFF)   # NaN wherever h is not written
    if inplace:
        out.copy_(base.reshape(-1))
        base = out.view(M, D)
    dev = [a if isinstance(a, torch.Tensor) else to_dev(a) for a in (ids, w, W13, s13, W2, s2)]
    bs.moe_fp8(x, *dev, base=base, act=act, out=out, ws=ws)
    torch.cuda.synchronize()
    check_guards(full, -3.0)
    check_guards(fw, 0xEE)
    return out.view(M, D)


MOE = [(1, 1, 1, 128, 128), (1, 32, 8, 1024, 512), (5, 16, 2, 384, 640), (16, 8, 4, 256, 384), (17, 4, 2, 512, 256),
       (33, 3, 2, 128, 384), (64, 12, 8, 256, 128), (100, 1, 1, 128, 1152), (128, 6, 3, 384, 128), (128, 40, 8, 128, 256),
       (2, 70, 64, 128, 128), (16, 1000, 64, 128, 128), (3, 5, 3, 7168, 128), (3, 5, 3, 128, 2048),
       (1, 9, 8, 256, 384), (4, 3, 2, 384, 128), (8, 4, 1, 128, 256), (2, 30, 4, 512, 384), (3, 4, 3, 128, 128)]


@pytest.mark.parametrize("M,E,topk,D,I", MOE)
def test_moe(M, E, topk, D, I):
    for k, (mix, act, base, inplace) in enumerate((("distinct", "silu", True, False), ("shared", "gelu_tanh", False, False),
                                                   ("one", "gelu", True, True), ("repeats", "relu", False, False),
                                                   ("none", "none", True, False), ("none", "silu", False, False))):
        if E > 100 and k > 1:
            continue
        say(f"moe_fp8 M={M} E={E} topk={topk} D={D} I={I} {mix} {act} base={base}")
        x, ids, w, W13, s13, W2, s2, b = make(M, E, topk, D, I, k, mix)
        got = run_moe(x, ids, w, W13, s13, W2, s2, b if base else None, act, inplace)
        want, tol = ffnref.moe(values(x), ids, w.astype(float), ffnref.dequant(W13, s13), ffnref.dequant(W2, s2),
                               values(b) if base else None, act)
        ok, used = bounds.within(bits16(got), want, tol)
        say(f"  largest share of the interval {used.max():.3f}")
        assert ok.all(), mix
        again = run_moe(x, ids, w, W13, s13, W2, s2, b if base else None, act, inplace)
        assert torch.equal(got.view(torch.int16), again.view(torch.int16))


def test_moe_every_code():
    """Each e4m3 code as a weight, NaN included, comes out as its value."""
    say("moe_fp8 codes")
    E, D, I = 2, 256, 256
    codes = np.arange(256, dtype=np.uint8)
    W13, W2 = np.zeros((E, 2 * I, D), np.uint8), np.zeros((E, D, I), np.uint8)
    W13[0, 0, 0], W13[0, I, 0] = 0x38, 0x38      # h[0] = x[0]^2
    W2[0, :, 0] = codes
    x = np.zeros((1, D))
    x[0, 0] = 1.0
    one = np.ones
    got = run_moe(bf(x), np.zeros((1, 1), np.int32), one((1, 1), np.float32), W13, one((E, 4, 2), np.float32), W2,
                  one((E, 2, 2), np.float32), act="none")
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    assert torch.equal(torch.nan_to_num(got[0].float().cpu(), nan=1e9), torch.nan_to_num(want, nan=1e9))


def test_moe_not_finite_stays_in_its_row():
    """A NaN token, an expert of NaN codes, one of infinite scales, a NaN weight: only the rows
    that have them change."""
    say("moe_fp8 not finite")
    M, E, topk, D, I = 40, 6, 2, 256, 384
    x, ids, w, W13, s13, W2, s2, b = make(M, E, topk, D, I, 11)
    ids[:, 1] = np.where(ids[:, 1] >= 3, ids[:, 1], -1)      # experts 0..2 in the first slots only
    plain = run_moe(x, ids, w, W13, s13, W2, s2, b)
    W13b, s2b, xb, wb = W13.copy(), s2.copy(), x.clone(), w.copy()
    W13b[0, 5, 7] = 0x7F
    s2b[1] = INF
    xb[13, 3] = NAN
    wb[21, 0] = NAN
    ids[13], ids[21] = (2, 4), (2, 4)
    plain = run_moe(x, ids, w, W13, s13, W2, s2, b)
    got = run_moe(xb, ids, wb, W13b, s13, W2, s2b, b)
    hit = to_dev(np.isin(ids, (0, 1)).any(1) | np.isin(np.arange(M), (13, 21)))
    assert torch.equal(got[~hit].view(torch.int16), plain[~hit].view(torch.int16))
    assert bool((~torch.isfinite(got[hit])).any(1).all())


@pytest.mark.parametrize("D,I", [(1024, 512), (384, 1152)])
def test_moe_row_is_the_same_in_every_batch(D, I):
    say(f"moe_fp8 batches D={D} I={I}")
    x, ids, w, W13, s13, W2, s2, b = make(128, 9, 3, D, I, 4)
    W13, s13, W2, s2 = (to_dev(a) for a in (W13, s13, W2, s2))
    ref = run_moe(x, ids, w, W13, s13, W2, s2, b)
    for M in (100, 64, 17, 16, 2, 1):
        got = run_moe(x[:M].contiguous(), ids[:M], w[:M], W13, s13, W2, s2, b[:M].contiguous())
        assert torch.equal(got.view(torch.int16), ref[:M].view(torch.int16)), M
    order = np.random.default_rng(0).permutation(128)
    got = run_moe(x[to_dev(order)], ids[order][:, ::-1], w[order][:, ::-1], W13, s13, W2, s2, b[to_dev(order)])
    assert torch.equal(got.view(torch.int16), ref[to_dev(order)].view(torch.int16))


def test_moe_weights_past_32_bits():
    """A stack of more than 2^32 bytes, its first and last expert used."""
    E, D, I = 70, 8192, 4096
    say("moe_fp8 beyond 2^32 bytes of weights")
    W13 = torch.zeros((E, 2 * I, D), dtype=torch.uint8, device=device())
    W2 = torch.zeros((E, D, I), dtype=torch.uint8, device=device())
    s13 = torch.ones((E, 2 * I // 128, D // 128), device=device())
    s2 = torch.ones((E, D // 128, I // 128), device=device())
    for e, c in ((0, 0x38), (E - 1, 0x40)):     # 1.0 and 2.0
        W13[e, :I, D - 1], W13[e, I:, 0], W2[e] = c, c, c
    x = torch.zeros((3, D), dtype=torch.bfloat16, device=device())
    x[:, 0], x[:, D - 1] = 1.0, 0.5
    ids = torch.tensor([[0, E], [E - 1, -1], [E - 1, 0]], dtype=torch.int32, device=device())
    w = torch.tensor([[1.0, 9.0], [0.5, 9.0], [0.25, 2.0]], device=device())
    got = run_moe(x, ids, w, W13, s13, W2, s2, act="none")
    one, last = 0.5 * I, 2.0 * (2.0 * 1.0) * I   # per expert: (c/2 * c) * c * I
    want = torch.tensor([one, 0.5 * last, 0.25 * last + 2 * one], device=device()).to(torch.bfloat16)
    assert bool((got == want[:, None]).all())
