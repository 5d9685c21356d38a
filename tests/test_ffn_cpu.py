"""bsgemm_fp8_act, moe_route and moe_fp8 without a GPU: the C entry points refuse
malformed calls before any launch, and the binding refuses tensors of the wrong shape,
type or device.  Every call here is refused or has no rows, since the pointers are fake.
Also the references of the GPU tests, on cases worked by hand."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
import ffnref

INV, UNS, OK = bs.BS_ERR_INVALID, bs.BS_ERR_UNSUPPORTED, bs.BS_OK
P = 0x1000000   # fake, aligned "device" addresses, 16 MiB apart
ADDR = [P * (i + 1) for i in range(12)]
NAN, INF = float("nan"), float("inf")
u8, f32, b16, i32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def L():
    return bs.load()


def act(L, A=ADDR[0], sa=ADDR[1], B=ADDR[2], sb=ADDR[3], bias=ADDR[4], resid=ADDR[5], C=ADDR[6], M=64, N=512, K=256,
        code=2, gated=0, alpha=1.0, beta=1.0, bands=1, stride=0):
    return L.bsgemm_fp8_act(A, sa, B, sb, bias, resid, C, M, N, K, code, gated, alpha, beta, bands, stride, None)


def test_act_refusals(L):
    for k in ("A", "sa", "B", "sb", "C"):
        assert act(L, **{k: 0}) == INV, k
    assert act(L, M=-1) == INV and act(L, N=0) == INV and act(L, K=0) == INV and act(L, bands=0) == INV
    assert act(L, code=-1) == INV and act(L, code=5) == INV and act(L, gated=2) == INV
    for v in (NAN, INF, -INF):
        assert act(L, alpha=v) == INV and act(L, beta=v) == INV
    assert act(L, N=500) == UNS and act(L, K=200) == UNS and act(L, bands=3) == UNS and act(L, bands=65, M=65) == UNS
    assert act(L, bands=2, stride=32 * 512 - 8) == UNS and act(L, bands=2, stride=32 * 512 + 4) == UNS
    for k, i in (("A", 0), ("B", 2), ("bias", 4), ("resid", 5), ("C", 6)):
        assert act(L, **{k: ADDR[i] + 8}) == UNS, k
    for k, i in (("sa", 1), ("sb", 3)):
        assert act(L, **{k: ADDR[i] + 2}) == UNS, k
    for i in range(5):
        assert act(L, C=ADDR[i]) == INV, i
    assert act(L, C=ADDR[5] + 16) == INV                              # neither resid itself nor clear of it
    # gated: B and its scales and bias have twice the rows
    far = ADDR[2] + 512 * 256
    assert act(L, C=far, gated=1) == INV
    assert act(L, C=ADDR[3] + 4 * 2 * 4, gated=1) == INV and act(L, C=ADDR[4] + 1024, gated=1) == INV
    assert act(L, N=1 << 30, gated=1, K=128) == UNS                   # 2N rows of B
    assert act(L, M=1 << 20, N=1 << 20) == UNS                        # more tiles than a launch holds
    assert act(L, M=0) == OK and act(L, M=0, resid=ADDR[6]) == OK and act(L, M=0, bias=0, resid=0, gated=1) == OK


def route(L, logits=ADDR[0], bias=ADDR[1], ids=ADDR[2], w=ADDR[3], rows=64, E=256, topk=8, bf16=0, score=1, groups=8,
          keep=4, gtop=2, renorm=1, scale=1.0):
    return L.moe_route(logits, bias, ids, w, rows, E, topk, bf16, score, groups, keep, gtop, renorm, scale, None)


def test_route_refusals(L):
    for k in ("logits", "ids", "w"):
        assert route(L, **{k: 0}) == INV, k
    assert route(L, rows=-1) == INV and route(L, E=0) == INV and route(L, topk=0) == INV and route(L, groups=0) == INV
    assert route(L, bf16=2) == INV and route(L, score=-1) == INV and route(L, renorm=3) == INV
    assert route(L, topk=257) == INV and route(L, keep=0) == INV and route(L, keep=9) == INV
    assert route(L, gtop=0) == INV and route(L, gtop=3) == INV
    assert route(L, scale=NAN) == INV and route(L, scale=INF) == INV
    assert route(L, E=1032) == UNS and route(L, E=250) == UNS and route(L, topk=65) == UNS
    assert route(L, E=256, groups=128) == UNS and route(L, rows=1 << 32) == UNS
    assert route(L, logits=ADDR[0] + 2) == UNS and route(L, logits=ADDR[0] + 1, bf16=1) == UNS
    for k, i in (("bias", 1), ("ids", 2), ("w", 3)):
        assert route(L, **{k: ADDR[i] + 2}) == UNS, k
    assert route(L, ids=ADDR[0] + 64) == INV and route(L, w=ADDR[0]) == INV and route(L, ids=ADDR[1]) == INV
    assert route(L, w=ADDR[1] + 1020) == INV and route(L, w=ADDR[2] + 64) == INV
    assert route(L, rows=0) == OK and route(L, rows=0, logits=0, ids=0, w=0) == OK


def moe(L, a=ADDR, M=16, topk=4, E=8, D=256, I=384, code=2):
    return L.moe_fp8(*a[:10], M, topk, E, D, I, code, None)


def test_moe_refusals(L):
    def at(i, v):
        return ADDR[:i] + [v] + ADDR[i + 1:]
    for i in (0, 1, 2, 3, 4, 5, 6, 8, 9):   # 7, the base, may be null
        assert moe(L, at(i, 0)) == INV, i
    assert moe(L, M=-1) == INV and moe(L, topk=0) == INV and moe(L, E=0) == INV and moe(L, D=0) == INV
    assert moe(L, I=0) == INV and moe(L, code=5) == INV and moe(L, code=-1) == INV
    assert moe(L, M=129) == UNS and moe(L, topk=65) == UNS and moe(L, M=128, topk=9) == UNS and moe(L, E=1025) == UNS
    assert moe(L, D=200) == UNS and moe(L, I=200) == UNS and moe(L, D=65664) == UNS and moe(L, I=65664) == UNS
    for i in (0, 3, 5, 7, 8, 9):
        assert moe(L, at(i, ADDR[i] + 8)) == UNS, i
    for i in (1, 2, 4, 6):
        assert moe(L, at(i, ADDR[i] + 2)) == UNS, i
    for i in range(7):
        assert moe(L, at(8, ADDR[i])) == INV and moe(L, at(9, ADDR[i])) == INV, i
    assert moe(L, at(8, ADDR[7] + 16)) == INV and moe(L, at(9, ADDR[7])) == INV and moe(L, at(9, ADDR[8])) == INV
    assert moe(L, M=0) == OK and moe(L, [0, 0, 0, *ADDR[3:7], 0, 0, 0], M=0) == OK


def test_workspace(L):
    n = ctypes.c_int64()
    assert L.moe_fp8_workspace(16, 4, 8, 384, None) == INV and L.moe_fp8_workspace(16, 4, 8, 0, n) == INV
    assert L.moe_fp8_workspace(129, 4, 8, 384, n) == UNS and L.moe_fp8_workspace(16, 4, 8, 100, n) == UNS
    assert bs.moe_fp8_workspace(16, 4, 8, 384) >= 4 * 64 * 384   # h in 32 bits
    assert bs.moe_fp8_workspace(1, 1, 1024, 128) < bs.moe_fp8_workspace(128, 8, 1024, 128) < 1 << 24


def t(*shape, dtype=b16):
    return torch.zeros(shape, dtype=dtype)


def refused(match, fn, *a, **kw):
    with pytest.raises((ValueError, TypeError)) as e:
        fn(*a, **kw)
    assert match in str(e.value), str(e.value)


def test_binding_refusals():
    g = (t(64, 256, dtype=u8), t(64, 2, dtype=f32), t(512, 256, dtype=u8), t(4, 2, dtype=f32))
    f = bs.bsgemm_fp8_act
    refused("act must", f, *g, act="swish")
    refused("a_scale", f, g[0], t(64, 3, dtype=f32), *g[2:])
    refused("b_scale", f, *g[:3], t(2, 2, dtype=f32))
    refused("one K", f, *g[:2], t(512, 128, dtype=u8), g[3])
    refused("multiples", f, *g[:2], t(500, 256, dtype=u8), g[3])
    refused("multiples", f, *g[:2], t(384, 256, dtype=u8), t(3, 2, dtype=f32), gated=True)
    refused("A must", f, g[0].view(-1), *g[1:])
    refused("bias:", f, *g, bias=t(256))
    refused("bias:", f, *g, bias=t(256), gated=True)
    refused("resid:", f, *g, resid=t(64 * 512 - 1))
    refused("resid:", f, *g, resid=t(64 * 512), bands=2, band_stride=32 * 512 + 8)
    refused("C:", f, *g, C=t(64 * 512 - 1))
    refused("C:", f, *g, C=t(64 * 256 - 1), gated=True)
    refused("device tensor", f, *g)
    r = bs.moe_route
    x = t(64, 256, dtype=f32)
    refused("logits must", r, t(256, dtype=f32), 8)
    refused("score", r, x, 8, score="tanh")
    refused("topk", r, x, 0)
    refused("topk", r, x, 257)
    refused("groups", r, x, 8, groups=3)
    refused("topk_groups", r, x, 8, groups=4, topk_groups=5)
    refused("group_top", r, x, 8, groups=4, group_top=3)
    refused("bias:", r, x, 8, bias=t(128, dtype=f32))
    refused("ids:", r, x, 8, ids=t(64, 7, dtype=i32))
    refused("weights:", r, x, 8, weights=t(63, 8, dtype=f32))
    refused("device tensor", r, x, 8)
    m = bs.moe_fp8
    a = (t(16, 256), t(16, 4, dtype=i32), t(16, 4, dtype=f32), t(8, 768, 256, dtype=u8), t(8, 6, 2, dtype=f32),
         t(8, 256, 384, dtype=u8), t(8, 2, 3, dtype=f32))

    def but(i, v):
        return a[:i] + (v,) + a[i + 1:]
    refused("act must", m, *a, act="swiglu")
    refused("x must", m, *but(0, t(16 * 256)))
    refused("W2:", m, *but(0, t(16, 128)))
    refused("W13:", m, *but(3, t(8, 384, 256, dtype=u8)))
    refused("s13:", m, *but(4, t(8, 3, 2, dtype=f32)))
    refused("s2:", m, *but(6, t(8, 3, 2, dtype=f32)))
    refused("multiples", m, *but(5, t(8, 256, 200, dtype=u8)))
    refused("ids:", m, *but(1, t(15, 4, dtype=i32)))
    refused("weights:", m, *but(2, t(16, 5, dtype=f32)))
    refused("base:", m, *a, base=t(16, 128))
    refused("out:", m, *a, out=t(16, 128))
    refused("ws:", m, *a, ws=t(100, dtype=u8))
    refused("device tensor", m, *a)


def test_reference_route():
    x = np.array([[1.0, 3.0, 2.0, 3.0], [-INF, 0.0, NAN, -1.0], [-INF] * 4])
    ids, w = ffnref.route(x, 3)
    assert ids.tolist() == [[1, 3, 2], [1, 3, -1], [-1, -1, -1]]
    e = math.exp(-1)
    assert np.allclose(w[0], [1 / (2 + e), 1 / (2 + e), e / (2 + e)]) and np.isnan(w[1, 0]) and not w[2].any()
    # groups {0,1}, {2,3}: sums of the two best 1.0 against 1.1, of the best alone 0.9 against 0.6
    s = np.array([[0.9, 0.1, 0.5, 0.6]])
    x = np.log(s / (1 - s))
    assert ffnref.route(x, 2, "sigmoid", groups=2)[0].tolist() == [[3, 2]]
    assert ffnref.route(x, 2, "sigmoid", groups=2, group_top=1)[0].tolist() == [[0, 1]]
    ids, w = ffnref.route(x, 2, "sigmoid", bias=np.array([0, 0.6, 0, 0.0]), renorm=False, scale=2.0)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[1.8, 0.2]])


def test_reference_act():
    for name, at, want in (("silu", 1.0, 0.7310585786), ("gelu", -1.0, -0.1586552539), ("gelu_tanh", 1.0, 0.8411919906),
                           ("relu", -2.0, 0.0), ("none", -2.0, -2.0)):
        assert abs(ffnref.act(at, name) - want) < 1e-9, name
    x = np.linspace(-6, 6, 4001)
    for name in ffnref.ACTS:
        assert np.max(np.abs(np.diff(ffnref.act(x, name)))) <= ffnref.SLOPE * (x[1] - x[0]) * 1.0001, name


def test_step_refusals():
    from block_scaled_fp8_bsgemm_amd.pipeline import FFNServeStep
    z = torch.zeros((4, 256), dtype=torch.bfloat16)
    q, qs = torch.zeros((4, 256), dtype=torch.uint8), torch.ones((4, 2))
    dense = (torch.zeros((256, 256), dtype=torch.uint8), torch.ones((2, 2)),
             torch.zeros((256, 128), dtype=torch.uint8), torch.ones((2, 1)))
    experts = tuple(t.expand(8, *t.shape).contiguous() for t in dense)
    router = torch.zeros((8, 256), dtype=torch.bfloat16)
    for kw, message in ((dict(z=z, q=q, q_scale=qs), "need a dense part"), (dict(z=z, router=router), "go together"),
                        (dict(z=z, experts=experts), "go together"), (dict(z=z, dense=dense), "needs q"),
                        (dict(q=q, q_scale=qs, router=router, experts=experts), "need z"),
                        (dict(z=z, router=router[:4], experts=experts), "4 experts")):
        with pytest.raises(ValueError, match=message):
            FFNServeStep(**kw)
