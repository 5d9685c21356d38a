"""The feed-forward block (pipeline.FFNServeStep) behind resnorm: every stage against the
oracle or float64 on the device's own input to it; the step captured and replayed,
on its stream, beside another one.  The operators' own calls likewise: captured at every kernel's
sizes, on a stream given by argument, two graphs with one workspace in turn."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
import ffnref
import opsref
import oracle
import synth
from block_scaled_fp8_bsgemm_amd.pipeline import FFNServeStep
from gpuutil import bits16, device, say, to_dev
from oracle import bounds
from test_gpu_lora import bf, values

pytestmark = pytest.mark.gpu

SPIN_CYCLES = 50_000_000   # ~25 ms of torch's spin kernel


def weight(rows, K, seed):
    q, s = oracle.quant_blocks(synth.operand_fp32(8, rows, K, seed=seed, heavy=False)[1], 128, 128)
    return to_dev(q), to_dev(s)


def make(M=24, D=512, I=256, E=16, topk=4, Is=384, act="silu", seed=0, dense=True, routed=True, **route):
    rng = np.random.default_rng(seed)
    y, resid = bf(rng.standard_normal((M, D))), bf(rng.standard_normal((M, D)))
    r, z, q, qs = bs.resnorm(y, resid, z=torch.empty((M, D), dtype=torch.bfloat16, device=device()), quant=128)
    kw = {}
    if dense:
        kw["dense"] = weight(2 * Is, D, seed) + weight(D, Is, seed + 1)
    if routed:
        up, down = [weight(2 * I, D, 10 + seed + e) for e in range(E)], [weight(D, I, 50 + seed + e) for e in range(E)]
        kw.update(experts=tuple(torch.stack([t[i] for t in p]).contiguous() for p in (up, down) for i in (0, 1)),
                  router=bf(rng.standard_normal((E, D)) * D ** -0.5), topk=topk, **route)
    s = FFNServeStep(z, q, qs, act=act, **kw)
    s.resid = r
    return s


def outputs(s):
    names = (("h", "hq", "h_scale") if s.dense else ()) + (
        ("router_logits", "ids", "weights") if s.expert_weights else ())
    return [getattr(s, n).clone().view(torch.uint8) for n in names + ("out",)]


STEPS = [dict(), dict(M=1, D=1024, score="sigmoid", groups=4, topk_groups=2, scale=2.5, biased=True),
         dict(M=128, D=256, I=128, E=40, topk=8, act="gelu_tanh"), dict(M=300, routed=False, act="gelu"),
         dict(M=7, D=384, dense=False, renorm=False), dict(M=65, E=8, topk=8, I=128, Is=128)]


@pytest.mark.parametrize("kw", STEPS)
def test_step_vs_references(kw):
    say(f"feed-forward step {kw}")
    kw = dict(kw)
    E = kw.get("E", 16)
    bias = to_dev((0.1 * np.arange(E)).astype(np.float32)) if kw.pop("biased", False) else None
    s = make(**kw) if bias is None else make(bias=bias, **kw)
    M, D = s.out.shape
    base = None
    if s.dense:
        s.up()
        s.quantize()
        s.down()
        torch.cuda.synchronize()
        base = s.out.clone()
        q, qs = s.q.cpu().numpy(), s.q_scale.cpu().numpy()
        W13, s13, W2, s2 = (t.cpu().numpy() for t in s.dense)
        acc, _ = oracle.bsgemm(q, qs, W13, s13)
        want, tol = ffnref.epilogue(acc.astype(float), bounds.BsgemmBound(q, qs, W13, s13).rows(0, M), None, s.act, True,
                                    None, 1.0, 1.0)
        assert bounds.within(bits16(s.h), want, tol)[0].all()
        hq, hs = oracle.quant_blocks(s.h.float().cpu().numpy(), 1, 128)
        assert np.array_equal(s.hq.cpu().numpy(), hq)
        assert np.array_equal(s.h_scale.cpu().numpy().view(np.uint32), hs.view(np.uint32))
        acc, _ = oracle.bsgemm(hq, hs, W2, s2)
        assert bounds.within(bits16(base), acc.astype(float), bounds.BsgemmBound(hq, hs, W2, s2).rows(0, M))[0].all()
    s.out.fill_(float("nan"))
    s.step()
    torch.cuda.synchronize()
    if not s.expert_weights:
        assert torch.equal(s.out.view(torch.int16), base.view(torch.int16))
        return
    L, eL = opsref.shrink(values(s.z), values(s.router), np.zeros(M, np.int32))
    assert np.all(np.abs(values(s.router_logits) - L) <= eL)
    ids, w = ffnref.route(values(s.router_logits), s.topk, bias=None if s.bias is None else values(s.bias), **s.route_args)
    assert np.array_equal(s.ids.cpu().numpy(), ids)
    assert np.all(np.abs(values(s.weights) - w) <= 1.001 * ffnref.U * np.abs(w))
    W13, s13, W2, s2 = (t.cpu().numpy() for t in s.expert_weights)
    want, tol = ffnref.moe(values(s.z), ids, values(s.weights), ffnref.dequant(W13, s13), ffnref.dequant(W2, s2),
                           None if base is None else values(base), s.act)
    assert bounds.within(bits16(s.out), want, tol)[0].all()
    # and the block's output goes on as the next resnorm's y
    r, z, q, qs = bs.resnorm(s.out, s.resid, quant=128)
    assert bool(torch.isfinite(r.float()).all())


@pytest.mark.parametrize("kw", [dict(), dict(M=128, D=256, E=24, topk=6), dict(M=200, routed=False),
                                dict(M=1, dense=False, score="sigmoid", groups=4, topk_groups=2)])
def test_capture_and_replay(kw):
    """The step in a graph, replayed with other inputs and eager work between: every replay
    equals the eager step on the same inputs."""
    say(f"feed-forward step captured {kw}")
    s, other = make(seed=1, **kw), make(seed=2, **kw)
    stream = torch.cuda.Stream(device=device())
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        s.step()
    torch.cuda.synchronize()
    first = [t.clone() for t in (s.z, s.q, s.q_scale)]
    for r in range(4):
        for t, a, b in zip((s.z, s.q, s.q_scale), first, (other.z, other.q, other.q_scale)):
            t.copy_(a if r % 2 else b)
        s.step()
        torch.cuda.synchronize()
        want = outputs(s)
        s.out.fill_(float("nan"))
        if s.expert_weights:
            s.ids.fill_(-5)
            s.ws.fill_(0xFF)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(outputs(s), want)):
            assert torch.equal(a, b), (r, k)


def test_steps_follow_their_stream():
    """Inputs that land late on a side stream; two steps at a time on two streams."""
    say("feed-forward steps on side streams")
    want = []
    for seed in (4, 5):
        r = make(M=32, D=1024, seed=seed)
        r.step()
        torch.cuda.synchronize()
        want.append(outputs(r))
    steps = [make(M=32, D=1024, seed=seed) for seed in (4, 5)]
    streams = [torch.cuda.Stream(device=device()) for _ in steps]
    inputs = [[t.clone() for t in (s.z, s.q, s.q_scale)] for s in steps]
    for s in steps:
        for t in (s.z, s.q, s.q_scale):
            t.zero_()
    torch.cuda.synchronize()
    for k in range(5):
        for s, st, given in zip(steps, streams, inputs):
            with torch.cuda.stream(st):
                if k == 0:
                    torch.cuda._sleep(SPIN_CYCLES)
                    for t, a in zip((s.z, s.q, s.q_scale), given):
                        t.copy_(a, non_blocking=True)
                s.step()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        for a, b in zip(outputs(s), w):
            assert torch.equal(a, b)


def test_empty_batch():
    say("feed-forward step without rows")
    s = make(M=0)
    s.step()
    torch.cuda.synchronize()
    assert s.out.shape == (0, 512) and s.ids.shape == (0, 4)


# ------------------------------------------------------------ the calls --

def random_codes(shape, g):
    return torch.randint(0, 0x70, shape, generator=g, device=device(), dtype=torch.uint8)


def act_inputs(M, N, K, gated, seed):
    g = torch.Generator(device=device()).manual_seed(seed)
    rows = 2 * N if gated else N

    def scales(*shape):
        return torch.rand(shape, generator=g, device=device()) / K
    return (random_codes((M, K), g), scales(M, K // 128), random_codes((rows, K), g), scales(rows // 128, K // 128),
            torch.randn(rows, generator=g, device=device()).bfloat16(),
            torch.randn((M, N), generator=g, device=device()).bfloat16())


# few rows, 64-row groups, 64 x 128 tiles, whole tiles, the persistent kernel
CALLS = [(5, 512, 1024, True), (30, 384, 256, False), (130, 256, 1152, True), (520, 2176, 256, False),
         (2100, 2304, 384, False), (2100, 2304, 512, True), (2100, 2304, 384, True)]


@pytest.mark.parametrize("M,N,K,gated", CALLS)
def test_act_captured(M, N, K, gated):
    say(f"bsgemm_fp8_act captured M={M} N={N} K={K} gated={gated}")
    ins, other = act_inputs(M, N, K, gated, 1), act_inputs(M, N, K, gated, 2)
    out = torch.empty((M, N), dtype=torch.bfloat16, device=device())

    def call():
        A, sa, B, sb, bias, resid = ins
        bs.bsgemm_fp8_act(A, sa, B, sb, bias, "gelu", gated, resid.view(-1), 0.5, 2.0, out)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    first = [t.clone() for t in ins]
    for r in range(3):
        for t, a, b in zip(ins, first, other):
            t.copy_(a if r % 2 else b)
        call()
        torch.cuda.synchronize()
        want = out.clone()
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)), r


def moe_inputs(M, E, topk, D, I, seed):
    g = torch.Generator(device=device()).manual_seed(seed)
    return (torch.randn((M, D), generator=g, device=device()).bfloat16(),
            torch.randint(-1, E, (M, topk), generator=g, device=device(), dtype=torch.int32),
            torch.rand((M, topk), generator=g, device=device()),
            random_codes((E, 2 * I, D), g), torch.rand((E, 2 * I // 128, D // 128), generator=g, device=device()) / D,
            random_codes((E, D, I), g), torch.rand((E, D // 128, I // 128), generator=g, device=device()) / I)


def test_moe_graphs_share_a_workspace():
    """Two graphs of other sizes with one workspace, replayed in turn on one stream: each
    writes what it reads."""
    say("moe_fp8: two graphs, one workspace")
    sizes = ((3, 8, 2, 256, 384), (100, 12, 4, 512, 256))
    ws = torch.empty(max(bs.moe_fp8_workspace(M, k, E, I) for M, E, k, D, I in sizes), dtype=torch.uint8, device=device())
    ins = [moe_inputs(*s, seed=i) for i, s in enumerate(sizes)]
    want = [bs.moe_fp8(*a) for a in ins]
    outs = [torch.empty_like(w) for w in want]
    graphs = []
    for a, o in zip(ins, outs):
        bs.moe_fp8(*a, out=o, ws=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            bs.moe_fp8(*a, out=o, ws=ws)
        graphs.append(g)
    for r in range(4):
        for o in outs:
            o.fill_(float("nan"))
        ws.fill_(0xFF)
        if r % 2:
            torch.cuda.synchronize()
        for g in graphs if r < 2 else graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o.view(torch.int16), w.view(torch.int16)), r


def given_stream_calls():
    A, sa, B, sb, bias, resid = act_inputs(48, 256, 384, True, 3)
    g = torch.Generator(device=device()).manual_seed(1)
    logits = torch.randn((100, 64), generator=g, device=device())
    m = moe_inputs(20, 6, 3, 256, 128, 4)
    return {
        "bsgemm_fp8_act": lambda st: bs.bsgemm_fp8_act(A, sa, B, sb, bias, "silu", True, resid.view(-1), stream=st),
        "moe_route": lambda st: bs.moe_route(logits, 6, stream=st),
        "moe_fp8": lambda st: bs.moe_fp8(*m, stream=st),
    }


def test_outputs_belong_to_the_stream_that_is_given():
    """Outputs and the workspace that a call allocates for another stream than the current one
    are no memory that the current stream still uses."""
    stream = torch.cuda.Stream(device=device())
    for name, call in given_stream_calls().items():
        say(f"outputs on another stream: {name}")
        want = call(None)
        want = want if isinstance(want, tuple) else (want,)
        torch.cuda.synchronize()
        late = [torch.empty_like(t) for t in want] + [torch.empty(4 * 20 * 3 * 128, dtype=torch.uint8, device=device())]
        torch.cuda._sleep(SPIN_CYCLES)
        for t in late:
            t.view(torch.uint8).fill_(0x55)
        del late, t
        got = call(stream)
        torch.cuda.synchronize()
        for a, b in zip(got if isinstance(got, tuple) else (got,), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name


def test_the_given_stream_is_used():
    """The input is filled late on the stream that the call names."""
    say("feed-forward calls on a given stream")
    stream = torch.cuda.Stream(device=device())
    g = torch.Generator(device=device()).manual_seed(9)
    logits = torch.randn((33, 128), generator=g, device=device())
    want = bs.moe_route(logits, 4)
    m = moe_inputs(9, 5, 2, 256, 128, 6)
    want_m = bs.moe_fp8(*m)
    late_l, late_x = torch.zeros_like(logits), torch.zeros_like(m[0])
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(SPIN_CYCLES)
        late_l.copy_(logits)
        late_x.copy_(m[0])
    got = bs.moe_route(late_l, 4, stream=stream)
    got_m = bs.moe_fp8(late_x, *m[1:], stream=stream)
    stream.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(got_m.view(torch.int16), want_m.view(torch.int16))
