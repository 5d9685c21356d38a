"""The layer's serving step (pipeline.WoBServeStep): quantize, plan, shrink, GEMM
with adapters, reduce + quantize, and the gathered wire through resnorm.  Every
stage is checked against the oracle or float64 on the device's own input to it;
the step is captured and replayed, follows its stream, and its calls may run
beside each other."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
import opsref
import oracle
import synth
from block_scaled_fp8_bsgemm_amd.pipeline import WoBServeStep
from gpuutil import bf16_dev, bits16, device, say, to_dev
from oracle import bounds

pytestmark = pytest.mark.gpu

SPIN_CYCLES = 200_000_000   # ~0.1 s of torch's spin kernel


def values(t):
    return t.double().cpu().numpy()


def bf(x):
    return to_dev(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


def make(M=264, N=512, K=512, bands=8, L=5, R=24, quant=128, f32=False, post=True, seed=0):
    rng = np.random.default_rng(seed)
    _, W = synth.operand_fp32(8, N, K, seed=seed, heavy=False)
    qb, sb = oracle.quant_blocks(W, 128, 128)
    parts = synth.partial_bands(M // bands, N, P=bands, seed0=100 + seed)[1:]
    wq, ws = oracle.rowq(synth.wire_rows(M, N, seed=200 + seed))
    ids = np.repeat(rng.integers(-1, L, M // 8 + 1), 8)[:M].astype(np.int32)
    resid = rng.standard_normal((M, N))
    return WoBServeStep(
        bf(rng.standard_normal((M, K))), to_dev(qb), to_dev(sb), [bf16_dev(p) for p in parts], to_dev(wq), to_dev(ws),
        bands, to_dev(resid.astype(np.float32)) if f32 else bf(resid), to_dev(ids),
        bf(rng.standard_normal((L, R, K)) * K ** -0.5), bf(rng.standard_normal((L, N, R)) * 0.1),
        to_dev((0.5 + rng.random(L)).astype(np.float32)), post_w=bf(1 + 0.1 * rng.standard_normal(N)) if post else None,
        gate=bf(rng.standard_normal(N)), pre_w=bf(1 + 0.1 * rng.standard_normal(N)), alpha=0.75, beta=0.5, quant=quant)


def outputs(s):
    return [t.clone().view(torch.uint8) for t in (s.A, s.a_scale, s.lora_plan, s.H, s.C, s.wire_q, s.wire_s, s.resid_out,
                                                  s.q if s.q is not None else s.z) if t is not None]


@pytest.mark.parametrize("kw", [dict(), dict(quant=32, f32=True, post=False), dict(M=1000, N=1152, K=256, R=64, quant=0),
                                dict(M=8, N=384, K=128, L=2, R=8)])
def test_step_vs_references(kw):
    say(f"serve step {kw}")
    s = make(**kw)
    wq0, ws0 = s.wire_q.cpu().numpy(), s.wire_s.cpu().numpy()
    s.step()
    torch.cuda.synchronize()
    M, N = s.C.shape
    L, R, _ = s.lora_A.shape
    rows = M // s.bands
    ids = s.ids.cpu().numpy()

    qa, sa = oracle.quant_blocks(s.x.float().cpu().numpy(), 1, 128)
    assert np.array_equal(s.A.cpu().numpy(), qa)
    assert np.array_equal(s.a_scale.cpu().numpy().view(np.uint32), sa.view(np.uint32))
    assert np.array_equal(s.lora_plan.cpu().numpy(), opsref.plan(ids, L))
    H, eH = opsref.shrink(values(s.x), values(s.lora_A), ids)
    assert np.all(np.abs(values(s.H) - H) <= eH)

    qb, sb = s.B.cpu().numpy(), s.b_scale.cpu().numpy()
    acc, _ = oracle.bsgemm(qa, sa, qb, sb)
    d, eD = opsref.delta(values(s.H), values(s.lora_B), values(s.lora_scale), ids)
    own = bounds.BsgemmBound(qa, sa, qb, sb).rows(0, M)
    c = bits16(s.C)
    ok, _ = bounds.within(c, acc.astype(float) + d, own + eD + 4 * opsref.U * R * (np.abs(acc) + own))
    assert ok.all()

    parts = [bits16(p) for p in s.partials]
    q, sc = oracle.rowq(oracle.band_reduce([c[:rows]] + parts))
    wq0[:rows], ws0[:rows] = q, sc
    assert np.array_equal(s.wire_q.cpu().numpy(), wq0)
    assert np.array_equal(s.wire_s.cpu().numpy().view(np.uint32), ws0.view(np.uint32))

    y = opsref.e4m3_values()[wq0] * ws0.astype(float)[:, None]
    a = s.norm_args
    h, eh, z, ez = opsref.resnorm(y, values(s.resid), None if a["post_w"] is None else values(a["post_w"]),
                                  values(a["gate"]), values(a["pre_w"]), a["alpha"], a["beta"], a["eps"])
    if s.resid.dtype == torch.float32:
        assert np.all(np.abs(values(s.resid_out) - h) <= eh + opsref.U * np.abs(h))
    else:
        assert bounds.within(bits16(s.resid_out), h, eh)[0].all()
    if a["quant"] == 0:
        assert bounds.within(bits16(s.z), z, ez)[0].all()
    else:
        v = s.q_scale.cpu().numpy()
        v = v.astype(float) if a["quant"] == 128 else 2.0 ** (v - 127.0)
        opsref.check_quant(s.q.cpu().numpy(), v, z, ez, a["quant"])


@pytest.mark.parametrize("quant", [0, 32, 128])
def test_capture_and_replay(quant):
    """The whole step in a graph, replayed with other inputs in its buffers and eager
    work between: every replay equals the eager step on the same inputs."""
    say(f"serve step captured, quant={quant}")
    s, other = make(quant=quant, seed=1), make(quant=quant, seed=2)
    stream = torch.cuda.Stream(device=device())
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.step()
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        s.step()
    torch.cuda.synchronize()
    x0, ids0 = s.x.clone(), s.ids.clone()
    for r in range(4):
        s.x.copy_(x0 if r % 2 else other.x)
        s.ids.copy_(ids0 if r % 2 else other.ids)
        s.step()
        torch.cuda.synchronize()
        want = outputs(s)
        for t in (s.H, s.C, s.resid_out):
            t.fill_(float("nan"))
        s.lora_plan.fill_(-9)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(outputs(s), want)):
            assert torch.equal(a, b), (r, k)


def test_calls_follow_their_stream():
    """The input lands late on a side stream; the step enqueued behind it sees it."""
    say("serve step on a side stream")
    ref, s = make(seed=3), make(seed=3)
    ref.step()
    torch.cuda.synchronize()
    x = s.x.clone()
    s.x.zero_()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream(device=device())
    with torch.cuda.stream(stream):
        torch.cuda._sleep(SPIN_CYCLES // 4)
        s.x.copy_(x, non_blocking=True)
        s.step()
    stream.synchronize()
    for a, b in zip(outputs(s), outputs(ref)):
        assert torch.equal(a, b)


def test_an_explicit_stream_and_two_steps_at_once():
    """Steps on two streams at a time do not share anything; a stream given by
    argument is the one that is used."""
    say("two serve steps at once")
    want = []
    for seed in (4, 5):
        r = make(M=1040, N=1024, seed=seed)
        r.step()
        torch.cuda.synchronize()
        want.append(outputs(r))
    steps = [make(M=1040, N=1024, seed=seed) for seed in (4, 5)]
    streams = [torch.cuda.Stream(device=device()) for _ in steps]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.step()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        for a, b in zip(outputs(s), w):
            assert torch.equal(a, b)
    ids = torch.zeros(5, dtype=torch.int32, device=device())
    plan = torch.full((5 + 2 + 5,), -1, dtype=torch.int32, device=device())
    torch.cuda.synchronize()
    with torch.cuda.stream(streams[0]):
        torch.cuda._sleep(SPIN_CYCLES // 4)
        ids.fill_(2)
    bs.lora_plan(ids, 5, plan, stream=streams[0])
    streams[0].synchronize()
    assert plan.tolist() == [0, 0, 0, 5, 5, 5, 5, 0, 1, 2, 3, 4]


def test_empty_batches():
    """No rows: nothing is launched for, or written by, any call but the plan's starts."""
    say("empty batches")
    d = device()

    def e(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device=d)
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    plan = bs.lora_plan(e(0, dtype=i32), 3)
    assert plan.tolist() == [0] * 5
    assert bs.lora_shrink(e(0, 64), e(3, 16, 64), plan).shape == (0, 16)
    assert bs.lora_expand(e(0, 16, dtype=f32), e(3, 128, 16), plan, e(0)).numel() == 0
    assert bs.bsgemm_fp8_lora(e(0, 128, dtype=u8), e(0, 1, dtype=f32), e(128, 128, dtype=u8), e(1, 1, dtype=f32),
                              e(0, 16, dtype=f32), e(3, 128, 16), e(0, dtype=i32)).numel() == 0
    r, z, q, sc = bs.resnorm(e(0, 256), e(0, 256), quant=128)
    assert r.shape == (0, 256) and z is None and q.shape == (0, 256) and sc.shape == (0, 2)


def test_refusals_on_the_device():
    """What only device tensors can show: strides, types, and tensors that are not there."""
    say("refusals of device tensors")
    d = device()
    x = torch.zeros((8, 128), dtype=torch.bfloat16, device=d)
    A = torch.zeros((2, 16, 128), dtype=torch.bfloat16, device=d)
    plan = bs.lora_plan(torch.zeros(8, dtype=torch.int32, device=d), 2)
    wide = torch.zeros((8, 256), dtype=torch.bfloat16, device=d)
    with pytest.raises(ValueError, match="contiguous"):
        bs.lora_shrink(wide[:, ::2], A, plan)
    with pytest.raises(ValueError, match="contiguous"):
        bs.resnorm(wide[:, :128], x)
    with pytest.raises(TypeError, match="dtype"):
        bs.lora_shrink(x.half(), A, plan)
    with pytest.raises(TypeError, match="dtype"):
        bs.lora_plan(torch.zeros(8, dtype=torch.int64, device=d), 2)
    with pytest.raises(TypeError, match="dtype"):
        bs.resnorm(x, x.half())
    with pytest.raises(ValueError, match="device tensor"):
        bs.lora_shrink(x, A.cpu(), plan)
    with pytest.raises(bs.BSError):   # 16-byte alignment
        bs.resnorm(wide.view(-1)[4:4 + 1024].view(8, 128), x)
    with pytest.raises(bs.BSError):   # the output over an input
        bs.lora_shrink(x, A, plan, x.view(torch.float32).view(-1)[:128].view(8, 16))
    with pytest.raises(bs.BSError):
        bs.resnorm(x, x, eps=0.0)
