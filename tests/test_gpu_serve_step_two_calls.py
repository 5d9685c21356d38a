"""WoBServeStep with its adapters added by a call of their own (fused=False): against
float64 on the product's own output, captured and replayed."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
import opsref
from block_scaled_fp8_bsgemm_amd.pipeline import WoBServeStep
from gpuutil import bits16, device, say, to_dev
from oracle import bounds
from test_gpu_serve_step import make, outputs, values

pytestmark = pytest.mark.gpu


def two_calls(**kw):
    s = make(**kw)
    return WoBServeStep(s.x, s.B, s.b_scale, s.partials, s.wire_q, s.wire_s, s.bands, s.resid, s.ids, s.lora_A, s.lora_B,
                        s.lora_scale, fused=False, **s.norm_args)


@pytest.mark.parametrize("kw", [dict(), dict(M=1000, N=1152, K=256, R=64, quant=0), dict(M=8, N=384, K=128, L=2, R=8)])
def test_step(kw):
    say(f"serve step by two calls {kw}")
    s, fused = two_calls(**kw), make(**kw)
    s.step()
    fused.step()
    torch.cuda.synchronize()
    M, N = s.C.shape
    plain = bs.bsgemm_fp8(s.A, s.a_scale, s.B, s.b_scale).view(M, N)
    ids = s.ids.cpu().numpy()
    d, bound = opsref.delta(values(s.H), values(s.lora_B), values(s.lora_scale), ids)
    want = values(plain) + d
    assert bounds.within(bits16(s.C), want, bound + opsref.U * np.abs(want))[0].all()
    none = to_dev(ids < 0)
    assert torch.equal(s.C[none].view(torch.int16), fused.C[none].view(torch.int16))
    rows = M // s.bands
    q, sc = bs.band_rowq_e4m3([s.C[:rows]] + s.partials)
    assert torch.equal(s.wire_q[:rows], q) and torch.equal(s.wire_s[:rows], sc)


def test_capture_and_replay():
    say("serve step by two calls, captured")
    s, other = two_calls(seed=1), two_calls(seed=2)
    stream = torch.cuda.Stream(device=device())
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.step()
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
