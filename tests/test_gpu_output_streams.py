"""A call on a stream that is not the current one, with outputs that it allocates: their
memory is none that the current stream still uses."""
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
from gpuutil import device, say

pytestmark = pytest.mark.gpu

SPIN_CYCLES = 50_000_000   # ~25 ms of torch's spin kernel


def calls():
    """name -> the call, given its stream; inputs are ready on every stream."""
    g = torch.Generator(device=device()).manual_seed(0)
    M, N, K, L, R = 256, 512, 384, 3, 16

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=device()).to(dtype)
    x, w, y = normal(M, K), normal(N, K, dtype=torch.float32), normal(M, N)
    A, mx = bs.actq_e4m3(x), bs.mxq_e4m3(x)
    B, mb = bs.blockq_e4m3(w, 128), bs.mxq_e4m3(w.to(torch.bfloat16))
    Bp = bs.bprepack_e4m3(B[0])
    ids = torch.randint(-1, L, (M,), generator=g, device=device(), dtype=torch.int32)
    plan = bs.lora_plan(ids, L)
    la, lb = normal(L, R, K), normal(L, N, R)
    H = bs.lora_shrink(x, la, plan)
    q, s = bs.rowq_e4m3(y)
    return {
        "bsgemm_fp8": lambda st: bs.bsgemm_fp8(*A, *B, stream=st),
        "bsgemm_fp8_pb": lambda st: bs.bsgemm_fp8_pb(*A, Bp, B[1], stream=st),
        "mxgemm_fp8": lambda st: bs.mxgemm_fp8(*mx, *mb, stream=st),
        "band_reduce": lambda st: bs.band_reduce([y, y], stream=st),
        "band_rowq_e4m3": lambda st: bs.band_rowq_e4m3([y, y], stream=st),
        "rowq_e4m3": lambda st: bs.rowq_e4m3(y, stream=st),
        "rowdq_e4m3": lambda st: bs.rowdq_e4m3(q, s, stream=st),
        "blockq_e4m3": lambda st: bs.blockq_e4m3(w, 1, stream=st),
        "actq_e4m3": lambda st: bs.actq_e4m3(x, stream=st),
        "mxq_e4m3": lambda st: bs.mxq_e4m3(x, stream=st),
        "bprepack_e4m3": lambda st: bs.bprepack_e4m3(B[0], stream=st),
        "lora_plan": lambda st: bs.lora_plan(ids, L, stream=st),
        "lora_shrink": lambda st: bs.lora_shrink(x, la, plan, stream=st),
        "lora_expand": lambda st: bs.lora_expand(H, lb, plan, y.view(-1), stream=st),
        "bsgemm_fp8_lora": lambda st: bs.bsgemm_fp8_lora(*A, *B, H, lb, ids, stream=st),
        "resnorm": lambda st: bs.resnorm(y, y, stream=st),
        "resnorm to codes": lambda st: bs.resnorm(y, y, quant=128, stream=st),
    }


def tensors(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


def test_outputs_belong_to_the_stream_that_is_given():
    """Tensors of the outputs' sizes are freed while the current stream has yet to
    fill them; the call on another stream must not be given their memory."""
    stream = torch.cuda.Stream(device=device())
    for name, call in calls().items():
        say(f"outputs on another stream: {name}")
        want = tensors(call(None))
        torch.cuda.synchronize()
        late = [torch.empty_like(t) for t in want]
        torch.cuda._sleep(SPIN_CYCLES)
        for t in late:
            t.view(torch.uint8).fill_(0x55)
        del late, t
        got = tensors(call(stream))
        torch.cuda.synchronize()
        assert len(got) == len(want)
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
