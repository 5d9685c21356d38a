"""The adapter operators and resnorm on buffers of more than 2^31 elements: the
first rows, rows on either side of 2^31 elements and the last ones are compared
with the same rows computed in a small batch, bit for bit, which the small
tests hold to float64."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
import opsref
from gpuutil import device, say, to_dev

pytestmark = pytest.mark.gpu

N = 7168
M = 300032   # M * N = 2^31 + 3.2 M elements


def probe(rows, width):
    """Row numbers at the start, around 2^31 elements and at the end."""
    mid = 2**31 // width
    return np.unique(np.concatenate([np.arange(3), np.clip(np.arange(mid - 2, mid + 3), 0, rows - 1),
                                     np.arange(rows - 3, rows)]))


def gen():
    return torch.Generator(device=device()).manual_seed(0)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_expand_and_gemm():
    say(f"lora_expand, bsgemm_fp8_lora M={M} N={N}")
    d, g = device(), gen()
    L, R, K = 3, 16, 128
    H = torch.randn((M, R), generator=g, device=d)
    B = torch.randn((L, N, R), generator=g, device=d).to(torch.bfloat16)
    ids = torch.randint(-1, L, (M,), generator=g, device=d, dtype=torch.int32)
    base = torch.empty(M * N, dtype=torch.bfloat16, device=d)
    for i in range(0, M, 50016):
        base[i * N:min(M, i + 50016) * N].normal_(generator=g)
    out = torch.empty_like(base)
    plan = bs.lora_plan(ids, L)
    at = probe(M, N)
    rows = to_dev(at)
    assert np.array_equal(plan.cpu().numpy(), opsref.plan(ids.cpu().numpy(), L))
    bs.lora_expand(H, B, plan, base, out)
    few = ids[rows].contiguous()
    want = bs.lora_expand(H[rows], B, bs.lora_plan(few, L), base.view(M, N)[rows].contiguous())
    torch.cuda.synchronize()
    assert same(out.view(M, N)[rows], want.view(-1, N))
    del base
    qa, sa = bs.actq_e4m3(torch.randn((M, K), generator=g, device=d).to(torch.bfloat16))
    qb, sb = bs.blockq_e4m3(torch.randn((N, K), generator=g, device=d), 128)
    bs.bsgemm_fp8_lora(qa, sa, qb, sb, H, B, ids, C=out)
    want = bs.bsgemm_fp8_lora(qa[rows], sa[rows], qb, sb, H[rows], B, few)
    torch.cuda.synchronize()
    # another kernel, which adds in the same order
    assert same(out.view(M, N)[rows], want.view(-1, N))


def test_shrink():
    say(f"lora_shrink M={M} K={N}")
    d, g = device(), gen()
    L, R = 3, 8
    x = torch.empty((M, N), dtype=torch.bfloat16, device=d)
    at = probe(M, N)
    rows = to_dev(at)
    x.zero_()
    x[rows] = torch.randint(-3, 4, (len(at), N), generator=g, device=d).to(torch.bfloat16)
    A = torch.randint(-3, 4, (L, R, N), generator=g, device=d).to(torch.bfloat16)
    ids = torch.randint(-1, L, (M,), generator=g, device=d, dtype=torch.int32)
    H = bs.lora_shrink(x, A, bs.lora_plan(ids, L))
    want, _ = opsref.shrink(x[rows].double().cpu().numpy(), A.double().cpu().numpy(), ids[rows].cpu().numpy())
    assert np.array_equal(H[rows].double().cpu().numpy(), want)   # integers: exact
    H[rows] = 0
    assert not bool(H.any())


@pytest.mark.parametrize("quant", [0, 32, 128])
def test_resnorm(quant):
    say(f"resnorm rows={M} N={N} quant={quant}")
    d, g = device(), gen()
    y = torch.zeros((M, N), dtype=torch.uint8, device=d)
    at = probe(M, N)
    rows = to_dev(at)
    y[rows] = torch.randint(0, 0x7E, (len(at), N), generator=g, device=d, dtype=torch.uint8)
    s = torch.rand(M, generator=g, device=d)
    r = torch.zeros((M, N), dtype=torch.bfloat16, device=d)
    r[rows] = torch.randn((len(at), N), generator=g, device=d).to(torch.bfloat16)
    got = bs.resnorm(y, r, y_scale=s, quant=quant)
    # as many rows as take the same form of the kernel
    pad = lambda t: torch.cat([t[rows]] + [t[:1]] * (1024 - len(at))).contiguous()  # noqa: E731
    want = bs.resnorm(pad(y), pad(r), y_scale=pad(s), quant=quant)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert (a is None) == (b is None)
        if a is not None:
            assert same(a.view(M, -1)[rows], b.view(1024, -1)[:len(at)])
