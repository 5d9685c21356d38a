"""Adapters of more than 2^31 bytes each beside outputs of millions of columns: windows
of columns at the start, around 2^31 bytes of an adapter and at the end against the
same call on those columns alone, bit for bit."""
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
from gpuutil import device, say

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def windows(N, R, step):
    mid = 2**31 // (2 * R) // step * step
    return [(0, 512), (mid - 512, mid + 512), ((N - 700) // step * step, N)]


@pytest.mark.parametrize("M", [3, 70, 300])
def test_columns(M):
    L, R, N, K = 2, 256, (1 << 22) + 1152, 128
    say(f"lora_expand, bsgemm_fp8_lora M={M} N={N} R={R}")
    d = device()
    g = torch.Generator(device=d).manual_seed(M)
    B = torch.empty((L, N, R), dtype=torch.bfloat16, device=d).normal_(generator=g)
    H = torch.randn((M, R), generator=g, device=d)
    ids = torch.randint(-1, L, (M,), generator=g, device=d, dtype=torch.int32)
    plan = bs.lora_plan(ids, L)
    base = torch.empty((M, N), dtype=torch.bfloat16, device=d).normal_(generator=g)
    out = bs.lora_expand(H, B, plan, base.view(-1)).view(M, N)
    for lo, hi in windows(N, R, 8):
        want = bs.lora_expand(H, B[:, lo:hi].contiguous(), plan, base[:, lo:hi].contiguous().view(-1))
        assert same(out[:, lo:hi], want.view(M, -1)), lo
    A = bs.actq_e4m3(torch.randn((M, K), generator=g, device=d).to(torch.bfloat16))
    w = torch.randint(0, 0x7F, (N, K), generator=g, device=d, dtype=torch.uint8)
    ws = torch.rand((N // 128, 1), generator=g, device=d)
    C = bs.bsgemm_fp8_lora(*A, w, ws, H, B, ids).view(M, N)
    for lo, hi in windows(N, R, 128):
        want = bs.bsgemm_fp8_lora(*A, w[lo:hi], ws[lo // 128:hi // 128], H, B[:, lo:hi].contiguous(), ids)
        assert same(C[:, lo:hi], want.view(M, -1)), lo
    torch.cuda.synchronize()
