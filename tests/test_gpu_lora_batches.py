"""A row's adapter results are the same in every batch, bit for bit: rows of one
long batch against shorter ones on either side of each size at which another form
of a kernel takes over."""
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
from gpuutil import device, say

pytestmark = pytest.mark.gpu

CUTS = [(0, 1), (8999, 9000), (5, 37), (0, 200), (100, 611), (100, 612), (0, 1024), (7, 2054), (7, 2055), (500, 4596),
        (3, 8194), (3, 8195)]


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("K,N,L,R", [(2048, 1152, 5, 72), (640, 2304, 40, 16), (384, 1024, 3, 136)])
def test_a_row_does_not_depend_on_its_batch(K, N, L, R):
    M = 9000
    g = torch.Generator(device=device()).manual_seed(K)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=device()).to(dtype)
    x, base = normal(M, K), normal(M, N)
    A, B = normal(L, R, K), normal(L, N, R)
    scale = torch.rand(L, generator=g, device=device()) + 0.5
    w = bs.blockq_e4m3(normal(N, K, dtype=torch.float32), 128)
    for mix in ("tokens", "runs"):
        ids = torch.randint(-1, L, (M,) if mix == "tokens" else (M // 60,), generator=g, device=device(),
                            dtype=torch.int32)
        if mix == "runs":
            ids = ids.repeat_interleave(60).contiguous()

        def run(lo, hi):
            i, xs = ids[lo:hi].clone(), x[lo:hi].clone()
            plan = bs.lora_plan(i, L)
            H = bs.lora_shrink(xs, A, plan)
            return (H, bs.lora_expand(H, B, plan, base[lo:hi].clone(), scale=scale).view(-1, N),
                    bs.bsgemm_fp8_lora(*bs.actq_e4m3(xs), *w, H, B, i, scale).view(-1, N))
        want = run(0, M)
        for lo, hi in CUTS:
            say(f"adapters in batches: K={K} N={N} L={L} R={R} {mix} rows {lo}..{hi}")
            got = run(lo, hi)
            torch.cuda.synchronize()
            for k, (a, b) in enumerate(zip(got, want)):
                assert same(a, b[lo:hi]), k
