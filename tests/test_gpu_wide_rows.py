"""Whole tiles whose rows are millions of elements long, where the persistent kernels' stores
come to 2^31 bytes from a tile's first element and past them: the widest rows that those
kernels take, the next, and the widest whose B they could address."""
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
from gpuutil import device, say

pytestmark = pytest.mark.gpu

M, K = 300, 256
WIDTHS = (4210688, 4210688 + 256, (1 << 23) - 512)


@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("what", ["bsgemm_fp8", "mxgemm_fp8", "gated"])
def test_every_row_is_written(what, N):
    say(f"{what}: {M} rows of {N} columns")
    assert (N + 256) * K <= 0x7FFFFFFF    # B by itself fits the persistent kernels
    dev = device()
    A = torch.zeros((M, K), dtype=torch.uint8, device=dev)
    row = torch.arange(M, device=dev) % 13 - 6
    A[:, 200] = row.float().to(torch.float8_e4m3fn).view(torch.uint8)
    B = torch.zeros((N, K), dtype=torch.uint8, device=dev)
    col = torch.arange(N, device=dev) % 11 - 5
    B[:, 200] = col.float().to(torch.float8_e4m3fn).view(torch.uint8)
    if what == "mxgemm_fp8":
        one = [torch.full((n, K // 32), 127, dtype=torch.uint8, device=dev) for n in (M, N)]
        call = bs.mxgemm_fp8
    else:
        one = [torch.ones((n, K // 128), dtype=torch.float32, device=dev) for n in (M, N // 128)]
        call = bs.bsgemm_fp8
    if what == "gated":
        C = torch.full((M * (N // 2),), float("nan"), dtype=torch.bfloat16, device=dev)
        bs.bsgemm_fp8_act(A, one[0], B, one[1], act="none", gated=True, C=C)
        want, power = (col[: N // 2] * col[N // 2:]).bfloat16(), 2
    else:
        C = torch.full((M * N,), float("nan"), dtype=torch.bfloat16, device=dev)
        call(A, one[0], B, one[1], C)
        want, power = col.bfloat16(), 1
    C = C.view(M, -1)
    torch.cuda.synchronize()
    # products exact in fp32, then one rounding on either side
    wrong = [m for m in range(M) if not bool((C[m] == want * (int(row[m]) ** power)).all())]
    assert not wrong, (len(wrong), wrong[:5])
