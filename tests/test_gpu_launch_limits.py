"""The widest products of 64 x 128 tiles, whose workgroups rounded up to the 8 XCDs would be
2^32 lanes."""
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
from gpuutil import device, say

pytestmark = pytest.mark.gpu


def test_act_at_2_32_lanes():
    """2^23 - 1 tiles, gated 2^23 - 2, and 2^23 - 8 of both.  B has 128 GiB."""
    N, K = (1 << 30) - 128, 128
    dev = device()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GiB of free device memory")
    A = torch.zeros((1, K), dtype=torch.uint8, device=dev)
    A[0, 77] = 0x38                                   # 1.0
    sa = torch.ones((1, 1), dtype=torch.float32, device=dev)
    B = torch.full((N, K), 0x40, dtype=torch.uint8, device=dev)     # 2.0
    sb = (torch.arange(N // 128, device=dev) % 5 + 1).to(torch.float32).view(-1, 1)
    # the first 64 x 128 tiles that no launch holds, and the most that one does
    for n, gated in ((N, False), (N // 2 // 128 * 128, True), ((1 << 30) - 1024, False), ((1 << 29) - 512, True)):
        say(f"bsgemm_fp8_act 1 row of {n} columns, gated={gated}")
        C = torch.full((n,), float("nan"), dtype=torch.bfloat16, device=dev)
        rows = 2 * n if gated else n
        bs.bsgemm_fp8_act(A, sa, B[:rows], sb[:rows // 128], act="relu", gated=gated, C=C)
        t = 2.0 * sb.view(-1)[:rows // 128]
        want = t[:n // 128] * t[n // 128:] if gated else t
        assert bool((C.view(-1, 128) == want.bfloat16()[:, None]).all()), (n, gated)
        del C
    del B
    torch.cuda.empty_cache()
