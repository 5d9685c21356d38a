"""bsgemm_fp8_act: a row's result is the same bit for bit in every batch, whatever kernel the
sizes choose, with factors that are no powers of two, a bias, a residual and each activation."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
import ffnref
from gpuutil import bits16, device, say, to_dev
from oracle import bounds
from test_gpu_act import exact_acc, operands
from test_gpu_lora import bf, values

pytestmark = pytest.mark.gpu

BATCHES = (2100, 700, 64, 20, 16, 1)   # whole tiles, 64 x 128 tiles, 64, 32 and 16 rows to a workgroup


# K / 128 even: gated whole tiles by the persistent kernel, odd: by the tile kernel
@pytest.mark.parametrize("K", [512, 640])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ffnref.ACTS)
def test_every_kernel_rounds_alike(act, gated, K):
    N = 2304
    say(f"bsgemm_fp8_act batches {act} gated={gated} K={K}")
    rows = 2 * N if gated else N
    qa, sa, qb, sb = (to_dev(a) for a in operands(BATCHES[0], rows, K, 9, False))
    g = torch.Generator(device=device()).manual_seed(K)
    bias = torch.randn(rows, generator=g, device=device()).to(torch.bfloat16)
    resid = torch.randn((BATCHES[0], N), generator=g, device=device()).to(torch.bfloat16)
    for b, r, alpha, beta in ((True, True, 0.7, 0.3), (False, False, 1.0, 1.25), (True, False, 1.0, 0.3),
                              (False, True, 1.0, 1.0), (False, True, 0.1, 1.0), (True, True, 1.0, 1.25)):
        ref = None
        for M in BATCHES:
            got = bs.bsgemm_fp8_act(qa[:M].contiguous(), sa[:M].contiguous(), qb, sb, bias if b else None, act, gated,
                                    resid[:M].contiguous() if r else None, alpha, beta).view(M, N)
            ref = got if ref is None else ref
            diff = int((got.view(torch.int16) != ref[:M].view(torch.int16)).sum())
            assert diff == 0, (b, r, alpha, beta, M, diff)


@pytest.mark.parametrize("gated", [False, True])
def test_factors(gated):
    """alpha and beta of either sign and zero against float64, at every kernel's batch."""
    N, K = 2304, 256
    rows = 2 * N if gated else N
    host = operands(2100, rows, K, 4, True)
    acc = exact_acc(host)
    rng = np.random.default_rng(1)
    bias, resid = bf(rng.standard_normal(rows)), bf(rng.standard_normal((2100, N)) * 50)
    ops = [to_dev(a) for a in host]
    for alpha, beta in ((-0.3, 0.9), (0.0, -1.7), (1e-3, 0.0)):
        want, tol = ffnref.epilogue(acc, np.zeros_like(acc), values(bias), "silu", gated, values(resid), alpha, beta)
        for M in BATCHES:
            say(f"bsgemm_fp8_act alpha={alpha} beta={beta} gated={gated} M={M}")
            got = bs.bsgemm_fp8_act(ops[0][:M].contiguous(), ops[1][:M].contiguous(), *ops[2:], bias, "silu", gated,
                                    resid[:M].contiguous(), alpha, beta).view(M, N)
            # alpha and beta reach the kernel as fp32: half a step of each, relative to its term
            near = ffnref.U * (np.abs(want[:M]) + 2 * np.abs(alpha * values(resid[:M])))
            ok, used = bounds.within(bits16(got), want[:M], tol[:M] + near)
            assert ok.all(), float(used.max())
