"""resnorm row by row: a row's result is the same in every batch, bit for bit."""
import itertools

import numpy as np
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
from gpuutil import device, say

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def inputs(rows, N, wire, f32, seed=0):
    """y, resid and keyword arguments; the gate holds a row for each row."""
    g = torch.Generator(device=device()).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=device())
    y, kw = normal(rows, N).to(torch.bfloat16), {}
    if wire:
        y = torch.randint(0, 0x7F, (rows, N), generator=g, device=device(), dtype=torch.uint8)
        kw["y_scale"] = torch.rand(rows, generator=g, device=device()) * 0.01
    r = normal(rows, N) * 2
    r = r if f32 else r.to(torch.bfloat16)
    kw.update(gate=normal(rows, N).to(torch.bfloat16), post_w=normal(N).to(torch.bfloat16),
              pre_w=normal(N).to(torch.bfloat16), alpha=0.75, beta=0.5)
    return y, r, kw


def run(y, r, kw, rows, quant):
    """The call on the given rows alone; z is written besides q."""
    kw = {k: v[rows].clone() if k in ("gate", "y_scale") else v for k, v in kw.items()}
    z = torch.empty(y[rows].shape, dtype=torch.bfloat16, device=device())
    return bs.resnorm(y[rows].clone(), r[rows].clone(), quant=quant, z=z, **kw)


@pytest.mark.parametrize("N", [640, 1024, 1032, 1152, 2176, 4096, 5120, 7168, 8192, 8200, 16384])
def test_a_row_does_not_depend_on_its_batch(N):
    """Rows on either side of every batch size at which the kernel's form may change."""
    rows = 1500
    for wire, f32 in itertools.product((False, True), (False, True)):
        for quant in [0] + [b for b in (32, 128) if N % b == 0]:
            say(f"resnorm batches N={N} wire={wire} f32={f32} quant={quant}")
            y, r, kw = inputs(rows, N, wire, f32, N)
            want = run(y, r, kw, slice(0, rows), quant)
            for lo, hi in [(0, 1), (777, 778), (1499, 1500), (3, 10), (0, 511), (0, 512), (500, 1100)]:
                got = run(y, r, kw, slice(lo, hi), quant)
                for k, (g, w) in enumerate(zip(got, want)):
                    assert (g is None) == (w is None)
                    assert g is None or same(g, w[lo:hi]), (lo, hi, k)
