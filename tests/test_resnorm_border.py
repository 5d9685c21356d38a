"""resnorm's block scales where the definition turns: rows whose normed values are known
bit for bit, their blocks' largest at 448 * 2^k and one fp32 step to either side.

A row of 512 has two elements 2^13 in its last block of 128 and one, m with
1.7 < m < 1.8, in its first block.  m^2 is below 3.3, less than half a step of
2^26 in fp32 (4), so however the squares are added they sum to 2^27 exactly, and
the mean is 2^18 (eps, 1e-6, is far below its half step).  With y = 0 and
alpha = 1, h is the residual, and z = h * 2^-9 * w with w a power of two: exact."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs

N = 512
HALF = np.float32(1.75)   # 448 = 1.75 * 2^8
BORDER = [HALF, np.nextafter(HALF, np.float32(2)), np.nextafter(HALF, np.float32(1)),
          np.float32(1.7), np.float32(1.8)]
WEIGHTS = [0, -60, 60, -109, 100]   # exponents of w


def rows():
    r = np.zeros((len(BORDER), N), np.float32)
    r[:, 0] = BORDER
    r[:, 400] = r[:, 432] = 2.0 ** 13
    return r


def mx_byte(z, past=lambda a, b: a > b):
    """E8M0 byte of a block whose largest value is z: the least k >= -127 with
    z <= 448 * 2^k, in rational arithmetic; `past` tells z from the border."""
    k = -127
    while past(Fraction(float(z)), 448 * Fraction(2) ** k):
        k += 1
    return k + 127


def normed(w):
    """z of the first and of the two large elements, [rows, 3] float32."""
    z = rows()[:, [0, 400, 432]].astype(np.float64) * 2.0 ** (w - 9)
    assert np.array_equal(z, z.astype(np.float32))
    return z.astype(np.float32)


def codes(x):
    return torch.from_numpy(np.asarray(x, np.float64)).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def test_the_rows_tell_a_wrong_threshold():
    """The sums are what the rows were built for in any order, and a threshold that
    takes the border itself, or is one fp32 step off, gives another byte."""
    r, rng = rows(), np.random.default_rng(0)
    for row in r:
        for _ in range(20):
            total = np.float32(0)
            for v in rng.permutation(row):
                total = np.float32(total + v * v)
            assert total == 2.0 ** 27
        assert np.float32(np.float32(2.0 ** 27 / N) + np.float32(1e-6)) == 2.0 ** 18
    step = Fraction(2) ** -23
    for w in WEIGHTS:
        z = normed(w)[:, 0]
        right = [mx_byte(v) for v in z]
        assert right[1] == right[0] + 1 and right[2] == right[0] and right[3] == right[0] and right[4] == right[1]
        for wrong in (lambda a, b: a >= b, lambda a, b: a > b * (1 + step), lambda a, b: a > b * (1 - step)):
            assert [mx_byte(v, wrong) for v in z] != right


@pytest.mark.gpu
@pytest.mark.parametrize("quant", [32, 128])
def test_scales_at_the_border(quant):
    from gpuutil import say, to_dev
    y = to_dev(np.zeros((len(BORDER), N), np.float32)).to(torch.bfloat16)
    for w in WEIGHTS:
        say(f"resnorm border quant={quant} w=2^{w}")
        pre = torch.full_like(y[0], 2.0 ** w)
        _, zb, q, s = bs.resnorm(y, to_dev(rows()), pre_w=pre, quant=quant, z=torch.empty_like(y))
        torch.cuda.synchronize()
        z = normed(w)
        q, s = q.cpu().numpy(), s.cpu().numpy()
        at = [0, 400, 432]
        got = s[:, [c // quant for c in at]]
        if quant == 32:
            want = np.array([[mx_byte(v) for v in row] for row in z], np.uint8)
            scale = 2.0 ** (want.astype(float) - 127)
        else:
            want = (z / np.float32(448)).astype(np.float32)
            scale = want.astype(float)
        assert np.array_equal(got, want)
        # a block's largest value: 448 or next to it by the 1x128 scale, z / 2^k by the 1x32 one
        assert np.array_equal(q[:, at], codes(np.minimum(z / scale, 448.0)))
        assert torch.equal(zb[:, at].float().cpu(), torch.from_numpy(z).to(torch.bfloat16).float())
        rest = np.delete(np.arange(N), at)
        assert not q[:, rest].any()
