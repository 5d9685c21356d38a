"""Products of more tiles than one launch holds are refused: 2^23 workgroups of 512 lanes, 8 to
a step, would be 2^32 lanes, which the runtime refuses or takes for none.  Every call here is
refused before a launch, since the pointers are fake."""
import pytest

import block_scaled_fp8_bsgemm_amd as bs

UNS = bs.BS_ERR_UNSUPPORTED
GIB = 1 << 30
# A, a_scale, B, b_scale, C and the rest, far apart: B may have 256 GiB
A, SA, B, SB, C, X, Y, Z = (GIB * (1 + 1024 * i) for i in range(8))
N = (1 << 31) - 128     # 2^23 tiles, and with one 128 columns narrower 2^23 - 1, rounded up


@pytest.fixture(scope="module")
def L():
    return bs.load()


@pytest.mark.parametrize("n", [N, N - 128, N - 7 * 256])
def test_products(L, n):
    assert L.bsgemm_fp8(A, SA, B, SB, C, 1, n, 128, 1, 0, None) == UNS
    assert L.bsgemm_fp8_pb(A, SA, B, SB, C, 1, n, 128, 1, 0, None) == UNS
    assert L.mxgemm_fp8(A, SA, B, SB, C, 1, n, 128, 1, 0, None) == UNS
    assert L.bsgemm_fp8_act(A, SA, B, SB, None, None, C, 1, n, 128, 2, 0, 1.0, 1.0, 1, 0, None) == UNS
    assert L.bsgemm_fp8_lora(A, SA, B, SB, X, Y, None, Z, C, 1, n, 128, 4, 16, 1, 0, None) == UNS
    if n % 256 == 0:
        assert L.bsgemm_fp8_act(A, SA, B, SB, None, None, C, 1, n // 2, 128, 2, 1, 1.0, 1.0, 1, 0, None) == UNS


def test_rows(L):
    for f in (L.bsgemm_fp8, L.bsgemm_fp8_pb, L.mxgemm_fp8):
        assert f(A, SA, B, SB, C, 1 << 30, 2048, 128, 1, 0, None) == UNS
        assert f(A, SA, B, SB, C, 0, N, 128, 1, 0, None) == bs.BS_OK      # no rows, no tiles
