"""FFNServeStep refuses operands whose shapes do not belong together, also where every single
call would take them and leave a part of its output unwritten."""
import pytest
import torch

from block_scaled_fp8_bsgemm_amd.pipeline import FFNServeStep

M, D, I = 4, 256, 384


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def dense(rows=2 * I, D1=D, D2=D, I2=I):
    return u8(rows, D1), torch.ones((rows // 128, D1 // 128)), u8(D2, I2), torch.ones((D2 // 128, I2 // 128))


def step(M1=M, D1=D, z=True, **kw):
    return FFNServeStep(torch.zeros((M, D), dtype=torch.bfloat16) if z else None, u8(M1, D1), torch.ones((M1, D1 // 128)),
                        dense(**kw))


def test_shapes_that_fit():
    for z in (True, False):
        s = step(z=z)
        assert s.out.shape == (M, D) and s.h.shape == (M, I) and s.PHASES == FFNServeStep.DENSE


@pytest.mark.parametrize("kw,match", [
    (dict(M1=2), r"q: shape \(2, 256\), expected \(4, 256\)"),          # rows of out that down would make of old h
    (dict(M1=8), "q: shape"),
    (dict(D1=128), "q: shape"),
    (dict(rows=2 * I - 256), "dense B13: shape"),                       # columns of h that up would leave
    (dict(rows=2 * I + 256), "dense B13: shape"),
    (dict(D2=128), r"dense B2: shape \(128, 384\), expected \(256, 384\)"),   # columns of out that down would leave
    (dict(D2=384), "dense B2: shape"),
    (dict(I2=128), "dense B13: shape"),
    (dict(z=False, D2=128), "dense B2: shape"),
])
def test_shapes_that_do_not(kw, match):
    with pytest.raises(ValueError, match=match):
        step(**kw)
