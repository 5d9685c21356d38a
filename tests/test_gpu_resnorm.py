"""GPU parity of resnorm against a plain float64 implementation (opsref.py):
every input form, every output form, short and long rows, and single rows."""
import itertools

import numpy as np
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
import opsref
from gpuutil import bits16, device, say, to_dev
from oracle import bounds

pytestmark = pytest.mark.gpu


def bf(x):
    return to_dev(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16)


def values(t):
    return None if t is None else t.double().cpu().numpy()


def inputs(rows, N, wire, post, gate, f32, seed=0):
    rng = np.random.default_rng(seed)
    y = rng.standard_normal((rows, N)) * np.exp(rng.standard_normal((rows, 1)))
    kw = {}
    if wire:
        q, s = bs.rowq_e4m3(bf(y))
        yv = values(q.view(torch.float8_e4m3fn)) * values(s)[:, None]
        y = q
        kw["y_scale"] = s
    else:
        y = bf(y)
        yv = values(y)
    r = rng.standard_normal((rows, N)) * 2
    r = to_dev(r.astype(np.float32)) if f32 else bf(r)
    if post:
        kw["post_w"] = bf(1 + 0.2 * rng.standard_normal(N))
    if gate:
        kw["gate"] = bf(rng.standard_normal(N if gate == "channel" else (rows, N)))
    kw["pre_w"] = bf(1 + 0.2 * rng.standard_normal(N))
    return y, yv, r, kw


def check(rows, N, wire=False, post=True, gate="channel", f32=False, quant=0, z=True, inplace=False, seed=0,
          alpha=0.75, beta=0.5, eps=1e-6, pre=True):
    say(f"resnorm rows={rows} N={N} wire={wire} post={post} gate={gate} f32={f32} quant={quant} z={z} "
        f"inplace={inplace}")
    y, yv, r, kw = inputs(rows, N, wire, post, gate, f32, seed)
    if not pre:
        del kw["pre_w"]
    n = rows * N
    rt = torch.float32 if f32 else torch.bfloat16

    def guarded(count, dtype, fill):
        full = torch.full((count + 128,), fill, dtype=dtype, device=device())
        return full, full[64:64 + count]
    bufs = [guarded(n, rt, -3.0), guarded(n, torch.bfloat16, -3.0) if z else None]
    if quant:
        bufs += [guarded(n, torch.uint8, 0x7F),
                 guarded(n // quant, torch.float32, -3.0) if quant == 128 else guarded(n // quant, torch.uint8, 3)]
    rv = values(r)
    if inplace:
        bufs[0][1].copy_(r.view(-1))
        r = bufs[0][1].view(rows, N)
    ro, zo, q, sc = bs.resnorm(y, r, alpha=alpha, beta=beta, eps=eps, quant=quant, resid_out=bufs[0][1].view(rows, N),
                               z=bufs[1][1].view(rows, N) if z else None,
                               q=bufs[2][1].view(rows, N) if quant else None,
                               q_scale=bufs[3][1].view(rows, -1) if quant else None, **kw)
    torch.cuda.synchronize()
    for b in bufs:
        if b is not None:
            full = b[0].cpu()
            g = torch.cat([full[:64], full[-64:]])
            assert bool((g == g[0]).all()), "guard elements were written"
    h, eh, zz, ez = opsref.resnorm(yv, rv, values(kw.get("post_w")), values(kw.get("gate")), values(kw.get("pre_w")),
                                   alpha, beta, eps)
    if f32:
        assert np.all(np.abs(values(ro) - h) <= eh + opsref.U * np.abs(h))
    else:
        assert bounds.within(bits16(ro), h, eh)[0].all()
    if z:
        assert bounds.within(bits16(zo), zz, ez)[0].all()
    if quant:
        s = values(sc) if quant == 128 else np.where(sc.cpu().numpy() == 0, 2.0 ** -127, 2.0 ** (sc.cpu().numpy() - 127.0))
        opsref.check_quant(q.cpu().numpy(), s, zz, ez, quant)
    return ro, zo, q, sc


@pytest.mark.parametrize("wire,f32", itertools.product((False, True), (False, True)))
@pytest.mark.parametrize("quant", [0, 32, 128])
def test_forms(wire, f32, quant):
    for post, gate in itertools.product((False, True), (None, "channel", "full")):
        check(5, 1152, wire, post, gate, f32, quant)


@pytest.mark.parametrize("rows,N", [(1, 8), (3, 24), (2, 504), (1, 1016), (7, 1024), (2, 1032), (9, 2048), (1, 4096),
                                    (2, 4104), (1, 7168), (3, 5120), (4, 8192), (2, 8200), (1, 16384), (5, 16376),
                                    (1000, 136)])
def test_row_lengths(rows, N):
    check(rows, N, wire=rows % 2 == 0)


@pytest.mark.parametrize("rows,N,quant", [(1, 32, 32), (3, 96, 32), (1, 7168, 128), (2, 16384, 128), (2, 16384, 32),
                                          (5, 128, 128), (3, 8320, 128), (2, 4128, 32), (300, 640, 128),
                                          (2512, 7168, 128), (4000, 512, 32)])
def test_quantized_row_lengths(rows, N, quant):
    check(rows, N, wire=True, post=rows % 2 == 1, gate=None, quant=quant, z=False)
    check(rows, N, f32=True, quant=quant, z=True, pre=rows % 2 == 1)


def test_in_place_and_without_z():
    check(33, 1024, inplace=True)
    check(33, 1024, f32=True, inplace=True, quant=128, z=False)


def test_signs_and_multipliers():
    check(9, 640, alpha=-1.0, beta=2.0)
    check(9, 640, alpha=0.0, beta=1.0, quant=128)
    check(9, 640, alpha=1.0, beta=0.0, quant=32)
    check(9, 640, eps=0.5)


@pytest.mark.parametrize("quant", [32, 128])
def test_zero_rows(quant):
    """A row of zeros stays zero: no division by it, scale 0, codes 0."""
    say(f"resnorm zero rows quant={quant}")
    z0 = torch.zeros((3, 512), dtype=torch.bfloat16, device=device())
    r, z, q, s = bs.resnorm(z0, z0, post_w=torch.ones_like(z0[0]), quant=quant, z=torch.empty_like(z0))
    for t in (r, z, q, s):
        assert not bool(t.view(torch.uint8).any())


def test_mx_scales_at_the_power_of_two_border():
    """Blocks whose largest value is 448 * 2^k exactly, and one fp32 step to either
    side of it: the scale goes up only past it.  alpha = 1 and a row of known
    squares give z = resid * rs with rs a power of two."""
    say("resnorm mx border")
    N = 128
    rows = []
    for m in (1.75, np.nextafter(np.float32(1.75), np.float32(2)), np.nextafter(np.float32(1.75), np.float32(1))):
        v = np.zeros(N, np.float32)
        v[0] = m
        v[64] = np.sqrt(N * 4.0 - 1e-6 - float(m) ** 2)
        rows.append(v)
    r = to_dev(np.stack(rows))
    y = torch.zeros((3, N), dtype=torch.bfloat16, device=device())
    _, _, q, s = bs.resnorm(y, r, quant=32)
    _, _, zz, ez = opsref.resnorm(np.zeros((3, N)), values(r), None, None, None, 1.0, 1.0, 1e-6)
    sv = np.where(s.cpu().numpy() == 0, 2.0 ** -127, 2.0 ** (s.cpu().numpy() - 127.0))
    opsref.check_quant(q.cpu().numpy(), sv, zz, ez, 32)


def test_repeated_runs_are_identical():
    a = check(700, 7168, wire=True, post=True, gate="full", quant=128, seed=3)
    b = check(700, 7168, wire=True, post=True, gate="full", quant=128, seed=3)
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_agrees_with_the_separate_calls():
    """The wire path against rowdq_e4m3, torch's own add and actq_e4m3, which round
    to bf16 in between: each of those roundings moves a value by 2^-8 at most."""
    say("resnorm against the separate calls")
    rows, N = 64, 7168
    y, yv, r, kw = inputs(rows, N, True, False, None, False)
    ro, z, q, s = bs.resnorm(y, r, quant=128, z=torch.empty_like(r), **kw)
    h = (bs.rowdq_e4m3(y, kw["y_scale"]).float() + r.float()).to(torch.bfloat16)
    scale = bs.rowdq_e4m3(y, kw["y_scale"]).float().abs() + r.float().abs()
    assert bool(((ro.float() - h.float()).abs() <= 2.0 ** -8 * 2 * scale).all())
    q2, s2 = bs.actq_e4m3(z)
    assert bool(((s - s2).abs() <= 2.0 ** -8 * s2).all())
