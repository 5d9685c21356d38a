"""resnorm row by row: a row's result is the same in every batch, bit for bit, and what is
not finite in it reaches its own results and no other row's."""
import itertools

import numpy as np
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
import opsref
from gpuutil import bits16, device, say
from oracle import bounds

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


NAN, INF = float("nan"), float("inf")
SPOILS = [("y", NAN, False), ("y", INF, False), ("y", -INF, True), ("resid", NAN, False), ("resid", INF, True),
          ("resid", -INF, False), ("gate", NAN, True), ("y_scale", NAN, False), ("code", 0x7F, True)]


@pytest.mark.parametrize("N", [512, 1152, 5120])
@pytest.mark.parametrize("quant", [0, 32, 128])
def test_what_is_not_finite_stays_visible_and_in_its_row(N, quant):
    """One value of row 2 is NaN or infinite.  The other rows come out as they do
    without it.  Row 2 has the formula's NaN in z, a NaN scale and NaN codes in every
    block with such a z, zeros in the others; and the projection behind gives a
    row of NaN, its other rows unchanged."""
    rows, row, col = 7, 2, 300
    g = torch.Generator(device=device()).manual_seed(N)
    W = torch.randn((256, N), generator=g, device=device())
    for what, bad, post in SPOILS:
        say(f"resnorm not finite: N={N} quant={quant} {what}={bad} post={post}")
        wire, f32 = what in ("y_scale", "code"), what == "resid"
        y, r, kw = inputs(rows, N, wire, f32, N + 1)
        if not post:
            del kw["post_w"]
        want = run(y, r, kw, slice(0, rows), quant)
        y, r, kw = y.clone(), r.clone(), {k: v.clone() if torch.is_tensor(v) else v for k, v in kw.items()}
        if what == "y_scale":
            kw["y_scale"][row] = bad
        else:
            {"y": y, "code": y, "resid": r, "gate": kw["gate"]}[what][row, col] = bad
        got = run(y, r, kw, slice(0, rows), quant)
        torch.cuda.synchronize()
        others = torch.arange(rows, device=device()) != row
        for k, (a, b) in enumerate(zip(got, want)):
            assert (a is None) == (b is None)
            assert a is None or same(a[others], b[others]), (what, k)
        # an infinity in h makes 1 / rms 0, so z is NaN where it stands and 0 elsewhere; any
        # NaN, and an infinity that the norm after the block divides, makes all of it NaN
        one = np.isinf(bad) and not (what == "y" and post)
        nan = np.arange(N) == col if one else np.ones(N, bool)
        z = got[1][row].float().cpu().numpy()
        assert np.array_equal(np.isnan(z), nan) and not z[~nan].any(), what
        assert not np.isfinite(got[0][row].float().cpu().numpy()).all()
        if not quant:
            continue
        q, s = got[2][row].cpu().numpy().reshape(-1, quant), got[3][row].cpu().numpy()
        block = nan.reshape(-1, quant).any(1)
        assert ((q[block] & 0x7F) == 0x7F).all() and not q[~block].any(), what
        if quant == 128:
            assert np.array_equal(np.isnan(s), block) and not s[~block].any(), what
        else:
            assert (s[block] == 0xFF).all() and not s[~block].any(), what
        if quant == 128:
            B = bs.blockq_e4m3(W, 128)
            c, c0 = (bs.bsgemm_fp8(t[2], t[3], *B).view(rows, -1) for t in (got, want))
        else:
            B = bs.mxq_e4m3(W.to(torch.bfloat16))
            c, c0 = (bs.mxgemm_fp8(t[2], t[3], *B).view(rows, -1) for t in (got, want))
        torch.cuda.synchronize()
        assert bool(c[row].isnan().all()) and same(c[others], c0[others]), what


@pytest.mark.parametrize("quant", [32, 128])
def test_an_infinite_weight_spoils_its_block_alone(quant):
    """z is infinite in one column: no scale holds it, so its blocks decode to NaN."""
    say(f"resnorm infinite weight, quant={quant}")
    rows, N, col = 5, 1152, 700
    y, r, kw = inputs(rows, N, False, False, 1)
    want = run(y, r, kw, slice(0, rows), quant)
    kw["pre_w"] = kw["pre_w"].clone()
    kw["pre_w"][col] = INF
    got = run(y, r, kw, slice(0, rows), quant)
    torch.cuda.synchronize()
    hit = np.arange(N) // quant == col // quant
    keep = torch.from_numpy(~hit).to(device())
    assert bool(got[1][:, col].isinf().all()) and same(got[0], want[0]) and same(got[2][:, keep], want[2][:, keep])
    s = got[3].cpu().numpy()
    v = s.astype(float) if quant == 128 else np.where(s == 0xFF, np.nan, 2.0 ** (s.astype(float) - 127))
    code = got[2].view(torch.float8_e4m3fn).double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        assert np.isnan((code * v.repeat(quant, 1))[:, hit]).all()


def values(t):
    return None if t is None else t.double().cpu().numpy()


def large(what, N, f32):
    """Eight rows, of which every second one has values whose squares, or their sum,
    lie past fp32."""
    wire = what == "y_scale"
    y, r, kw = inputs(8, N, wire, f32, N + 2)
    kw["gate"] = kw["gate"].clamp(-4, 4)
    if what == "y":                      # the largest bf16 among them
        y[1::2] *= 2.0 ** 120
        y[3] = y[3].sign() * torch.finfo(torch.bfloat16).max
    elif what == "y_scale":
        kw["y_scale"][1::2] = 2.0 ** 100
    elif what == "border":               # the sum of squares just past fp32 and just below it
        y.zero_()
        r[1::2] = 2.0 ** 64 / N ** 0.5 * 1.02
        r[0::2] = 2.0 ** 64 / N ** 0.5 * 0.98
        kw["alpha"] = 1.0
    elif what == "one":                  # a single one in its row
        r[1::2, 77] = 2.0 ** 100
    else:
        r[1::2] *= 2.0 ** 110
    return y, r, kw, wire


@pytest.mark.parametrize("N", [512, 1152, 8192])
@pytest.mark.parametrize("what", ["y", "y_scale", "resid", "one", "border"])
def test_squares_past_fp32(what, N):
    """Held to the same bounds as rows of ordinary size: the powers of two in between
    are exact."""
    for f32, quant in itertools.product((False, True), (0, 32, 128)):
        say(f"resnorm squares past fp32: {what} N={N} f32={f32} quant={quant}")
        y, r, kw, wire = large(what, N, f32)
        got = run(y, r, kw, slice(0, 8), quant)
        torch.cuda.synchronize()
        yv = values(y.view(torch.float8_e4m3fn)) * values(kw["y_scale"])[:, None] if wire else values(y)
        h, eh, z, ez = opsref.resnorm(yv, values(r), values(kw["post_w"]), values(kw["gate"]), values(kw["pre_w"]),
                                      kw["alpha"], kw["beta"], 1e-6)
        assert np.isfinite(values(got[0])).all() and np.isfinite(values(got[1])).all()
        if f32:
            assert np.all(np.abs(values(got[0]) - h) <= eh + opsref.U * np.abs(h))
        else:
            assert bounds.within(bits16(got[0]), h, eh)[0].all()
        assert bounds.within(bits16(got[1]), z, ez)[0].all()
        if quant:
            s = values(got[3]) if quant == 128 else 2.0 ** (got[3].cpu().numpy() - 127.0)
            opsref.check_quant(got[2].cpu().numpy(), s, z, ez, quant)
