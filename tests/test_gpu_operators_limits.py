"""Batches of more rows than one launch of a workgroup a row, or a row tile, may
hold (2^32 lanes a launch): short rows, a few of them compared with the same
rows in a small batch, bit for bit, or with exact integers."""
import pytest
import torch

import block_scaled_fp8_bsgemm_amd as bs
from gpuutil import device, say

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("N,quant", [(8, 0), (32, 32), (128, 128)])
def test_resnorm_rows(N, quant):
    """Rows around every 2^22nd are filled; the rest are zeros and come out so."""
    rows = (1 << 26) + 37
    say(f"resnorm rows={rows} N={N} quant={quant}")
    d = device()
    g = torch.Generator(device=d).manual_seed(N)
    edge = torch.arange(0, rows, 1 << 22, device=d)
    at = torch.unique(torch.cat([edge, (edge - 1).clamp_min(0), torch.arange(rows - 40, rows, device=d)]))
    y = torch.zeros((rows, N), dtype=torch.uint8, device=d)
    y[at] = torch.randint(0, 0x7F, (len(at), N), generator=g, device=d, dtype=torch.uint8)
    s = torch.zeros(rows, device=d)
    s[at] = torch.rand(len(at), generator=g, device=d)
    r = torch.zeros((rows, N), dtype=torch.bfloat16, device=d)
    r[at] = torch.randn((len(at), N), generator=g, device=d).to(torch.bfloat16)
    w = torch.randn(N, generator=g, device=d).to(torch.bfloat16)
    want = bs.resnorm(y[at], r[at], y_scale=s[at], post_w=w, gate=w, quant=quant)
    got = bs.resnorm(y, r, y_scale=s, post_w=w, gate=w, quant=quant)
    torch.cuda.synchronize()
    for k, (a, b) in enumerate(zip(got, want)):
        assert (a is None) == (b is None)
        if a is not None:
            assert same(a.view(rows, -1)[at], b.view(len(at), -1)), k
            a.view(rows, -1)[at] = 0
            assert int(a.count_nonzero()) == 0, k
    if quant:
        return
    # a gate row for each row, in place
    gate = torch.zeros((rows, N), dtype=torch.bfloat16, device=d)
    gate[at] = w
    bs.resnorm(y, r, y_scale=s, post_w=w, gate=gate, resid_out=r, z=got[1])
    torch.cuda.synchronize()
    assert same(r[at], want[0]) and same(got[1][at], want[1])


def thirds(M):
    """ids -1, 0, 1, -1, ... and the plan of two adapters for them, checked."""
    d = device()
    ids = torch.arange(M, dtype=torch.int32, device=d) % 3 - 1
    plan = bs.lora_plan(ids, 2)
    n = [(M - r + 2) // 3 for r in (1, 2, 0)]   # rows of adapter 0, of 1, and without
    assert plan[:4].tolist() == [0, n[0], n[0] + n[1], M]
    at = 4
    for r, k in zip((1, 2, 0), n):
        assert torch.equal(plan[at:at + k], torch.arange(r, M, 3, dtype=torch.int32, device=d))
        at += k
    return ids, plan


def check_rows(t, ids, table):
    """Each row of t is its adapter's row of table (the last one without)."""
    for i in range(0, len(t), 1 << 22):
        assert torch.equal(t[i:i + (1 << 22)], table[ids[i:i + (1 << 22)].long()]), i


def test_shrink_rows():
    M, K, R = (1 << 29) + 70, 8, 8
    say(f"lora_plan, lora_shrink M={M}")
    d = device()
    ids, plan = thirds(M)
    x = torch.ones((M, K), dtype=torch.bfloat16, device=d)
    A = torch.randint(-3, 4, (2, R, K), generator=torch.Generator(device=d).manual_seed(0), device=d)
    H = torch.full((M, R), float("nan"), device=d)
    bs.lora_shrink(x, A.to(torch.bfloat16), plan, H)
    torch.cuda.synchronize()
    check_rows(H, ids, torch.cat([A.float().sum(2), torch.zeros((1, R), device=d)]))


def test_expand_rows():
    M, N, R = (1 << 30) - 1, 8, 8
    say(f"lora_plan, lora_expand M={M}, in place")
    d = device()
    ids, plan = thirds(M)
    H = torch.ones((M, R), device=d)
    B = torch.randint(-3, 4, (2, N, R), generator=torch.Generator(device=d).manual_seed(1), device=d)
    out = torch.ones((M, N), dtype=torch.bfloat16, device=d)
    bs.lora_expand(H, B.to(torch.bfloat16), plan, out, out)
    torch.cuda.synchronize()
    check_rows(out, ids, 1 + torch.cat([B.sum(2), torch.zeros((1, N), device=d, dtype=B.dtype)]).to(torch.bfloat16))


def edges(rows, step):
    """Row numbers on either side of every step-th, and the last ones."""
    edge = torch.arange(0, rows, step, device=device())
    return torch.unique(torch.cat([edge, (edge - 1).clamp_min(0), torch.arange(rows - 40, rows, device=device())]))


@pytest.mark.parametrize("call,rows,N", [("rowq_e4m3", (1 << 26) + 37, 8), ("band_rowq_e4m3", (1 << 24) + 37, 8),
                                         ("blockq_e4m3", (1 << 28) + 37, 128)])
def test_quantizer_rows(call, rows, N):
    """The filled rows' codes and scales against a small batch's, zeros elsewhere."""
    say(f"{call} rows={rows} N={N}")
    d, block = device(), call == "blockq_e4m3"
    fn = {"rowq_e4m3": bs.rowq_e4m3, "band_rowq_e4m3": lambda x, *o: bs.band_rowq_e4m3([x, x.clone()], *o),
          "blockq_e4m3": lambda x, *o: bs.blockq_e4m3(x, 1, *o)}[call]
    at = edges(rows, 1 << 22)
    few = torch.randn((len(at), N), generator=torch.Generator(device=d).manual_seed(N), device=d)
    few = few if block else few.to(torch.bfloat16)
    x = torch.zeros((rows, N), dtype=few.dtype, device=d)
    x[at] = few
    q = torch.full((rows, N), 0x7F, dtype=torch.uint8, device=d)
    s = torch.full((rows, 1), -3.0, device=d)
    fn(x, q, s)
    want = fn(few)
    torch.cuda.synchronize()
    for got, w in zip((q, s), want):
        assert same(got[at], w.view(len(at), -1))
        got[at] = 0
        assert all(int(part.count_nonzero()) == 0 for part in got.split(1 << 24))
