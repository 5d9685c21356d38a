"""The operators of the feed-forward block that follows the projection, in their plain
form and as the library's calls, over the sizes they are used at.

  act    bsgemm_fp8_act  the blockscale fp8 product with bias, activation (gated or not)
                         and residual:  C = alpha resid + beta act(A . B^T + bias)
  route  moe_route       a token's experts and their weights from the router's logits
  moe    moe_fp8         the experts of a few tokens:  out[m] = base[m] +
                         sum_k w[m,k] W2[e] (act(W1[e] x[m]) * (W3[e] x[m])), e = ids[m,k]

The sizes are those of the wo_b projection turned round (hidden size 7168, 2048 between
the two products; the mxfp8 layer's 5120; chunks of up to 16384 rows; a ragged batch's
20096 / 8 rows) and generic ones around them.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token through the gated first product of the block
        dict(name="act token", op="act", M=1, N=2048, K=7168, act="silu", gated=True, bias=False, resid=False, bands=1),
        # one decode step of a batch: the second product, into the residual stream
        dict(name="act decode", op="act", M=64, N=7168, K=2048, act="none", gated=False, bias=False, resid=True,
             bands=1),
        # one band of the ragged batch, a plain two-layer block with biases
        dict(name="act ragged", op="act", M=2512, N=5120, K=2048, act="gelu_tanh", gated=False, bias=True, resid=False,
             bands=1),
        # the prefill chunk's second product with bias and residual, in the layer's 8 bands
        dict(name="act residual chunk", op="act", M=16384, N=7168, K=2048, act="none", gated=False, bias=True,
             resid=True, bands=8),
        # the prefill chunk's gated first product
        dict(name="act gated chunk", op="act", M=16384, N=2048, K=7168, act="silu", gated=True, bias=False,
             resid=False, bands=1),
        # decode: sigmoid scores with a balancing bias, groups of experts
        dict(name="route decode", op="route", M=64, E=256, topk=8, score="sigmoid", bias=True, groups=8, topk_groups=4,
             dtype="f32"),
        # an odd batch, softmax over a small set of experts
        dict(name="route softmax", op="route", M=3001, E=60, topk=4, score="softmax", bias=False, groups=1,
             topk_groups=1, dtype="bf16"),
        # the prefill chunk, as the decode step
        dict(name="route chunk", op="route", M=16384, E=256, topk=8, score="sigmoid", bias=True, groups=8,
             topk_groups=4, dtype="f32"),
        # a small layer: latency counts
        dict(name="moe small", op="moe", M=5, E=16, of=16, topk=2, D=1024, I=384, act="gelu_tanh", base=False),
        # one token, all of its experts here
        dict(name="moe token", op="moe", M=1, E=32, of=32, topk=8, D=7168, I=2048, act="silu", base=True),
        # a few tokens, most experts in use by one or two of them
        dict(name="moe few", op="moe", M=16, E=64, of=64, topk=8, D=7168, I=2048, act="silu", base=True),
        # this GPU's eighth of the experts for the tokens of all GPUs
        dict(name="moe shared out", op="moe", M=128, E=32, of=256, topk=8, D=7168, I=2048, act="silu", base=False),
    ]


ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["act", "act", "route", "moe", "moe"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, 4, 384 // groups)
        keep = rng.randint(max(1, groups // 2), groups)
        return dict(op=op, M=_log(rng, 1, 16384), E=E, topk=rng.randint(1, min(8, keep * (E // groups))),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    topk_groups=keep, dtype=rng.choice(["f32", "bf16"]))
    if op == "moe":
        topk = rng.randint(1, 8)
        E = _log(rng, topk, 64)
        return dict(op=op, M=_log(rng, 1, 128), E=E, of=E * rng.choice([1, 1, 2, 8]), topk=topk,
                    D=_log(rng, 128, 7168, 128), I=_log(rng, 128, 2048, 128), act=rng.choice(ACTS[1:]),
                    base=rng.random() < 0.5)
    gated = rng.random() < 0.5
    N, K = _log(rng, 128, 2048 if gated else 7168, 128), _log(rng, 128, 7168, 128)
    top = 16384 * 2048 * 7168 * 2
    M = min(_log(rng, 1, 16384), top // (N * K * (2 if gated else 1)))
    bands = rng.choice([1, 1, 2, 4, 8])
    M = max(bands, M // bands * bands)
    return dict(op=op, M=M, N=N, K=K, act=rng.choice(ACTS), gated=gated, bias=rng.random() < 0.5,
                resid=rng.random() < 0.5, bands=bands)


# ----------------------------------------------------------------- inputs --

def _codes(x, rows, cols):
    """fp32 x [.., R, C] as e4m3 codes (uint8) with one fp32 scale for each rows x cols block."""
    R, C = x.shape[-2:]
    b = x.view(*x.shape[:-2], R // rows, rows, C // cols, cols)
    s = b.abs().amax((-3, -1)) / 448.0
    q = (b / s.clamp_min(1e-30)[..., :, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(x.shape).view(torch.uint8), s


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)

    op = case["op"]
    st = dict(case)
    M = case["M"]
    if op == "act":
        N, K = case["N"], case["K"]
        rows = N * (2 if case["gated"] else 1)
        st["qa"], st["sa"] = _codes(normal(M, K, dtype=torch.float32), 1, 128)
        st["qb"], st["sb"] = _codes(normal(rows, K, std=1.5 * K ** -0.5, dtype=torch.float32), 128, 128)
        st["bv"] = normal(rows, std=0.5) if case["bias"] else None
        st["rv"] = normal(M * N, std=2.0) if case["resid"] else None
        st["alpha"], st["beta"] = (0.75, 0.5) if case["resid"] else (1.0, 1.0)
        st["out"] = torch.empty(M * N, dtype=torch.bfloat16, device=DEV)
        return st
    if op == "route":
        E = case["E"]
        st["logits"] = normal(M, E, std=1.5, dtype=torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
        st["bv"] = normal(E, std=0.1, dtype=torch.float32) if case["bias"] else None
        st["scale"] = 2.5 if case["score"] == "sigmoid" else 1.0
        st["ids"] = torch.empty(M, case["topk"], dtype=torch.int32, device=DEV)
        st["w"] = torch.empty(M, case["topk"], dtype=torch.float32, device=DEV)
        return st
    E, D, I, topk = case["E"], case["D"], case["I"], case["topk"]
    st["x"] = normal(M, D)
    # the experts of all GPUs; those past the first E are other GPUs'
    st["ids"] = torch.rand(M, case["of"], generator=gen, device=DEV).argsort(1)[:, :topk].to(torch.int32).contiguous()
    w = torch.rand(M, topk, generator=gen, device=DEV) + 0.1
    st["w"] = (w / w.sum(1, keepdim=True)).contiguous()
    st["w13"] = torch.empty(E, 2 * I, D, dtype=torch.uint8, device=DEV)
    st["s13"] = torch.empty(E, 2 * I // 128, D // 128, dtype=torch.float32, device=DEV)
    st["w2"] = torch.empty(E, D, I, dtype=torch.uint8, device=DEV)
    st["s2"] = torch.empty(E, D // 128, I // 128, dtype=torch.float32, device=DEV)
    for e in range(E):
        st["w13"][e], st["s13"][e] = _codes(normal(2 * I, D, std=1.5 * D ** -0.5, dtype=torch.float32), 128, 128)
        st["w2"][e], st["s2"][e] = _codes(normal(D, I, std=I ** -0.5, dtype=torch.float32), 128, 128)
    st["bv"] = normal(M, D) if case["base"] else None
    st["out"] = torch.empty(M, D, dtype=torch.bfloat16, device=DEV)
    return st


# ------------------------------------------------------------- plain forms --

def _values(q):
    return q.view(torch.float8_e4m3fn).to(torch.float32)


def _weights(q, s):
    """The values of e4m3 codes [.., R, C] with a scale for each 128 x 128 block."""
    R, C = q.shape[-2:]
    v = _values(q).view(*q.shape[:-2], R // 128, 128, C // 128, 128)
    return (v * s[..., :, None, :, None]).view(q.shape)


def _plain_act(t, act):
    if act == "relu":
        return t.clamp_min(0.0)
    if act == "silu":
        return t / (1.0 + torch.exp(-t))
    if act == "gelu":
        return 0.5 * t * (1.0 + torch.erf(t * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return t / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (t + 0.044715 * t * t * t)))
    return t


def _plain_route(s):
    M, E, topk, groups = s["M"], s["E"], s["topk"], s["groups"]
    x = s["logits"].double()    # 64 bits: a chosen expert's key may be next to one that is not chosen
    ok = x > -math.inf
    if s["score"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    key = x if s["bv"] is None and groups == 1 else score
    if s["bv"] is not None:
        key = score + s["bv"].double()
        ok = ok & (s["bv"] > -math.inf)
    key = torch.where(ok, key, -math.inf)
    if groups > 1:
        per = key.view(M, groups, E // groups)
        best = per.sort(dim=2, descending=True).values[:, :, :2]
        best = torch.where(best > -math.inf, best, 0.0).sum(2)
        best = torch.where(ok.view(M, groups, -1).any(2), best, -math.inf)
        order = best.sort(dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        keep = torch.zeros(M, groups, dtype=torch.bool, device=x.device).scatter_(1, order, True)
        key = torch.where(keep[:, :, None], per, -math.inf).view(M, E)
    key, ids = key.sort(dim=1, descending=True, stable=True)
    has, ids = key[:, :topk] > -math.inf, ids[:, :topk]
    w = torch.where(has, score.gather(1, ids), 0.0)
    total = w.sum(1, keepdim=True)
    w = torch.where(total > 0, w / total, 0.0) * s["scale"]
    return {"ids": torch.where(has, ids, -1).to(torch.int32), "weights": w.float()}


def _plain_moe(s):
    M, E, D, I, topk = s["M"], s["E"], s["D"], s["I"], s["topk"]
    x = s["x"].float()
    here = (s["ids"] >= 0) & (s["ids"] < E)
    w = torch.where(here, s["w"], 0.0)
    at = torch.where(here, s["ids"], 0).to(torch.int64)
    if M * topk < E:   # each token's experts taken out of the stack
        at = at.view(-1)
        t = torch.bmm(_weights(s["w13"][at], s["s13"][at]), x.repeat_interleave(topk, 0)[:, :, None])[:, :, 0]
        h = _plain_act(t[:, :I], s["act"]) * t[:, I:]
        y = torch.bmm(_weights(s["w2"][at], s["s2"][at]), h[:, :, None])[:, :, 0]
        y = (y.view(M, topk, D) * w[:, :, None]).sum(1)
    else:              # every expert for every token
        share = torch.zeros(M, E, device=x.device).scatter_add_(1, at, w)
        t = (_weights(s["w13"], s["s13"]).view(-1, D) @ x.t()).view(E, 2 * I, M)
        h = _plain_act(t[:, :I], s["act"]) * t[:, I:] * share.t()[:, None, :]
        y = torch.bmm(_weights(s["w2"], s["s2"]), h).sum(0).t()
    if s["bv"] is not None:
        y = y + s["bv"].float()
    return y.to(torch.bfloat16).contiguous()


def run(state):
    s = state
    if own:
        return _own_run(s)
    if s["op"] == "route":
        return _plain_route(s)
    if s["op"] == "moe":
        return _plain_moe(s)
    M, N, K = s["M"], s["N"], s["K"]
    a = (_values(s["qa"]).view(M, K // 128, 128) * s["sa"][:, :, None]).view(M, K)
    t = a @ _weights(s["qb"], s["sb"]).t()
    if s["bv"] is not None:
        t = t + s["bv"].float()
    v = _plain_act(t[:, :N], s["act"])
    if s["gated"]:
        v = v * t[:, N:]
    if s["rv"] is not None:
        v = s["alpha"] * s["rv"].float().view(M, N) + s["beta"] * v
    return v.to(torch.bfloat16).reshape(-1)


def _own_run(s):
    import block_scaled_fp8_bsgemm_amd as bs
    if s["op"] == "act":
        return bs.bsgemm_fp8_act(s["qa"], s["sa"], s["qb"], s["sb"], bias=s["bv"], act=s["act"], gated=s["gated"],
                                 resid=s["rv"], alpha=s["alpha"], beta=s["beta"], C=s["out"], bands=s["bands"])
    if s["op"] == "route":
        ids, w = bs.moe_route(s["logits"], s["topk"], score=s["score"], bias=s["bv"], groups=s["groups"],
                              topk_groups=s["topk_groups"], renorm=True, scale=s["scale"], ids=s["ids"], weights=s["w"])
        return {"ids": ids, "weights": w}
    return bs.moe_fp8(s["x"], s["ids"], s["w"], s["w13"], s["s13"], s["w2"], s["s2"], base=s["bv"], act=s["act"],
                      out=s["out"])


# ----------------------------------------------------------- work and exact --

def work(case):
    op, M = case["op"], case["M"]
    if op == "act":
        N, K = case["N"], case["K"]
        rows = N * (2 if case["gated"] else 1)
        n = M * K + rows * K + M * K // 32 + rows * K // 4096 + 2 * M * N * (2 if case["resid"] else 1)
        return dict(bytes=n + 2 * rows * case["bias"], flops=2 * M * rows * K)
    if op == "route":
        E = case["E"]
        return dict(bytes=M * E * (4 if case["dtype"] == "f32" else 2) + 8 * M * case["topk"] + 4 * E * case["bias"],
                    flops=M * E * 8)
    E, D, I, topk = case["E"], case["D"], case["I"], case["topk"]
    used = max(1.0, E * (1.0 - (1.0 - topk / case["of"]) ** M))   # experts that some token uses
    pairs = M * topk * E / case["of"]
    return dict(bytes=int(used * 3 * D * I * (1 + 4 / 16384) + M * D * (4 + 2 * case["base"]) + 8 * M * topk),
                flops=int(pairs * 6 * D * I))


def _exact_act(t, act):
    if act == "relu":
        return torch.where(t > 0, t, 0.0)
    if act == "silu":
        return t * torch.sigmoid(t)
    if act == "gelu":
        return t * torch.special.erfc(-t / 2.0 ** 0.5) / 2.0
    if act == "gelu_tanh":
        return t / 2.0 * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (t + 0.044715 * t.pow(3))))
    return t


def _exact_route(case, s):
    M, E, G = case["M"], case["E"], case["groups"]
    x = s["logits"].double().cpu()
    score = torch.softmax(x, 1) if case["score"] == "softmax" else torch.sigmoid(x)
    key = (x if G == 1 and s["bv"] is None else score).clone()
    if s["bv"] is not None:
        key += s["bv"].double().cpu()
    if G > 1:
        per = key.view(M, G, -1).clone()
        first = per.amax(2)
        per.scatter_(2, per.argmax(2, keepdim=True), -math.inf)
        second = per.amax(2)
        rank = first + torch.where(torch.isinf(second), 0.0, second)
        out = torch.ones(M, G, dtype=torch.bool)
        for _ in range(case["topk_groups"]):
            best = rank.argmax(1, keepdim=True)
            out.scatter_(1, best, False)
            rank.scatter_(1, best, -math.inf)
        key[out.repeat_interleave(E // G, 1)] = -math.inf
    ids, w = [], []
    for _ in range(case["topk"]):
        at = key.argmax(1, keepdim=True)
        ids.append(at)
        w.append(score.gather(1, at))
        key.scatter_(1, at, -math.inf)
    w = torch.cat(w, 1)
    return {"ids": torch.cat(ids, 1).to(torch.int32), "weights": w / w.sum(1, keepdim=True) * s["scale"]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)

    def product(q, sb, rows, at):
        """x . W^T in 64 bits, a 128-deep block at a time; at(kb) gives x's block."""
        t = 0.0
        for kb in range(sb.shape[1]):
            w = q[:, 128 * kb:128 * kb + 128].view(torch.float8_e4m3fn).double()
            t = t + at(kb) @ (w * sb[:, kb].double().repeat_interleave(128)[:, None]).t()
        return t

    if case["op"] == "moe":
        E, I = case["E"], case["I"]
        out = torch.zeros(case["M"], case["D"], dtype=torch.float64, device=DEV)
        for e in range(E):
            hit = s["ids"] == e
            rows = hit.any(1).nonzero()[:, 0]
            if not len(rows):
                continue
            x = s["x"][rows].double()
            t = product(s["w13"][e], s["s13"][e], len(rows), lambda kb: x[:, 128 * kb:128 * kb + 128])
            h = _exact_act(t[:, :I], case["act"]) * t[:, I:]
            y = product(s["w2"][e], s["s2"][e], len(rows), lambda kb: h[:, 128 * kb:128 * kb + 128])
            out[rows] += y * (s["w"].double() * hit).sum(1)[rows][:, None]
        return out if s["bv"] is None else out + s["bv"].double()
    M, N = case["M"], case["N"]
    t = product(s["qb"], s["sb"], M, lambda kb: s["qa"][:, 128 * kb:128 * kb + 128].view(torch.float8_e4m3fn).double()
                * s["sa"][:, kb, None].double())
    if s["bv"] is not None:
        t = t + s["bv"].double()
    v = _exact_act(t[:, :N], case["act"])
    if case["gated"]:
        v = v * t[:, N:]
    if s["rv"] is not None:
        v = s["alpha"] * s["rv"].double().view(M, N) + s["beta"] * v
    return v.reshape(-1)
