"""Plain float64 implementations of the feed-forward operators (bsgemm_fp8_act,
moe_route, moe_fp8) and the error bounds their results are held to.  Nothing here
uses the library.

u = 2^-24 is fp32's half step, and an fp32 addition inside an MFMA is counted as
2u, whether it rounds or truncates.
"""
import math

import numpy as np

U = 2.0 ** -24
ACT_REL = 2.0 ** -15    # what an activation may be off, relative to its value
# What may come out as zero: the reciprocal of 1 + e^a, a = -t, has no subnormals, so it is zero where
# 1 + e^a > 2^126, from a = 126 ln 2 = 87.33 on.  silu's result there is a / (1 + e^a), which falls with
# a, so at most 87.34 * 2^-126 < 2^(6.45 - 126) = 2^-119.55; gelu_tanh has |x| < 10 there, gelu's
# exponential 2^-126 and |x| < 14.
ACT_ABS = 2.0 ** -119
SLOPE = 1.13            # the steepest any of the activations is (gelu's largest slope, 1.129)
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")

_erfc = np.vectorize(math.erfc)


def act(t, name):
    t = np.asarray(t, np.float64)
    with np.errstate(over="ignore"):
        if name == "relu":
            return np.maximum(t, 0.0)
        if name == "silu":
            return t / (1.0 + np.exp(-t))
        if name == "gelu":
            return 0.5 * t * _erfc(-t / math.sqrt(2.0)) if t.size else t
        if name == "gelu_tanh":
            return t / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (t + 0.044715 * t ** 3)))
    return t


def act_err(t, et, name):
    """What act(t) is off in fp32, for t off by et."""
    v = np.abs(act(t, name))
    own = 0.0 if name in ("none", "relu") else ACT_REL * (v + SLOPE * et) + ACT_ABS
    return SLOPE * et + own


def epilogue(acc, eacc, bias, name, gated, resid, alpha, beta):
    """(C before its rounding to bf16, bound) for accumulators [M, rows of B] off by eacc."""
    t, et = acc, eacc
    if bias is not None:
        t = acc + bias
        et = et + U * (np.abs(t) + et)
    if gated:
        N = t.shape[1] // 2
        g, up, eg, eu = t[:, :N], t[:, N:], et[:, :N], et[:, N:]
        a = act(g, name)
        ea = act_err(g, eg, name)
        v = a * up
        ev = ea * (np.abs(up) + eu) + np.abs(a) * eu
        ev = ev + 2 * U * (np.abs(v) + ev)
    else:
        v, ev = act(t, name), act_err(t, et, name)
    c, ec = beta * v, np.abs(beta) * ev
    ec = ec + 2 * U * (np.abs(c) + ec)
    if resid is not None:
        c = c + alpha * resid
        ec = ec + 2 * U * np.abs(alpha * resid)
        ec = ec + U * (np.abs(c) + ec)
    return c, ec


def dequant(q, s):
    """float64 values of e4m3 codes [.., R, C] with a scale for each 128 x 128 block."""
    import opsref
    return opsref.e4m3_values()[q] * np.repeat(np.repeat(s.astype(float), 128, -2), 128, -1)


def moe(x, ids, weights, W13, W2, base, name):
    """(out before its rounding to bf16, bound), all arguments float64 but ids; W13 [E,2I,D],
    W2 [E,D,I].  A first product of D terms, the folds of its 64 deep pieces and the waves'
    sums: |err| <= 2u (D + D/32 + 24) |W| |x|; h, its split to 2^-17; the second product, of
    two parts for each of I terms, likewise; the weights' sum and the experts' by fp32 additions."""
    M, D = x.shape
    E, _, I = W2.shape
    out = np.zeros((M, D)) if base is None else base.copy()
    err, mag = np.zeros((M, D)), np.abs(out)
    for m in range(M):
        for e in sorted({int(i) for i in ids[m] if 0 <= i < E}):
            w = float(sum(weights[m][ids[m] == e]))
            t = W13[e] @ x[m]
            et = 2 * U * (D + D / 32 + 24) * (np.abs(W13[e]) @ np.abs(x[m]))
            a, ea = act(t[:I], name), act_err(t[:I], et[:I], name)
            h = a * t[I:]
            eh = ea * (np.abs(t[I:]) + et[I:]) + np.abs(a) * et[I:]
            eh = eh + (2.0 ** -17 + 2 * U) * (np.abs(h) + eh)
            y, ay = W2[e] @ h, np.abs(W2[e]) @ (np.abs(h) + eh)
            ey = np.abs(W2[e]) @ eh + 2 * U * (2 * I + I / 32 + 24) * ay
            out[m] += w * y
            err[m] += abs(w) * ey + 2 * U * ids.shape[1] * abs(w) * (np.abs(y) + ey)
            mag[m] += abs(w) * ay
    return out, err + 2 * U * (ids.shape[1] + 12) * mag


def route(logits, topk, score="softmax", bias=None, groups=1, topk_groups=1, group_top=2, renorm=True, scale=1.0):
    """(ids, weights) by the definition, row by row, from float64 logits [M, E]."""
    M, E = logits.shape
    ids, out = np.full((M, topk), -1, np.int32), np.zeros((M, topk))
    per = E // groups
    for m in range(M):
        x = logits[m]
        with np.errstate(all="ignore"):
            if score == "softmax":
                # the largest of what is not NaN; a NaN among the logits is one in the sum
                top = -math.inf if np.all(np.isnan(x)) else np.nanmax(x)
                p = np.exp(x - top)
                s = p / p.sum()
            else:
                s = 1.0 / (1.0 + np.exp(-x))
            key = x.copy() if bias is None and groups == 1 else s.copy()
            ok = x > -math.inf
            if bias is not None:
                key = key + bias
                ok &= bias > -math.inf
        ok &= ~np.isnan(key)
        chosen = [e for e in range(E) if ok[e]]
        if groups > 1:
            best = {}
            for g in range(groups):
                k = sorted((key[e] for e in chosen if e // per == g), reverse=True)[:group_top]
                if k:
                    best[g] = sum(k)
            kept = sorted(best, key=lambda g: (-best[g], g))[:topk_groups]
            chosen = [e for e in chosen if e // per in kept]
        chosen = sorted(chosen, key=lambda e: (-key[e], e))[:topk]
        w = s[chosen]
        if renorm:
            w = np.zeros(len(chosen)) if w.sum() == 0 else w / w.sum()
        ids[m, :len(chosen)] = chosen
        out[m, :len(chosen)] = w * scale
    return ids, out
