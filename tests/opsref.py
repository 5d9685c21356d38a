"""Plain float64 implementations of the adapter operators and of resnorm, and
the error bounds their results are held to.  Nothing here uses the library.

u = 2^-24 is fp32's half step, and an fp32 addition inside an MFMA is counted
as 2u, whether it rounds or truncates.
"""
import numpy as np

U = 2.0 ** -24


def plan(ids, L):
    key = np.where((ids >= 0) & (ids < L), ids, L)
    order = np.argsort(key, kind="stable")
    start = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=L + 1))])
    return np.concatenate([start, order]).astype(np.int32)


def shrink(x, A, ids):
    """(H, bound) for float64 x [M,K], A [L,R,K].  At most K products are added
    one by one, and W <= 16 partial sums after them: |err| <= 2u (K + 16) |x| |A|^T."""
    M, K = x.shape
    L, R, _ = A.shape
    H, S = np.zeros((M, R)), np.zeros((M, R))
    for m in range(M):
        if 0 <= ids[m] < L:
            H[m] = A[ids[m]] @ x[m]
            S[m] = np.abs(A[ids[m]]) @ np.abs(x[m])
    return H, 2 * U * (K + 16) * S


def delta(H, B, scale, ids):
    """(D, bound) with D[m] = scale[a] (H[m] B[a]^T).  scale * H is rounded to fp32
    and carried to 2^-17 by its two bf16, and 2R products are added:
    |err| <= (2^-17 + u + 2u * 2R) scale |H| |B|^T."""
    M, R = H.shape
    L, N, _ = B.shape
    D, S = np.zeros((M, N)), np.zeros((M, N))
    for a in range(L):
        rows = ids == a
        if rows.any():
            s = 1.0 if scale is None else float(scale[a])
            D[rows] = s * (H[rows] @ B[a].T)
            S[rows] = abs(s) * (np.abs(H[rows]) @ np.abs(B[a]).T)
    return D, (2.0 ** -17 + U + 4 * U * R) * S


def resnorm(y, resid, post_w, gate, pre_w, alpha, beta, eps):
    """(h, eh, z, ez): float64 results and bounds of what fp32 makes of them before
    the final rounding.  A mean of squares sums N positive terms, in a lane's
    order and then by a tree over lanes and waves: at most 8 * 4 + 6 + 16 additions
    and a few more roundings, so it is off by 64u at most, its root by half of
    that, and a normed value, with its products, by 48u.  h adds one rounding of each term and
    of the sum.  An error of h (eh) reaches z directly, and through rms(h) by at
    most the mean of |h| eh over rms(h)^2."""
    N = y.shape[1]
    p = y
    if post_w is not None:
        p = y / np.sqrt(np.mean(y * y, 1, keepdims=True) + eps) * post_w
    if gate is not None:
        p = p * gate
    h = alpha * resid + beta * p
    eh = 56 * U * (np.abs(alpha * resid) + np.abs(beta * p))
    ms = np.mean(h * h, 1, keepdims=True) + eps
    w = np.ones(N) if pre_w is None else pre_w
    z = h / np.sqrt(ms) * w
    off = np.mean(np.abs(h) * eh, 1, keepdims=True) / ms
    ez = (eh / np.sqrt(ms)) * np.abs(w) + np.abs(z) * (off + 48 * U)
    return h, eh, z, 1.001 * ez


def e4m3_values():
    import torch
    return torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def check_quant(q, s, z, ez, block):
    """e4m3 codes q and scales s (values) of z +- ez in blocks of `block` columns:
    the scale is the definition's for some amax in reach, and every code is within half a step
    of z / s, widened by what z is off."""
    rows, N = z.shape
    zb, eb = z.reshape(rows, -1, block), ez.reshape(rows, -1, block)
    hi = (np.abs(zb) + eb).max(2)
    lo = (np.abs(zb) - eb).max(2).clip(0)
    if block == 128:
        assert np.all(s <= hi / 448 * (1 + 2 * U)) and np.all(s >= lo / 448 * (1 - 2 * U)), "scales"
    else:
        def k_of(a):
            with np.errstate(divide="ignore"):
                m, e = np.frexp(a)
            return np.where(a == 0, -127, np.maximum(e - 9 + (m > 0.875), -127))
        k = np.log2(s)
        assert np.all((k >= k_of(lo)) & (k <= k_of(hi))), "scales"
    v = e4m3_values()[q].reshape(zb.shape)
    with np.errstate(divide="ignore", invalid="ignore"):
        want = np.where(s[..., None] == 0, 0.0, zb / s[..., None])
        slack = np.where(s[..., None] == 0, 0.0, eb / s[..., None]) + 2 * U * np.abs(want)
    want = np.clip(want, -448, 448)
    # half a step: 2^-4 of the power of two below |want| (2^-10 in the subnormal range)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(want) + slack, 2.0 ** -20))), -6) - 4)
    assert np.all(np.abs(v - want) <= step + slack), ("codes", float(np.max(np.abs(v - want) - step - slack)))
