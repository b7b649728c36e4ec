"""64-bit definitions of int8 rows and products with token and channel scales, of a route's pairs
sorted by expert, and of the route's gradient (numpy, no code of the library)."""
import numpy as np


def quantise(x):
    """(codes, scales) of x [rows][n] of any float type, value by value: both divisions in fp32."""
    x = np.asarray(x).astype(np.float32)
    bad = ~np.isfinite(x).all(1)
    x = np.where(bad[:, None], np.float32(0), x)
    scale = np.abs(x).max(1) / np.float32(127)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        v = (x / scale[:, None]).astype(np.float64)
    v = np.where(scale[:, None] > 0, v, 0)
    codes = np.clip(np.trunc(v + np.copysign(0.5, v)), -127, 127)
    return codes.astype(np.int8), np.where(bad, np.float32(np.nan), scale).astype(np.float32)


def dot(a, b):
    """a [M][K] b [N][K]^T of int8 codes, exactly (sums below 2^53)."""
    return a.astype(np.float64) @ b.astype(np.float64).T


def product32(acc, row, channel):
    """(float)acc * (row * channel), in fp32."""
    return acc.astype(np.float32) * (row[:, None] * channel[None, :])


def sort_pairs(idx, E):
    """off, perm (the pairs that are there), pos, active of a route idx [T][k]."""
    flat = np.asarray(idx).reshape(-1)
    ok = (flat >= 0) & (flat < E)
    there = np.nonzero(ok)[0]
    perm = there[np.argsort(flat[there], kind="stable")]
    pos = np.full(flat.size, -1, np.int64)
    pos[perm] = np.arange(perm.size)
    cnt = np.bincount(flat[there], minlength=E)
    off = np.concatenate([[0], np.cumsum(cnt)])
    return off, perm, pos, np.nonzero(cnt)[0]


def scores(z, kind):
    z = np.asarray(z, np.float64)
    here = z > -np.inf  # false for NaN
    if kind == "sigmoid":
        e = np.exp(-np.abs(np.where(here, z, 0)))
        return np.where(here, np.where(z >= 0, 1, e) / (1 + e), 0)
    top = np.where(here, z, -np.inf).max(-1, keepdims=True)
    top = np.where(np.isfinite(top), top, 0)
    e = np.where(here, np.exp(np.where(here, z, -np.inf) - top), 0)
    s = e.sum(-1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def weights(z, idx, kind, renorm, scale):
    """The weights of the taken experts idx [T][k], in 64 bits."""
    p = np.where(idx >= 0, np.take_along_axis(scores(z, kind), np.maximum(idx, 0), -1), 0)
    if renorm:
        s = p.sum(-1, keepdims=True)
        p = np.divide(p, s, out=np.zeros_like(p), where=s > 0)
    return p * scale


def route_grad(z, idx, g, kind, renorm, scale):
    """sum_j g_j d w_j / d z, by the derivative of every weight (finite logits and -inf)."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    k = idx.shape[1]
    p = scores(z, kind)
    out = np.zeros((T, E))
    for t in range(T):
        jac = np.zeros((k, E))  # d p_j / d z_e
        for j in range(k):
            e = idx[t, j]
            if e < 0:
                continue
            if kind == "sigmoid":
                jac[j, e] = p[t, e] * (1 - p[t, e])
            else:
                jac[j] = -p[t, e] * p[t]
                jac[j, e] += p[t, e]
        if renorm:
            pj = np.where(idx[t] >= 0, p[t][np.maximum(idx[t], 0)], 0)
            s = pj.sum()
            jac = jac / s - np.outer(pj, jac.sum(0)) / s ** 2 if s > 0 else 0 * jac
        out[t] = scale * np.where(idx[t] >= 0, g[t], 0) @ jac
    return out
