"""64-bit definitions of MXFP4 quantisation and products and of the route from logits (numpy,
written from the formats' tables; no code of the library)."""
import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def e8m0(u):
    u = np.asarray(u)
    return np.where(u == 255, np.nan, np.exp2(u.astype(np.float64) - 127))


def unpack(codes, scales):
    """float64 values of rows of codes [..., n / 2] with E8M0 bytes [..., n / 32]."""
    b = codes.reshape(*codes.shape[:-1], -1, 16)
    v = E2M1[np.concatenate([b & 15, b >> 4], -1)] * e8m0(scales)[..., None]
    return v.reshape(*codes.shape[:-1], -1)


def quantise(x):
    """(codes, scales) of x [rows][n] (any float type), value by value on E2M1's grid."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0, b)
    top = np.abs(b).max(-1)
    _, e = np.frexp(top)  # top = f 2^e, f in [1/2, 1)
    u = np.where(top > 0, np.clip(e - 1 - 2 + 127, 0, 254), 0)
    v = np.abs(b) * np.exp2(127.0 - u)[..., None]
    grid = E2M1[:8]
    mid = (grid[1:] + grid[:-1]) / 2
    code = np.searchsorted(mid, v, side="left")  # a tie at mid[i] gives i ..
    tie = np.isin(v, mid) & (code % 2 == 1)      # .. and goes up when i is odd (even codes: even mantissas)
    code = np.minimum(code + tie, 7)
    code = code | (np.signbit(b) << 3)
    code = np.where(bad[..., None], 0, code)
    u = np.where(bad, 255, u)
    packed = code[..., :16] | (code[..., 16:] << 4)
    return packed.astype(np.uint8).reshape(x.shape[0], -1), u.astype(np.uint8)


def route(z, k, G=1, Gk=1, score="sigmoid", group_top=2, renorm=True, scale=1.0, bias=None):
    """(idx, w) of logits z [T][E], one token at a time."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    m = E // G
    idx, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        there = z[t] > -np.inf
        with np.errstate(all="ignore"):
            if score == "sigmoid":
                p = 1 / (1 + np.exp(-z[t]))
            else:
                zz = np.where(there, z[t], -np.inf)
                top = zz.max()
                p = np.where(there, (zz == np.inf) if top == np.inf else np.exp(zz - top), 0.0)
                p = p / p.sum() if p.sum() > 0 else p
        c = p if bias is None else p + np.asarray(bias, np.float64)
        there = there & (c > -np.inf)
        key = z[t] if bias is None else c
        by = key if group_top == 1 or m == 1 else c
        groups = []
        for g in range(G):
            best = sorted((by[e] for e in range(g * m, g * m + m) if there[e]), reverse=True)[:group_top]
            groups.append((-(sum(best)) if best else np.inf, g))
        kept = {g for _, g in sorted(groups)[:Gk]}
        order = sorted((-key[e], e) for e in range(E) if there[e] and e // m in kept)[:k]
        taken = [e for _, e in order]
        total = sum(p[e] for e in taken)
        for j, e in enumerate(taken):
            idx[t, j] = e
            w[t, j] = ((p[e] / total if total > 0 else 0.0) if renorm else p[e]) * scale
    return idx, w


def group(idx, E):
    """perm (pairs by expert, then pair), off, active (padded with zeros), n_active of a route."""
    flat = idx.reshape(-1)
    pairs = np.nonzero(flat >= 0)[0]
    order = pairs[np.argsort(flat[pairs], kind="stable")]
    cnt = np.bincount(flat[pairs], minlength=E)
    off = np.concatenate([[0], np.cumsum(cnt)])
    act = np.nonzero(cnt)[0]
    perm = np.full(flat.size, -7)
    perm[:order.size] = order
    return (perm.astype(np.int32), off.astype(np.int32), np.pad(act, (0, E - act.size)).astype(np.int32),
            np.array([act.size], np.int32))


def dot_bound(K, abs_sum):
    """Error of K exact products added in fp32 in any order: each addition is off by at most one
    step (truncation allowed) of a partial sum that abs_sum = sum |a w| bounds."""
    return K * 2.0 ** -23 * abs_sum


def round_bound(v, dtype):
    """One rounding of v to a torch dtype: half a step, or half the smallest subnormal."""
    import torch
    f = torch.finfo(dtype)
    return np.abs(v) * (f.eps / 2) + f.tiny * f.eps / 2
