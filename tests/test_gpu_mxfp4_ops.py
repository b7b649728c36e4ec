"""The MXFP4 x MXFP4 operators (quantise, dequantise, dense product, the experts' gate/up and
down products over a route) against their 64-bit definitions. Quantisation is compared bit for
bit; products within the bound of fp32 sums of exact products and one rounding of the output,
and bit for bit where every sum is exact."""
import numpy as np
import pytest

import mxref

pytestmark = pytest.mark.gpu

DT = ["float32", "bfloat16", "float16"]


@pytest.fixture(scope="module")
def q():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_moe_sigmoid_amd as q
    q.lib()
    return q


def _t(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(getattr(torch, dtype))


def _n(t):
    return t.detach().cpu().double().numpy()


def _dt(name):
    import torch
    return getattr(torch, name)


def _quantise(q, x):
    import torch
    rows, cols = x.shape
    codes = torch.full((rows, cols // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, cols // 32), 0xA5, dtype=torch.uint8, device="cuda")
    q.mxfp4_quantize(x, codes, scales)
    torch.cuda.synchronize()
    return codes, scales


def _weights(rng, *shape):
    """Random codes and scale bytes of a few binades: [..., n] values."""
    n = shape[-1]
    return (rng.integers(0, 256, (*shape[:-1], n // 2), dtype=np.uint8),
            rng.integers(119, 124, (*shape[:-1], n // 32), dtype=np.uint8))


# ------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (16, 2080), (257, 64)])
def test_quantise_random(q, dtype, rows, cols):
    rng = np.random.default_rng(rows * cols)
    x = rng.standard_normal((rows, cols)) * np.exp2(3 * rng.standard_normal((rows, cols // 32))).repeat(32, 1)
    x = _t(x.astype(np.float32), dtype)
    codes, scales = _quantise(q, x)
    rc, rs = mxref.quantise(_n(x))
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)


@pytest.mark.parametrize("dtype", DT)
def test_quantise_every_boundary(q, dtype):
    """Each grid value and halfway point, its neighbours one step off, in blocks whose largest
    value is 4, 6, just below 8 (saturates), at ordinary, smallest and largest binades."""
    import torch
    f = torch.finfo(_dt(dtype))
    vals = []
    for v in (0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7):
        for s in (1, -1):
            vals += [s * v, s * v * (1 + f.eps), s * v * (1 - f.eps)]
    rows = []
    for top in (4.0, 6.0, 8 * (1 - f.eps)):
        body = [v for v in vals if abs(v) <= top]
        body += [0.0] * (-len(body) % 31)
        for i in range(0, len(body), 31):
            rows.append([top] + body[i:i + 31])
    x = np.array(rows)
    e = {"float32": (0, -100, 124, -127, -140), "bfloat16": (0, -100, 124, -127, -130), "float16": (0, -10, 12, -16, -20)}
    x = np.concatenate([x * 2.0 ** s for s in e[dtype]])
    x = torch.from_numpy(x).to(_dt(dtype)).cuda()
    codes, scales = _quantise(q, x)
    rc, rs = mxref.quantise(_n(x))
    assert np.array_equal(scales.cpu().numpy(), rs)
    got, want = mxref.unpack(codes.cpu().numpy(), scales.cpu().numpy()), mxref.unpack(rc, rs)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("dtype", DT)
def test_quantise_special_blocks(q, dtype):
    """Zeros (scale byte 0), an infinity or NaN (byte 255, codes 0), neighbours untouched."""
    x = np.zeros((5, 96), np.float32)
    x[1, 40] = np.inf
    x[2, 95] = np.nan
    x[3, 0] = -np.inf
    x[4] = 1.0
    x[1, :32] = -3.0
    codes, scales = _quantise(q, _t(x, dtype))
    rc, rs = mxref.quantise(x)
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)


@pytest.mark.parametrize("dtype", DT)
def test_dequantise_every_code_and_scale(q, dtype):
    import torch
    codes = np.arange(256, dtype=np.uint8).reshape(1, 16, 16).repeat(256, 0)  # each byte value, each scale
    scales = np.arange(256, dtype=np.uint8)[:, None].repeat(16, 1)
    codes = codes.reshape(256, 256)
    out = torch.full((256, 512), 7.0, dtype=_dt(dtype), device="cuda")
    q.mxfp4_dequantize(_t(codes), _t(scales), out)
    want = torch.from_numpy(mxref.unpack(codes, scales)).float().to(_dt(dtype))  # exact in fp32, rounded once
    got = out.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got.float()), torch.nan_to_num(want.float()))


# ------------------------------------------------------------------ dense product
LINEAR = [(1, 16, 128), (1, 1, 32), (2, 17, 96), (5, 100, 160), (16, 64, 512), (17, 33, 544), (31, 128, 1056),
          (33, 257, 2080), (64, 96, 288), (77, 301, 2080), (100, 515, 256), (129, 256, 768), (200, 130, 1312),
          (257, 384, 1024), (300, 515, 640), (513, 771, 320)]


def _check_linear(q, M, N, K, dtype, seed, ws=None):
    import torch
    rng = np.random.default_rng(seed)
    x = _t(rng.standard_normal((M, K)).astype(np.float32), dtype)
    wc, wsc = _weights(rng, N, K)
    out = torch.full((M, N), float("nan"), dtype=_dt(dtype), device="cuda")
    ws = q.alloc_mxfp4_linear_workspace(M, N, K) if ws is None else ws
    ws.fill_(0xFF)  # whatever an earlier call left
    q.mxfp4_linear(x, _t(wc), _t(wsc), out, ws)
    a, w = mxref.unpack(*mxref.quantise(_n(x))), mxref.unpack(wc, wsc)
    y = a @ w.T
    tol = mxref.dot_bound(K, np.abs(a) @ np.abs(w).T)
    tol = tol + mxref.round_bound(np.abs(y) + tol, _dt(dtype))
    err = np.abs(_n(out) - y)
    assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("M,N,K", LINEAR)
@pytest.mark.parametrize("dtype", DT)
def test_linear(q, M, N, K, dtype):
    print(f"linear M={M} N={N} K={K} {dtype}", flush=True)
    _check_linear(q, M, N, K, dtype, M + N + K)


def test_linear_workspace_covers_smaller_batches(q):
    ws = q.alloc_mxfp4_linear_workspace(300, 130, 416)
    for M in (300, 1, 2, 16, 40, 129):
        _check_linear(q, M, 130, 416, "bfloat16", M, ws)


@pytest.mark.parametrize("M,N,K", [(1, 48, 2048), (16, 200, 608), (40, 300, 2080), (300, 600, 1024)])
def test_linear_exact_sums_bitidentical(q, M, N, K):
    """Values on E2M1's grid with scale 1 on both sides: every partial sum is a multiple of 1/4
    below 2^22, so fp32 adds them exactly in any order."""
    import torch
    rng = np.random.default_rng(K)
    x = mxref.E2M1[rng.integers(0, 16, (M, K))].astype(np.float32)
    x[:, ::32] = 6.0
    wc = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    wsc = np.full((N, K // 32), 127, np.uint8)
    out = torch.empty((M, N), device="cuda")
    q.mxfp4_linear(_t(x), _t(wc), _t(wsc), out, q.alloc_mxfp4_linear_workspace(M, N, K))
    assert np.array_equal(_n(out), x.astype(np.float64) @ mxref.unpack(wc, wsc).T)


@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_linear_special_scales(q, M):
    """A NaN scale byte of a weight row or a NaN block of x reaches its row or column alone; the
    smallest scale (byte 0) on either side counts as 2^-127."""
    import torch
    N, K = 70, 288
    rng = np.random.default_rng(M)
    x = rng.standard_normal((M, K)).astype(np.float32)
    wc, wsc = _weights(rng, N, K)
    wsc[3, 1] = 255
    wsc[5, :] = 0
    xt = _t(x)
    xt[M - 1, K - 1] = float("inf") if M > 1 else xt[M - 1, K - 1]
    out = torch.empty((M, N), device="cuda")
    q.mxfp4_linear(xt, _t(wc), _t(wsc), out, q.alloc_mxfp4_linear_workspace(M, N, K))
    got = _n(out)
    nan = np.zeros((M, N), bool)
    nan[:, 3] = True
    nan[M - 1, :] |= M > 1
    assert np.array_equal(np.isnan(got), nan)
    a, w = mxref.unpack(*mxref.quantise(_n(xt))), mxref.unpack(wc, wsc)
    rows = ~nan[:, 5]
    y = a[rows] @ w[5]
    # sums of 2^-127-sized terms are subnormal: one step of 2^-149 for each addition
    assert (np.abs(got[rows, 5] - y) <= K * 2.0 ** -149 + mxref.dot_bound(K, np.abs(a[rows]) @ np.abs(w[5]))).all()


# ------------------------------------------------------------------ experts
def _route_of(rng, T, E, k, dropped, skew):
    z = rng.standard_normal((T, E)) - (np.log1p(rng.permutation(E)) if skew else 0)
    idx = np.argsort(-z, axis=1)[:, :k].astype(np.int32)
    w = rng.random((T, k)).astype(np.float32) * 2
    if dropped:
        gone = rng.random((T, k)) < dropped
        idx[gone], w[gone] = -1, 0
    return idx, w


EXPERTS = [  # T, H, F, E, k, shared, dropped, skew
    (1, 256, 128, 8, 1, False, 0, False),
    (1, 384, 256, 60, 4, True, 0, False),
    (2, 128, 128, 16, 8, True, 0.5, False),
    (3, 1152, 384, 8, 2, True, 1.0, False),      # no routed pair at all
    (16, 640, 512, 64, 8, True, 0, False),
    (16, 256, 128, 8, 8, False, 0.2, False),     # every expert sees every token
    (29, 512, 256, 16, 4, True, 0.2, True),
    (70, 256, 384, 8, 3, False, 0, True),
    (100, 768, 256, 16, 4, True, 0, False),
    (300, 256, 128, 8, 2, True, 0.2, True),
    (513, 384, 640, 60, 5, True, 0.1, True),
]


def _setup(q, case, seed):
    T, H, F, E, k, shared, dropped, skew = case
    rng = np.random.default_rng(seed)
    idx, w = _route_of(rng, T, E, k, dropped, skew)
    perm, off, act, na = mxref.group(idx, E)
    wc, wsc = _weights(rng, E + shared, 3, F * H)
    cfg = q.make_cfg(H, F, E, k, has_shared=shared, wbits=q.W_MXFP4, scale_group=32)
    weights = q.Weights(_t(wc.reshape(E + shared, -1)), _t(wsc.reshape(E + shared, -1)), None, None)
    return rng, cfg, weights, idx, w, [_t(a) for a in (off, perm, act, na)], wc, wsc


def _mats(wc, wsc, e, m, rows):
    return mxref.unpack(wc[e, m].reshape(rows, -1), wsc[e, m].reshape(rows, -1))


def _rows_of(idx, T, k, shared, E):
    """(expert, pair rows, tokens) of the hit experts and the shared one."""
    flat = idx.reshape(-1)
    for e in range(E):
        p = np.nonzero(flat == e)[0]
        if p.size:
            yield e, p, p // k
    if shared:
        yield E, T * k + np.arange(T), np.arange(T)


@pytest.mark.parametrize("case", EXPERTS, ids=str)
@pytest.mark.parametrize("dtype", DT)
def test_gate_up(q, case, dtype):
    import torch
    print(f"gate_up {case} {dtype}", flush=True)
    T, H, F, E, k, shared, _, _ = case
    rng, cfg, weights, idx, w, grouping, wc, wsc = _setup(q, case, 11 + T)
    x = _t(rng.standard_normal((T, H)).astype(np.float32), dtype)
    h = torch.full((T * (k + shared), F), 77.0, dtype=_dt(dtype), device="cuda")
    ws = q.alloc_mxfp4_experts_workspace(cfg, T)
    ws.fill_(0xFF)
    q.mxfp4_gate_up(cfg, weights, x, *grouping, h, ws)
    got, a = _n(h), mxref.unpack(*mxref.quantise(_n(x)))
    seen = np.zeros(got.shape[0], bool)
    for e, p, t in _rows_of(idx, T, k, shared, E):
        seen[p] = True
        wg, wu = _mats(wc, wsc, e, 0, F), _mats(wc, wsc, e, 1, F)
        g, u = a[t] @ wg.T, a[t] @ wu.T
        eg, eu = (mxref.dot_bound(H, np.abs(a[t]) @ np.abs(m).T) for m in (wg, wu))
        s = g / (1 + np.exp(-g))
        # |silu'| < 1.1; exp, division and two products in fp32: four steps each of at most 2 ulp
        tol = 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu + 8 * 2.0 ** -23 * np.abs(s * u)
        tol = tol + mxref.round_bound(np.abs(s * u) + tol, _dt(dtype))
        err = np.abs(got[p] - s * u)
        assert (err <= tol).all(), (e, (err / tol).max())
    assert (got[~seen] == 77.0).all()  # rows of empty slots stay as they were


@pytest.mark.parametrize("case", EXPERTS, ids=str)
@pytest.mark.parametrize("dtype", DT)
def test_down(q, case, dtype):
    import torch
    print(f"down {case} {dtype}", flush=True)
    T, H, F, E, k, shared, _, _ = case
    rng, cfg, weights, idx, w, grouping, wc, wsc = _setup(q, case, 23 + T)
    h = _t(rng.standard_normal((T * (k + shared), F)).astype(np.float32), dtype)
    h[:T * k][torch.from_numpy(idx.reshape(-1) < 0).cuda()] = float("nan")  # rows of empty slots do not enter
    out = torch.full((T, H), float("nan"), dtype=_dt(dtype), device="cuda")
    ws = q.alloc_mxfp4_experts_workspace(cfg, T)
    ws.fill_(0xFF)
    q.mxfp4_down(cfg, weights, h, _t(idx), _t(w), *grouping, out, ws)
    hn = np.nan_to_num(_n(h))
    a = mxref.unpack(*mxref.quantise(hn))
    want, tol, mag = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    wt = np.concatenate([w.reshape(-1).astype(np.float64), np.ones(T * shared)])
    for e, p, t in _rows_of(idx, T, k, shared, E):
        wd = _mats(wc, wsc, e, 2, H)
        y = a[p] @ wd.T
        np.add.at(want, t, wt[p, None] * y)
        np.add.at(mag, t, np.abs(wt[p, None] * y))
        np.add.at(tol, t, wt[p, None] * mxref.dot_bound(F, np.abs(a[p]) @ np.abs(wd).T))
    tol = tol + (k + 2) * 2.0 ** -23 * (mag + tol)
    tol = tol + mxref.round_bound(np.abs(want) + tol, _dt(dtype))
    err = np.abs(_n(out) - want)
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()


@pytest.mark.parametrize("T", [1, 4, 90])
def test_down_repeated_expert(q, T):
    """A token may name one expert in two slots: each counts with its own row and weight."""
    import torch
    case = (T, 256, 128, 8, 3, True, 0, False)
    rng, cfg, weights, idx, w, _, wc, wsc = _setup(q, case, 5)
    idx[:, 2] = idx[:, 0]
    perm, off, act, na = mxref.group(idx, 8)
    h = _t(rng.standard_normal((T * 4, 128)).astype(np.float32))
    out = torch.empty((T, 256), device="cuda")
    q.mxfp4_down(cfg, weights, h, _t(idx), _t(w), *[_t(a) for a in (off, perm, act, na)], out,
                 q.alloc_mxfp4_experts_workspace(cfg, T))
    a = mxref.unpack(*mxref.quantise(_n(h)))
    want, mag = np.zeros((T, 256)), np.zeros((T, 256))
    for e, p, t in _rows_of(idx, T, 3, True, 8):
        wd = _mats(wc, wsc, e, 2, 256)
        f = np.where(p < T * 3, w.reshape(-1)[np.minimum(p, T * 3 - 1)], 1.0)[:, None]
        np.add.at(want, t, f * (a[p] @ wd.T))
        np.add.at(mag, t, f * (np.abs(a[p]) @ np.abs(wd).T))
    assert (np.abs(_n(out) - want) <= (128 + 5) * 2.0 ** -23 * mag * (1 + 2.0 ** -10)).all()


# ------------------------------------------------------------------ how they are called
def test_layer_of_operators(q):
    """Route from logits, group, gate/up, down on one stream other than the current one, eagerly
    and as a replayed graph, against the eager result of the default stream bit for bit."""
    import torch
    T, H, F, E, k = 24, 256, 128, 16, 4
    rng = np.random.default_rng(3)
    wc, wsc = _weights(rng, E + 1, 3 * F * H)
    cfg = q.make_cfg(H, F, E, k, has_shared=True, wbits=q.W_MXFP4, scale_group=32)
    w = q.Weights(_t(wc), _t(wsc), None, None)
    r = q.make_router(E, k, 4, 2, scale=2.5)
    z, x = _t(rng.standard_normal((T, E)).astype(np.float32)), _t(rng.standard_normal((T, H)).astype(np.float32))
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = q.alloc_mxfp4_experts_workspace(cfg, T)

    def layer(out):
        idx, tw = i32(T, k), torch.zeros((T, k), device="cuda")
        cnt, off, perm, act, na = i32(E), i32(E + 1), i32(T * k), i32(E), i32(1)
        h = torch.zeros((T * (k + 1), F), device="cuda")
        q.route_logits(r, z, idx, tw)
        q.group(cfg, idx, T, cnt, off, perm, act, na)
        q.mxfp4_gate_up(cfg, w, x, off, perm, act, na, h, ws)
        q.mxfp4_down(cfg, w, h, idx, tw, off, perm, act, na, out, ws)

    out = torch.empty((T, H), device="cuda")
    layer(out)
    want = out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out.zero_()
        layer(out)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer(out)
    for i in range(4):
        x.copy_(_t(np.random.default_rng(i).standard_normal((T, H)).astype(np.float32)))
        g.replay()
        torch.cuda.synchronize()
        eager = torch.empty_like(out)
        layer(eager)
        assert torch.equal(out, eager), i


@pytest.mark.parametrize("M,N,K", [(1, 64, 2048), (300, 300, 512)])
def test_linear_reproducible(q, M, N, K):
    import torch
    rng = np.random.default_rng(0)
    x = _t(rng.standard_normal((M, K)).astype(np.float32))
    wc, wsc = (_t(a) for a in _weights(rng, N, K))
    ws = q.alloc_mxfp4_linear_workspace(M, N, K)
    outs = [torch.empty((M, N), device="cuda") for _ in range(4)]
    for o in outs:
        q.mxfp4_linear(x, wc, wsc, o, ws)
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_empty_calls(q):
    import torch
    e = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    u8 = torch.uint8
    q.mxfp4_quantize(e(0, 64), e(0, 32, dtype=u8), e(0, 2, dtype=u8))
    q.mxfp4_dequantize(e(0, 32, dtype=u8), e(0, 2, dtype=u8), e(0, 64))
    ws = q.alloc_mxfp4_linear_workspace(4, 8, 64)
    q.mxfp4_linear(e(0, 64), e(8, 32, dtype=u8), e(8, 2, dtype=u8), e(0, 8), ws)
    q.mxfp4_linear(e(4, 64), e(0, 32, dtype=u8), e(0, 2, dtype=u8), e(4, 0), ws)
    torch.cuda.synchronize()


def test_refused_tensors(q):
    """The binding's own checks: types, shapes, strides, device."""
    import torch
    x = torch.zeros((4, 64), device="cuda")
    c, s = torch.zeros((4, 32), dtype=torch.uint8, device="cuda"), torch.zeros((4, 2), dtype=torch.uint8, device="cuda")
    with pytest.raises(TypeError):
        q.mxfp4_quantize(x.double(), c, s)
    with pytest.raises(ValueError):
        q.mxfp4_quantize(x, c[:3], s)
    with pytest.raises(ValueError):
        q.mxfp4_quantize(torch.zeros((64, 4), device="cuda").t(), c, s)
    with pytest.raises(ValueError):
        q.mxfp4_quantize(x.cpu(), c, s)
    with pytest.raises(q.ColiError) as e:  # 16-byte alignment of x
        q.mxfp4_quantize(torch.zeros(4 * 64 + 1, device="cuda")[1:].view(4, 64), c, s)
    assert e.value.status == q.COLI_E_ALIGN
    ws = q.alloc_mxfp4_linear_workspace(1, 4, 64)
    with pytest.raises(q.ColiError) as e:
        q.mxfp4_linear(x, c, s, torch.zeros((4, 4), device="cuda"), ws[:256])
    assert e.value.status == q.COLI_E_WORKSPACE
    with pytest.raises(TypeError):
        q.mxfp4_linear(x, c, s, torch.zeros((4, 4), device="cuda", dtype=torch.bfloat16), ws)


# ------------------------------------------------------------------ sizes of the tiled kernels
TILED = [  # 128 x 128 tiles: several strips, odd N, short rows; then 256 x 256 ones
    (33, 10300, 96), (40, 11003, 544), (129, 3500, 288), (300, 2304, 640), (257, 2101, 1024), (513, 1300, 1312),
    (1025, 9801, 320), (2048, 6144, 128)]


@pytest.mark.parametrize("M,N,K", TILED)
@pytest.mark.parametrize("dtype", DT)
def test_linear_tiled(q, M, N, K, dtype):
    print(f"linear M={M} N={N} K={K} {dtype}", flush=True)
    _check_linear(q, M, N, K, dtype, M + N + K)


def test_linear_writes_its_output_alone(q):
    """Rows that end inside a 16-byte piece: neighbours of the output keep what they held."""
    import torch
    for M, N in ((5, 13), (300, 2305), (200, 3507)):
        K = 96
        rng = np.random.default_rng(N)
        buf = torch.full((64 + M * N + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
        out = buf[64:64 + M * N].view(M, N)
        wc, wsc = _weights(rng, N, K)
        x = _t(rng.standard_normal((M, K)).astype(np.float32), "bfloat16")
        q.mxfp4_linear(x, _t(wc), _t(wsc), out, q.alloc_mxfp4_linear_workspace(M, N, K))
        assert (buf[:64] == 5).all() and (buf[64 + M * N:] == 5).all()


def test_linear_unaligned_scales(q):
    """Scale bytes at any address, for both kernels."""
    import torch
    for M, N, K in ((1, 40, 512), (20, 40, 1024), (300, 2304, 640)):
        rng = np.random.default_rng(K)
        wc, wsc = _weights(rng, N, K)
        x = _t(rng.standard_normal((M, K)).astype(np.float32))
        want, got = (torch.empty((M, N), device="cuda") for _ in range(2))
        ws = q.alloc_mxfp4_linear_workspace(M, N, K)
        q.mxfp4_linear(x, _t(wc), _t(wsc), want, ws)
        off = torch.zeros(wsc.size + 1, dtype=torch.uint8, device="cuda")
        off[1:] = _t(wsc).flatten()
        q.mxfp4_linear(x, _t(wc), off[1:].view(N, K // 32), got, ws)
        assert torch.equal(got, want)


EXPERTS_MORE = [
    (20, 640, 512, 64, 1, True, 0, False),       # down of two blocks of 16 tokens
    (48, 384, 256, 256, 8, True, 0.2, False),    # three, the experts of each its own
    (33, 256, 640, 128, 2, False, 0, True),      # a last block of one token
    (1200, 256, 128, 4, 2, True, 0, False),      # more row tiles of an expert than go together
    (5, 2048, 384, 16, 2, True, 0, False),       # 8 down rows to a workgroup, K = 3 * 128
    (3, 5248, 128, 8, 2, False, 0, False),       # 24 rows, the last workgroup short
]


@pytest.mark.parametrize("case", EXPERTS_MORE, ids=str)
@pytest.mark.parametrize("dtype", DT)
def test_gate_up_more(q, case, dtype):
    test_gate_up(q, case, dtype)


@pytest.mark.parametrize("case", EXPERTS_MORE, ids=str)
@pytest.mark.parametrize("dtype", DT)
def test_down_more(q, case, dtype):
    test_down(q, case, dtype)


@pytest.mark.parametrize("T", [1, 16, 40])
def test_gate_up_extremes(q, T):
    """Gates far from 0, both signs: silu is g or 0 there, never NaN."""
    import torch
    H, F, E, k = 256, 128, 4, 2
    cfg = q.make_cfg(H, F, E, k, has_shared=False, wbits=q.W_MXFP4, scale_group=32)
    codes = np.full((E, 3, F * H // 2), 0x22, np.uint8)           # every weight 1 ..
    codes[:, 0, F * H // 4:] = 0xAA                               # .. the gate's upper half -1
    scales = np.full((E, 3, F * H // 32), 127, np.uint8)
    idx = np.tile(np.array([[0, 3]], np.int32), (T, 1))
    grouping = [_t(a) for a in (lambda p, o, a, n: (o, p, a, n))(*mxref.group(idx, E))]
    w = q.Weights(_t(codes.reshape(E, -1)), _t(scales.reshape(E, -1)), None, None)
    h = torch.empty((T * k, F), device="cuda")
    for v in (1.0, 64.0, 2.0 ** 40, 2.0 ** 60):
        x = torch.full((T, H), v, device="cuda")
        q.mxfp4_gate_up(cfg, w, x, *grouping, h, q.alloc_mxfp4_experts_workspace(cfg, T))
        got = _n(h)
        # e^-256 is nothing beside 1; past fp32's largest (2^128) the rounded value is inf
        want = (v * H) ** 2 if (v * H) ** 2 < 2.0 ** 128 else np.inf
        assert np.array_equal(got[:, :F // 2], np.full((T * k, F // 2), want)), v
        assert (np.abs(got[:, F // 2:]) <= 2.0 ** -120).all(), v                            # -256 v e^(-256 v) 256 v


def test_layer_on_side_stream_with_reused_workspace(q):
    """Two layers one after another on a stream of their own, with one workspace and outputs that
    another stream wrote before: the second equals a fresh run."""
    import torch
    case = (70, 256, 384, 8, 3, True, 0.1, False)
    rng, cfg, weights, idx, w, grouping, _, _ = _setup(q, case, 77)
    T, H, F, k = 70, 256, 384, 3
    x = _t(rng.standard_normal((T, H)).astype(np.float32), "bfloat16")
    it, wt = _t(idx), _t(w)

    def layer(ws):
        h = torch.zeros((T * (k + 1), F), dtype=torch.bfloat16, device="cuda")
        out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        q.mxfp4_gate_up(cfg, weights, x, *grouping, h, ws)
        q.mxfp4_down(cfg, weights, h, it, wt, *grouping, out, ws)
        return out

    want = layer(q.alloc_mxfp4_experts_workspace(cfg, T))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ws = q.alloc_mxfp4_experts_workspace(cfg, 100)
        outs = [layer(ws) for _ in range(3)]
    s.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_down_token_blocks_bitidentical(q):
    """A token's down row does not depend on the tokens beside it while both calls take 16 at a time."""
    import torch
    case = (20, 640, 512, 64, 2, True, 0, False)
    T, H, F, E, k = case[:5]
    rng, cfg, weights, idx, w, grouping, _, _ = _setup(q, case, 9)
    h = _t(rng.standard_normal((T * (k + 1), F)).astype(np.float32))
    out, one = torch.empty((T, H), device="cuda"), torch.empty((4, H), device="cuda")
    ws = q.alloc_mxfp4_experts_workspace(cfg, T)
    q.mxfp4_down(cfg, weights, h, _t(idx), _t(w), *grouping, out, ws)
    rows = torch.cat([h[16 * k:20 * k], h[T * k + 16:]]).contiguous()  # the last four tokens alone
    perm, off, act, na = mxref.group(idx[16:], E)
    q.mxfp4_down(cfg, weights, rows, _t(idx[16:]), _t(w[16:]), *[_t(a) for a in (off, perm, act, na)], one, ws)
    assert torch.equal(out[16:], one)


def test_gate_up_extremes_tiled(q):
    """The same through the tiled kernel."""
    test_gate_up_extremes(q, 300)


@pytest.mark.parametrize("T,K", [(1, 1920), (1, 640), (5, 1152), (16, 896), (300, 1920)])
def test_experts_rows_between_groups(q, T, K):
    """Rows that end at every place of a group of 16 blocks that their length allows."""
    for dtype in DT:
        test_gate_up(q, (T, K, 256, 16, 2, True, 0, False), dtype)
        test_down(q, (T, 256, K, 16, 2, True, 0, False), dtype)


@pytest.mark.parametrize("blocks", range(16, 33))
def test_linear_rows_between_groups(q, blocks):
    _check_linear(q, 1, 40, 32 * blocks, "bfloat16", blocks)
    _check_linear(q, 9, 40, 32 * blocks, "bfloat16", blocks)


# a short last column tile behind strips of several whole ones: 128 x 128 tiles, 256 x 256 tiles
@pytest.mark.parametrize("M,N,K", [(1000, 11003, 96), (2048, 9000, 96), (1800, 9001, 544)])
def test_linear_short_tile_after_strips(q, M, N, K):
    print(f"linear M={M} N={N} K={K}", flush=True)
    _check_linear(q, M, N, K, "bfloat16", M + N + K)


@pytest.mark.parametrize("H", [384, 896, 1408, 1920])
def test_down_short_tile_after_strips(q, H):
    test_down(q, (300, H, 256, 16, 2, True, 0, False), "bfloat16")


@pytest.mark.parametrize("K", [640, 768, 1152, 1280, 1664, 2176])
def test_experts_odd_stages_of_several_column_tiles(q, K):
    """Rows of 3, 5, 7 and 9 stages of 256 inputs, several column tiles, tokens past one row tile."""
    test_gate_up(q, (300, K, 512, 8, 2, True, 0, False), "bfloat16")
    test_down(q, (300, 1024, K, 8, 2, True, 0, False), "bfloat16")


@pytest.mark.parametrize("T,H,F,E,k", [(2, 256, 2048, 64, 8), (16, 640, 2048, 64, 8), (16, 256, 1152, 16, 3),
                                       (40, 384, 1024, 8, 2), (90, 256, 640, 16, 8)])
@pytest.mark.parametrize("shared", [False, True])
def test_down_row_whatever_its_neighbours(q, T, H, F, E, k, shared):
    """A token's down row is the same bits whichever experts the tokens beside it hold."""
    import torch
    rng, cfg, weights, idx, w, _, _, _ = _setup(q, (T, H, F, E, k, shared, 0, False), T + F)
    h = _t(rng.standard_normal((T * (k + shared), F)).astype(np.float32))
    ws = q.alloc_mxfp4_experts_workspace(cfg, T)
    rows = []
    for i in range(6):
        other, _ = _route_of(np.random.default_rng(i), T, E, k, 0.3 if i else 0, False)
        other[T // 2] = idx[T // 2]
        perm, off, act, na = mxref.group(other, E)
        out = torch.empty((T, H), device="cuda")
        q.mxfp4_down(cfg, weights, h, _t(other), _t(w), *[_t(a) for a in (off, perm, act, na)], out, ws)
        rows.append(out[T // 2].clone())
    assert all(torch.equal(r, rows[0]) for r in rows)


@pytest.mark.parametrize("T,H,F,E,k", [(1, 256, 128, 8, 4), (1, 384, 2048, 64, 8), (3, 5248, 640, 16, 5), (16, 640, 512, 64, 8),
                                       (16, 256, 1152, 8, 3), (20, 384, 2048, 8, 4), (90, 256, 640, 16, 8), (300, 256, 384, 8, 2)])
@pytest.mark.parametrize("shared", [False, True])
def test_down_adds_in_slot_order(q, T, H, F, E, k, shared):
    """Rows that are exact and weights of powers of two: the sum over slots, then the shared expert's
    row, rounded to fp32 at every step, bit for bit. Empty slots and repeated experts among them."""
    import torch
    rng = np.random.default_rng(T * F + k)
    idx, _ = _route_of(rng, T, E, k, 0.1, False)
    if k > 2:
        idx[::3, k - 1] = idx[::3, 0]  # an expert in two slots
    w = np.exp2(rng.integers(-18, 19, (T, k))).astype(np.float32)
    cfg = q.make_cfg(H, F, E, k, has_shared=shared, wbits=q.W_MXFP4, scale_group=32)
    codes = rng.integers(0, 256, (E + shared, 3, F * H // 2), dtype=np.uint8)
    scales = np.full((E + shared, 3, F * H // 32), 127, np.uint8)
    x = mxref.E2M1[rng.integers(0, 16, (T * (k + shared), F))]
    x[:, ::32] = 6.0  # a block's power of two is 1: every sum of a row is a multiple of 1/4 below 2^22
    perm, off, act, na = mxref.group(idx, E)
    out = torch.empty((T, H), device="cuda")
    q.mxfp4_down(cfg, q.Weights(_t(codes.reshape(E + shared, -1)), _t(scales.reshape(E + shared, -1)), None, None),
                 _t(x.astype(np.float32)), _t(idx), _t(w), *[_t(a) for a in (off, perm, act, na)], out,
                 q.alloc_mxfp4_experts_workspace(cfg, T))
    y = np.zeros((T * (k + shared), H), np.float32)
    for e, p, _ in _rows_of(idx, T, k, shared, E):
        y[p] = x[p] @ _mats(codes, scales, e, 2, H).T
    want = np.zeros((T, H), np.float32)
    for j in range(k):
        there = idx[:, j] >= 0
        want[there] += (w[there, j, None] * y[:T * k].reshape(T, k, H)[there, j])
    if shared:
        want += y[T * k:]
    assert np.array_equal(out.cpu().numpy(), want)


EXPERTS_LIMITS = [  # most slots of the kernel for few tokens and more than it takes, most experts
    (1, 256, 128, 24, 16, True, 0, False), (16, 128, 640, 24, 16, True, 0.1, False), (40, 256, 128, 32, 16, False, 0, False),
    (1, 128, 256, 24, 20, True, 0, False), (16, 256, 128, 24, 20, False, 0.1, False), (40, 128, 128, 24, 20, True, 0, False),
    (1, 128, 128, 1024, 8, True, 0, False), (16, 256, 128, 1024, 16, True, 0, False), (600, 128, 128, 1024, 2, True, 0.1, True),
    (9, 128, 128, 64, 64, False, 0.2, False),
]


@pytest.mark.parametrize("case", EXPERTS_LIMITS, ids=str)
def test_gate_up_limits(q, case):
    test_gate_up(q, case, "bfloat16")


@pytest.mark.parametrize("case", EXPERTS_LIMITS, ids=str)
def test_down_limits(q, case):
    test_down(q, case, "bfloat16")


@pytest.mark.parametrize("T", [1, 5, 40, 300])
def test_experts_scales_at_any_dword(q, T):
    """Scales that start 4 bytes past a 16-byte address: the results of aligned ones, bit for bit."""
    import torch
    H, F, E, k = 512, 512, 8, 2
    rng, cfg, weights, idx, w, grouping, _, _ = _setup(q, (T, H, F, E, k, True, 0, False), T)
    moved = torch.empty(weights.scales.numel() + 16, dtype=torch.uint8, device="cuda")
    at = (4 - moved.data_ptr()) % 16
    moved = moved[at:at + weights.scales.numel()].view(weights.scales.shape)
    moved.copy_(weights.scales)
    assert moved.data_ptr() % 16 == 4 and weights.scales.data_ptr() % 16 == 0
    x, h = _t(rng.standard_normal((T, H)).astype(np.float32)), _t(rng.standard_normal((T * (k + 1), F)).astype(np.float32))
    ws = q.alloc_mxfp4_experts_workspace(cfg, T)
    got = []
    for scales in (weights.scales, moved):
        wt = q.Weights(weights.experts, scales, None, None)
        hh, out = torch.empty((T * (k + 1), F), device="cuda"), torch.empty((T, H), device="cuda")
        q.mxfp4_gate_up(cfg, wt, x, *grouping, hh, ws)
        q.mxfp4_down(cfg, wt, h, _t(idx), _t(w), *grouping, out, ws)
        got.append((hh, out))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("T", [1, 8, 300])
def test_gate_up_gates_near_the_exponentials_end(q, T):
    """Gates from -80 to -88.6, whose e^-g is still a finite fp32 value: g / (1 + e^-g) is not 0 there."""
    import torch
    H, F, E, k = 128, 128, 4, 2
    codes = np.zeros((3, F, H), np.uint8)
    steps = 640 + np.arange(F) % 70  # -8 g, as a sum of E2M1 values of weight 2^-3
    for f in range(F):
        left, i = steps[f], 0
        while left:
            c, v = next((c, v) for c, v in ((7, 6), (6, 4), (5, 3), (4, 2), (2, 1)) if v <= left)
            codes[0, f, i] = c | 8
            left, i = left - v, i + 1
    codes[1, :, 0] = 2  # every up value 1
    blocks = codes.reshape(3, F, H // 32, 32)
    packed = (blocks[..., :16] | (blocks[..., 16:] << 4)).reshape(3, -1)
    scales = np.full((3, F * H // 32), 127, np.uint8)
    scales[0] = 124
    cfg = q.make_cfg(H, F, E, k, has_shared=False, wbits=q.W_MXFP4, scale_group=32)
    w = q.Weights(_t(np.stack([packed.reshape(-1)] * E)), _t(np.stack([scales.reshape(-1)] * E)), None, None)
    perm, off, act, na = mxref.group(np.tile(np.array([[0, 3]], np.int32), (T, 1)), E)
    h = torch.empty((T * k, F), device="cuda")
    q.mxfp4_gate_up(cfg, w, torch.ones((T, H), device="cuda"), *[_t(a) for a in (off, perm, act, na)], h,
                    q.alloc_mxfp4_experts_workspace(cfg, T))
    g = -steps / 8.0  # exact in fp32 in any order
    want = g / (1 + np.exp(-g))
    # exp, sum, division, product: four steps each of at most 2 ulp
    assert (np.abs(_n(h) - want) <= 8 * 2.0 ** -23 * np.abs(want)).all()
