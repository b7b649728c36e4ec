"""The int8 operators with token and channel scales (quantise, dense product, the experts' gate/up
and down products over a route) against their 64-bit definitions. Codes and scales are compared bit
for bit, and so are products without a bias, whose integer sums are exact; the rest within the
roundings that the definitions leave open."""
import numpy as np
import pytest

import i8ref

pytestmark = pytest.mark.gpu

DT = ["float32", "bfloat16", "float16"]
U = 2.0 ** -24  # half a step of fp32


@pytest.fixture(scope="module")
def q():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_moe_sigmoid_amd as q
    q.lib()
    return q


def _dt(name):
    import torch
    return getattr(torch, name)


def _t(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(_dt(dtype))


def _n(t):
    return t.detach().cpu().double().numpy()


def _half(dtype):
    import torch
    return torch.finfo(_dt(dtype)).eps / 2


def _tiny(dtype):
    """Half a step of the type's subnormal numbers."""
    import torch
    f = torch.finfo(_dt(dtype))
    return f.tiny * f.eps / 2


def _near(got, want, tol, dtype):
    """Within tol and the type's rounding, by which values from the middle between its largest number
    and the next power of two on are infinite."""
    import torch
    f = torch.finfo(_dt(dtype))
    infinite = np.isinf(got) & (np.sign(got) == np.sign(want)) & (np.abs(want) + tol >= f.max * (1 + f.eps / 4))
    with np.errstate(invalid="ignore"):
        return (np.abs(got - want) <= tol + _half(dtype) * (np.abs(want) + tol) + _tiny(dtype)) | infinite


def _rows(rng, M, K, dtype):
    """Rows of very different sizes, in range of the type."""
    x = rng.standard_normal((M, K)) * np.exp2(2 * rng.standard_normal((M, 1)))
    return _t(x.astype(np.float32), dtype)


def _quantise(q, x):
    import torch
    codes = torch.full(x.shape, 0x55, dtype=torch.int8, device="cuda")
    scales = torch.full((x.shape[0],), -7.0, device="cuda")
    q.int8_quantize(x, codes, scales)
    torch.cuda.synchronize()
    return codes.cpu().numpy(), scales.cpu().numpy()


# ------------------------------------------------------------------ quantisation
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (1, 512), (5, 528), (257, 64), (2, 1040), (7, 2048), (9, 2064),
                                       (4, 4112), (3, 6144), (2, 8192), (2, 8208), (1, 131072), (0, 64)])
def test_quantise_random(q, dtype, rows, cols):
    rng = np.random.default_rng(rows * 7919 + cols)
    x = _rows(rng, rows, cols, dtype)
    codes, scales = _quantise(q, x)
    if not rows:
        return
    rc, rs = i8ref.quantise(x.float().cpu().numpy())
    assert np.array_equal(scales, rs)
    assert np.array_equal(codes, rc)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("top", [127.0, 1.0, 3.0, 1e-3, 6e4])
def test_quantise_borders(q, dtype, top):
    """Values at and one step beside every half between two codes."""
    import torch
    s = np.float32(np.float32(torch.tensor(top, dtype=_dt(dtype)).item()) / np.float32(127))
    half = torch.tensor(((np.arange(127) + 0.5) * np.float64(s)).astype(np.float32)).to(_dt(dtype))
    big = torch.tensor([3.0e4], dtype=_dt(dtype))
    vals = torch.cat([half, torch.nextafter(half, big), torch.nextafter(half, -big)])
    vals = torch.cat([vals, -vals])
    vals = vals[vals.abs().float() <= top]
    pad = (-(vals.numel() + 1)) % 16
    x = torch.cat([torch.tensor([top], dtype=_dt(dtype)), vals, torch.zeros(pad, dtype=_dt(dtype))])[None].cuda()
    codes, scales = _quantise(q, x)
    rc, rs = i8ref.quantise(x.float().cpu().numpy())
    assert np.array_equal(scales, rs)
    assert np.array_equal(codes, rc)


@pytest.mark.parametrize("cols", [64, 2048, 9216])
def test_quantise_smallest_and_largest(q, cols):
    """Rows whose scale is subnormal, rounds to 0 or is near the end of fp32; rows of zeros."""
    rng = np.random.default_rng(cols)
    x = rng.standard_normal((12, cols)).astype(np.float32)
    x /= np.abs(x).max(1, keepdims=True)
    for i, top in enumerate([2.0 ** -149, 2.0 ** -143, 2.0 ** -142, 5 * 2.0 ** -140, 2.0 ** -130, 2.0 ** -126, 2.0 ** -119.5,
                             2.0 ** -118, 0.0, 2.0 ** 127, float(np.finfo(np.float32).max), 1.0]):
        x[i] = (x[i].astype(np.float64) * top).astype(np.float32)
    codes, scales = _quantise(q, _t(x))
    rc, rs = i8ref.quantise(x)
    assert np.array_equal(scales, rs)
    assert np.array_equal(codes, rc)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("cols", [96, 1536, 8224])
def test_quantise_not_finite(q, dtype, cols):
    """A row with an infinity or a NaN: scale NaN, codes 0; its neighbours as they are."""
    rng = np.random.default_rng(cols)
    x = rng.standard_normal((6, cols)).astype(np.float32)
    x[1, cols - 1] = np.inf
    x[2, 0] = np.nan
    x[4, cols // 2] = -np.inf
    codes, scales = _quantise(q, _t(x, dtype))
    rc, rs = i8ref.quantise(_t(x, dtype).float().cpu().numpy())
    assert np.array_equal(scales, rs, equal_nan=True) and np.isnan(scales[[1, 2, 4]]).all()
    assert np.array_equal(codes, rc)


def test_quantise_more_rows_than_one_launch(q):
    import torch
    rows = 8 * (1 << 23) + 9
    x = torch.zeros((rows, 16), dtype=torch.bfloat16, device="cuda")
    at = [0, 1 << 26, rows - 10, rows - 9, rows - 1]
    for i in at:
        x[i] = torch.randn(16, device="cuda")
    codes, scales = torch.full((rows, 16), 5, dtype=torch.int8, device="cuda"), torch.full((rows,), 5.0, device="cuda")
    q.int8_quantize(x, codes, scales)
    rc, rs = i8ref.quantise(x[at].float().cpu().numpy())
    assert np.array_equal(codes[at].cpu().numpy(), rc) and np.array_equal(scales[at].cpu().numpy(), rs)
    assert int((codes != 0).any(1).sum()) == len(set(at)) and int((scales != 0).sum()) == len(set(at))


# ------------------------------------------------------------------ dense product
def _weights(rng, N, K):
    return (rng.integers(-128, 128, (N, K), dtype=np.int8),
            ((0.5 + rng.random(N)) / (73 * np.sqrt(K))).astype(np.float32))


def _linear(q, x, codes, scales, bias=None, M_max=None):
    import torch
    M, K = x.shape
    N = codes.shape[0]
    out = torch.full((M, N), 77.0, dtype=x.dtype, device="cuda")
    ws = q.alloc_int8_linear_workspace(M_max or M, N, K)
    ws.fill_(0xFF)
    q.int8_linear(x, codes, scales, out, ws, bias=bias)
    torch.cuda.synchronize()
    return out


LINEAR = [(1, 1, 16), (1, 16, 64), (1, 77, 2064), (1, 300, 6144), (1, 5, 49168), (2, 33, 272), (15, 17, 4096), (16, 64, 256),
          (17, 31, 1040), (33, 129, 528), (64, 48, 2048), (65, 130, 4112), (200, 77, 784), (7, 2051, 144), (129, 1, 48),
          (300, 515, 1008), (513, 1031, 320), (1000, 257, 2064), (257, 256, 16), (770, 520, 112), (512, 512, 8192),
          (20, 20500, 48), (70, 5200, 272), (300, 2051, 1008), (1000, 1031, 2064), (129, 3460, 16), (513, 4096, 8192), (2900, 4100, 144),
          (3001, 4361, 400), (3000, 4096, 1024), (257, 49160, 16), (32, 12700, 80), (64, 9510, 656), (512, 1200, 528),
          (1500, 3001, 272), (1300, 4096, 1040), (1601, 3090, 144), (48, 3125, 1296), (48, 3126, 1296), (49, 63, 400), (9, 17000, 640),
          (8, 19000, 640), (1025, 1023, 7200)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear_exact(q, dtype, M, N, K):
    """Without a bias every step is fixed: an exact sum, two fp32 products, the output's rounding."""
    import torch
    rng = np.random.default_rng(M * 31 + N * 7 + K)
    x = _rows(rng, M, K, dtype)
    codes, scales = _weights(rng, N, K)
    out = _linear(q, x, _t(codes), _t(scales))
    rc, rs = i8ref.quantise(x.float().cpu().numpy())
    want = torch.from_numpy(i8ref.product32(i8ref.dot(rc, codes), rs, scales)).to(_dt(dtype))
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("M,N,K", [(1, 300, 2064), (7, 77, 528), (65, 130, 4112), (515, 1027, 272), (300, 768, 1024), (515, 4099, 272),
                                   (2900, 4352, 528), (1500, 3001, 272), (130, 8000, 1040), (61, 190, 2064)])
def test_linear_bias(q, dtype, M, N, K):
    rng = np.random.default_rng(M + N + K)
    x = _rows(rng, M, K, dtype)
    codes, scales = _weights(rng, N, K)
    bias = rng.standard_normal(N).astype(np.float32)
    got = _n(_linear(q, x, _t(codes), _t(scales), _t(bias)))
    rc, rs = i8ref.quantise(x.float().cpu().numpy())
    y = i8ref.dot(rc, codes) * rs.astype(np.float64)[:, None] * scales.astype(np.float64)
    # the sum's way to fp32, two products, the addition (or one fused with it), the output's rounding
    want = y + bias
    tol = 3 * U * np.abs(y) + U * (np.abs(want) + 3 * U * np.abs(y))
    assert _near(got, want, tol, dtype).all()


@pytest.mark.parametrize("M", [1, 3, 40, 300, 4100])
def test_linear_largest_sums(q, M):
    """K = 2^17 with every product at its largest: the sums end just below 2^31."""
    import torch
    K, N = 131072, 20 if M < 4000 else 400
    x = torch.full((M, K), 3.0, device="cuda")
    x[:, 1::2] *= -1
    codes = np.full((N, K), -128, np.int8)
    codes[:, 1::2] = 127
    codes[1] = -codes[0] - 1  # -128 and 127 the other way round
    scales = np.ones(N, np.float32)
    out = _linear(q, x, _t(codes), _t(scales)).cpu().numpy()
    rc, rs = i8ref.quantise(x[:1].cpu().numpy())
    want = i8ref.product32(i8ref.dot(rc, codes), rs, scales)
    assert abs(i8ref.dot(rc, codes)).max() == 127 * 127.5 * K  # 0.988 of 2^31
    assert np.array_equal(out, np.repeat(want, M, 0))


@pytest.mark.parametrize("M", [1, 5, 70, 600, 3000])
def test_linear_rows_stand_alone(q, M):
    """Rows with an infinity or a NaN give NaN in their own row only, rows of zeros the bias; a row does
    not depend on the rows beside it or on the workspace's size."""
    import torch
    rng = np.random.default_rng(M)
    N, K = 4200, 1040
    x = _rows(rng, M, K, "float32")
    codes, scales = _weights(rng, N, K)
    wt, st = _t(codes), _t(scales)
    one = torch.cat([_linear(q, x[i:i + 1], wt, st, M_max=M + 3) for i in range(min(M, 6))])
    x2 = x.clone()
    if M > 4:
        x2[1, 7], x2[2, K - 1] = float("nan"), float("-inf")
        x2[3] = 0
    out = _linear(q, x2, wt, st, M_max=2 * M)
    if M > 4:
        assert out[1].isnan().all() and out[2].isnan().all() and (out[3] == 0).all()
        assert torch.equal(out[[0, 4]], one[[0, 4]]) and not out[4:].isnan().any()
        bias = torch.arange(N, device="cuda", dtype=torch.float32)
        assert torch.equal(_linear(q, x2, wt, st, bias)[3], bias)
    else:
        assert torch.equal(out, one)


# ------------------------------------------------------------------ experts
EXPERTS = [  # T, H, F, E, k, shared, dropped
    (1, 256, 128, 4, 2, False, False), (1, 1280, 384, 16, 8, True, False), (3, 640, 256, 8, 3, True, True),
    (17, 384, 640, 16, 4, True, False), (40, 512, 256, 5, 1, False, True), (70, 256, 384, 64, 8, True, True),
    (130, 896, 128, 3, 2, True, False), (300, 384, 512, 16, 4, True, True), (600, 256, 256, 60, 6, False, False),
    (90, 512, 384, 200, 7, True, True), (257, 640, 896, 2, 2, False, True),
    (1, 6144, 2048, 12, 8, True, False), (2, 2048, 1024, 64, 8, False, True), (16, 1024, 1408, 100, 16, True, True), (15, 896, 256, 1024, 17, True, False),
    (33, 640, 2048, 256, 8, False, False), (64, 384, 128, 500, 12, True, True), (49, 6144, 256, 64, 2, True, False),
    (49, 256, 1024, 4, 1, True, True), (48, 256, 1024, 4, 1, False, False), (97, 4096, 512, 32, 4, False, False), (700, 128, 1152, 6, 3, True, False),
    (270, 1408, 128, 1, 1, True, True)]


def _case(rng, T, H, F, E, k, shared, dropped, unused=True):
    idx = np.stack([rng.permutation(E if E < 8 or not unused else E - 2)[:k] for _ in range(T)]).astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    if dropped:
        gone = rng.random((T, k)) < 0.25
        gone[T // 2] = True  # a token that no expert takes
        idx[gone], w[gone] = -1, 0
    n = E + int(shared)
    codes = rng.integers(-128, 128, (n, 3 * F * H), dtype=np.int8)
    scales = ((0.5 + rng.random((n, 2 * F + H))) / 73).astype(np.float32)
    scales[:, :2 * F] /= np.sqrt(H)
    scales[:, 2 * F:] /= np.sqrt(F)
    return idx, w, codes, scales


def _grouped(q, idx, E):
    import torch
    T, k = idx.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    g = dict(off=torch.empty(E + 1, **i32), perm=torch.zeros(T * k, **i32), active=torch.empty(E, **i32), n_active=torch.empty(1, **i32))
    pos = torch.empty(T * k, **i32)
    q.sort_pairs(_t(idx), g["off"], g["perm"], pos, g["active"], g["n_active"], q.alloc_sort_pairs_workspace(T * k, E))
    return g


def _rows_of(idx, E, shared):
    """(expert, its rows of h, their tokens)."""
    T, k = idx.shape
    for e in range(E):
        p = np.nonzero(idx.reshape(-1) == e)[0]
        if p.size:
            yield e, p, p // k
    if shared:
        yield E, T * k + np.arange(T), np.arange(T)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,H,F,E,k,shared,dropped", EXPERTS)
def test_gate_up(q, dtype, T, H, F, E, k, shared, dropped):
    import torch
    rng = np.random.default_rng(T * 13 + H + F + E)
    idx, _, codes, scales = _case(rng, T, H, F, E, k, shared, dropped)
    x = _rows(rng, T, H, dtype)
    cfg = q.make_cfg(H, F, E, k, has_shared=shared, wbits=8)
    h = torch.full((T * (k + shared), F), 9.0, dtype=_dt(dtype), device="cuda")
    ws = q.alloc_int8_experts_workspace(cfg, T)
    ws.fill_(0xFF)
    g = _grouped(q, idx, E)
    q.int8_gate_up(cfg, q.Weights(_t(codes.view(np.uint8) if T % 2 else codes), _t(scales), None, None), x, **g, h=h, workspace=ws)
    got = _n(h)
    rc, rs = i8ref.quantise(x.float().cpu().numpy())
    seen = np.zeros(h.shape[0], bool)
    for e, rows, tokens in _rows_of(idx, E, shared):
        wg, sc = codes[e, :2 * F * H].reshape(2 * F, H), scales[e, :2 * F].astype(np.float64)
        gu = i8ref.dot(rc[tokens], wg) * rs[tokens].astype(np.float64)[:, None] * sc
        gate, up = gu[:, :F], gu[:, F:]
        with np.errstate(over="ignore"):
            want = gate / (1 + np.exp(-gate)) * up
        # gate and up: 3 roundings each; silu moves by at most (1 + |gate|) of gate's error; its own
        # exponential, sum and quotient (7 half steps), the product, the output's rounding; below fp32's
        # smallest normal number a step more
        tol = (3 * (1 + np.abs(gate)) + 3 + 7 + 1) * U * np.abs(want) + 2.0 ** -126 * (1 + np.abs(up))
        assert _near(got[rows], want, tol, dtype).all(), e
        seen[rows] = True
    assert (got[~seen] == 9.0).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,H,F,E,k,shared,dropped", EXPERTS)
def test_down(q, dtype, T, H, F, E, k, shared, dropped):
    import torch
    rng = np.random.default_rng(T * 17 + H + F + E)
    idx, w, codes, scales = _case(rng, T, H, F, E, k, shared, dropped)
    h = _rows(rng, T * (k + shared), F, dtype)
    h[:T * k][_t(idx.reshape(-1) < 0)] = float("nan")  # rows of empty slots do not enter
    cfg = q.make_cfg(H, F, E, k, has_shared=shared, wbits=8)
    out = torch.full((T, H), 9.0, dtype=_dt(dtype), device="cuda")
    ws = q.alloc_int8_experts_workspace(cfg, T)
    ws.fill_(0xFF)
    q.int8_down(cfg, q.Weights(_t(codes), _t(scales), None, None), h, _t(idx), _t(w), **_grouped(q, idx, E), out=out, workspace=ws)
    got = _n(out)
    rc, rs = i8ref.quantise(h.float().cpu().numpy())
    want, size = np.zeros((T, H)), np.zeros((T, H))
    for e, rows, tokens in _rows_of(idx, E, shared):
        y = i8ref.dot(rc[rows], codes[e, 2 * F * H:].reshape(H, F)) * rs[rows].astype(np.float64)[:, None] * scales[e, 2 * F:].astype(np.float64)
        if e < E:
            y = y * w.reshape(-1)[rows, None].astype(np.float64)
        np.add.at(want, tokens, y)
        np.add.at(size, tokens, np.abs(y))
    # 3 roundings of a pair's row, a product and an addition for each slot, the output's rounding
    tol = (3 + 1 + k + 1) * U * size
    assert _near(got, want, tol, dtype).all()


@pytest.mark.parametrize("T,k", [(1, 4), (5, 3), (16, 6), (40, 5)])
def test_down_expert_twice_in_a_token(q, T, k):
    """Slots of one token that hold the same expert, and ids out of range, which are empty slots."""
    import torch
    rng = np.random.default_rng(T)
    H, F, E = 384, 512, 64
    _, w, codes, scales = _case(rng, T, H, F, E, k, True, False)
    idx = rng.integers(0, 3 if T < 20 else E, (T, k)).astype(np.int32)
    idx[T // 2, 0] = -1
    idx[0, :2] = idx[0, 1]
    if T > 4:
        idx[4, 2], idx[3, 1] = E, -5
    cfg = q.make_cfg(H, F, E, k, has_shared=True, wbits=8)
    h = _rows(rng, T * (k + 1), F, "float32")
    out, ws = torch.full((T, H), 9.0, device="cuda"), q.alloc_int8_experts_workspace(cfg, T)
    g = _grouped(q, np.where((idx >= 0) & (idx < E), idx, -1), E)
    q.int8_down(cfg, q.Weights(_t(codes), _t(scales), None, None), h, _t(idx), _t(w), **g, out=out, workspace=ws)
    rc, rs = i8ref.quantise(h.cpu().numpy())
    want, size = np.zeros((T, H)), np.zeros((T, H))
    for e, rows, tokens in _rows_of(idx, E, True):
        y = i8ref.dot(rc[rows], codes[e, 2 * F * H:].reshape(H, F)) * rs[rows].astype(np.float64)[:, None] * scales[e, 2 * F:].astype(np.float64)
        if e < E:
            y = y * w.reshape(-1)[rows, None].astype(np.float64)
        np.add.at(want, tokens, y)
        np.add.at(size, tokens, np.abs(y))
    assert (np.abs(_n(out) - want) <= (3 + 1 + k + 1) * U * size + U * np.abs(want)).all()


def test_experts_one_token_as_in_a_batch(q):
    """A token's rows and output do not depend on the tokens beside it, whatever kernel its batch takes."""
    import torch
    rng = np.random.default_rng(5)
    T, H, F, E, k = 300, 512, 384, 8, 3
    idx, w, codes, scales = _case(rng, T, H, F, E, k, True, False)
    cfg = q.make_cfg(H, F, E, k, has_shared=True, wbits=8)
    wt = q.Weights(_t(codes), _t(scales), None, None)
    x = _rows(rng, T, H, "float32")
    ws = q.alloc_int8_experts_workspace(cfg, T)

    def run(a, b):
        n = b - a
        g = _grouped(q, idx[a:b], E)
        h = torch.zeros((n * (k + 1), F), device="cuda")
        out = torch.empty((n, H), device="cuda")
        q.int8_gate_up(cfg, wt, x[a:b].contiguous(), **g, h=h, workspace=ws)
        hd = _rows(np.random.default_rng(1), T * (k + 1), F, "float32")  # down: rows of its own, the same for a token
        hd = torch.cat([hd[a * k:b * k], hd[T * k + a:T * k + b]]).contiguous()
        q.int8_down(cfg, wt, hd, _t(idx[a:b]), _t(w[a:b]), **g, out=out, workspace=ws)
        return h, out

    h, out = run(0, T)
    for a, b in ((0, 1), (7, 9), (100, 140)):
        n = b - a
        h1, out1 = run(a, b)
        assert torch.equal(out1, out[a:b])
        # the few-row kernel's silu and the tiled one's may differ by a few steps
        near = lambda x, y: ((x - y).abs() <= 2.0 ** -20 * y.abs() + 2.0 ** -126).all()  # noqa: E731
        assert near(h1[:n * k], h[a * k:b * k]) and near(h1[n * k:], h[T * k + a:T * k + b])


# T, k, E: one token (gate and up rows in half tiles), few rows, tiles over the route
@pytest.mark.parametrize("T,k,E", [(1, 2, 8), (5, 2, 8), (130, 2, 4)])
def test_gate_up_silu_of_any_gate(q, T, k, E):
    """Gates from -103.5, where silu is among fp32's smallest numbers, to 20: known exactly, since a row has
    one value, so that only silu's own roundings and the product's are left."""
    import torch
    rng = np.random.default_rng(T)
    H, F, up = 128, 1280, 96.0
    want_gate = np.linspace(-103.5, 20.0, F)
    want_gate[-100:] = np.linspace(-44.6, -44.2, 100)
    codes = np.zeros((E + 1, 3 * F * H), np.int8)
    scales = np.ones((E + 1, 2 * F + H), np.float32)
    for e in range(E + 1):
        mine = rng.permutation(want_gate)
        codes[e, :F * H:H] = np.where(mine < 0, -127, 127)
        codes[e, F * H:2 * F * H:H] = 127
        scales[e, :F] = np.abs(mine) / 127
        scales[e, F:2 * F] = up / 127
    x = torch.zeros((T, H), device="cuda")
    x[:, 0] = 1.0  # scale 1 / 127, code 127
    row = np.float32(1.0) / np.float32(127.0)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    cfg = q.make_cfg(H, F, E, k, has_shared=True, wbits=8)
    h = torch.full((T * (k + 1), F), 9.0, device="cuda")
    q.int8_gate_up(cfg, q.Weights(_t(codes), _t(scales), None, None), x, **_grouped(q, idx, E), h=h,
                   workspace=q.alloc_int8_experts_workspace(cfg, T))
    got = _n(h)
    for e, rows, _ in _rows_of(idx, E, True):
        sign = codes[e, :F * H:H].astype(np.float32)
        gate = (sign * 127 * (row * scales[e, :F])).astype(np.float64)  # an fp32 product each, as the kernels have it
        u = np.float64(np.float32(127 * 127) * (row * scales[e, F:2 * F]))
        silu = gate / (1 + np.exp(-gate))
        # relative, half steps U: the hardware's exponential 2 and the sum with its correction 1 (e^-|g|), 1 + e^-|g| 1,
        # its reciprocal 2, two products 2, the product with up 1; the correction's own terms (ln 2 l of 2^-16,
        # rounded, and its square) below 2^-34. Subnormal results: half a step of 2^-149 of silu and of h.
        tol = 9.1 * U * np.abs(silu * u) + 2.0 ** -150 * (np.abs(u) + 1)
        assert (np.abs(got[rows] - silu * u) <= tol).all(), e


@pytest.mark.parametrize("dtype", DT)
def test_gate_up_same_bits_in_every_kernel(q, dtype):
    """A row of h is the same to the bit in the half-tile kernel of one token, the few-row and the tiled one."""
    import torch
    rng = np.random.default_rng(11)
    T, H, F, E, k = 300, 512, 384, 8, 3
    idx, _, codes, scales = _case(rng, T, H, F, E, k, True, False)
    scales[:, :F] *= 6  # gates past -44 and -88 too
    cfg = q.make_cfg(H, F, E, k, has_shared=True, wbits=8)
    wt = q.Weights(_t(codes), _t(scales), None, None)
    x = _rows(rng, T, H, dtype)
    ws = q.alloc_int8_experts_workspace(cfg, T)

    def run(a, b):
        h = torch.zeros(((b - a) * (k + 1), F), dtype=_dt(dtype), device="cuda")
        q.int8_gate_up(cfg, wt, x[a:b].contiguous(), **_grouped(q, idx[a:b], E), h=h, workspace=ws)
        return h

    h = run(0, T)
    for a, b in ((0, 1), (299, 300), (7, 9), (100, 130), (100, 140)):  # one token, few rows (up to 12 pairs an expert), tiles
        n, part = b - a, run(a, b)
        assert torch.equal(part[:n * k], h[a * k:b * k]) and torch.equal(part[n * k:], h[T * k + a:T * k + b]), (a, b)


@pytest.mark.parametrize("H,F", [(128, 7040), (7040, 128)])
def test_experts_offsets_past_31_bits(q, H, F):
    """The most pairs with the widest rows: 131070 rows of 7040 fp32 values are 3.7 GB of h or of the down product's
    rows, near the most that 32-bit offsets reach. Every row as in slices of the batch."""
    import torch
    T, E, k = 65535, 3, 1
    rng = np.random.default_rng(H)
    idx, w, codes, scales = _case(rng, T, H, F, E, k, True, False)
    idx[::7] = -1
    cfg = q.make_cfg(H, F, E, k, has_shared=True, wbits=8)
    wt = q.Weights(_t(codes), _t(scales), None, None)
    g = torch.Generator(device="cuda")
    g.manual_seed(H)
    x = torch.randn((T, H), device="cuda", generator=g)
    hd = torch.randn((2 * T, F), device="cuda", generator=g) if F < H else None
    ids, tw = _t(idx), _t(w)

    def run(a, b):
        n, group = b - a, _grouped(q, idx[a:b], E)
        ws = q.alloc_int8_experts_workspace(cfg, n)
        if hd is None:
            h = torch.full((2 * n, F), 9.0, device="cuda")
            q.int8_gate_up(cfg, wt, x[a:b], **group, h=h, workspace=ws)
            return h[:n], h[n:]
        out = torch.full((n, H), 9.0, device="cuda")
        q.int8_down(cfg, wt, torch.cat([hd[a:b], hd[T + a:T + b]]), ids[a:b], tw[a:b], **group, out=out, workspace=ws)
        return (out,)

    whole = run(0, T)
    for a in range(0, T, 8192):
        b = min(T, a + 8192)
        for i, (part, all_) in enumerate(zip(run(a, b), whole)):
            assert torch.equal(part, all_[a:b]), (i, a)
    assert not any(v.isnan().any() for v in whole)
    if hd is None:
        assert (whole[0][::7] == 9.0).all() and (whole[0][1::7] != 9.0).any(1).all()
