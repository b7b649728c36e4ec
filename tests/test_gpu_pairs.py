"""Pairs sorted by expert, tokens' rows laid out in that order and summed back, and the gradients,
against their definitions in 64 bits: whole numbers and copies exactly, sums within the roundings of
fp32 sums in slot order (or exactly, on whole numbers) and one rounding of the output."""
import numpy as np
import pytest

import i8ref

pytestmark = pytest.mark.gpu

DT = ["float32", "bfloat16", "float16"]
U = 2.0 ** -24


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
    import torch
    f = torch.finfo(_dt(dtype))
    return f.tiny * f.eps / 2


def _sort(q, idx, E, pairs_max=None):
    import torch
    T, k = idx.shape
    new = lambda n: torch.full((n,), -77, dtype=torch.int32, device="cuda")  # noqa: E731
    o = dict(off=new(E + 1), perm=new(T * k), pos=new(T * k), active=new(E), n_active=new(1))
    ws = q.alloc_sort_pairs_workspace(pairs_max or T * k, E)
    ws.fill_(0xFF)
    q.sort_pairs(_t(idx.astype(np.int32)), **o, workspace=ws)
    return {n: t.cpu().numpy() for n, t in o.items()}


SORTS = [(1, 1, 1), (1, 8, 256), (3, 5, 7), (16, 8, 256), (127, 8, 64), (128, 8, 64), (129, 8, 64), (257, 4, 1024), (1023, 1, 3),
         (1025, 1, 1000), (2048, 8, 256), (8191, 8, 60), (5000, 6, 1), (40000, 8, 64), (300001, 1, 1024)]


@pytest.mark.parametrize("dropped", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("T,k,E", SORTS)
def test_sort_pairs(q, T, k, E, dropped):
    rng = np.random.default_rng(T * 11 + k + E)
    idx = (E * rng.random((T, k)) ** 2).astype(np.int32)  # unevenly; an expert may be there twice in a token
    idx[rng.random((T, k)) < dropped] = -1
    o = _sort(q, idx, E, pairs_max=None if T % 2 else 3 * T * k)
    off, perm, pos, active = i8ref.sort_pairs(idx, E)
    assert np.array_equal(o["off"], off) and np.array_equal(o["pos"], pos)
    assert np.array_equal(o["perm"][:perm.size], perm) and (o["perm"][perm.size:] == -77).all()
    assert o["n_active"][0] == active.size
    assert np.array_equal(o["active"][:active.size], active) and (o["active"][active.size:] == -77).all()


@pytest.mark.parametrize("T,k,E", [(16, 8, 256), (2000, 8, 64), (8191, 8, 256)])
def test_sort_pairs_is_group_with_places(q, T, k, E):
    import torch
    rng = np.random.default_rng(T)
    idx = rng.integers(-1, E, (T, k)).astype(np.int32)
    o = _sort(q, idx, E)
    new = lambda n: torch.full((n,), -77, dtype=torch.int32, device="cuda")  # noqa: E731
    g = dict(cnt=new(E), off=new(E + 1), perm=new(T * k), active=new(E), n_active=new(1))
    q.group(q.make_cfg(256, 128, E, k), _t(idx), T, **g)
    for n in ("off", "perm", "active", "n_active"):
        assert np.array_equal(o[n], g[n].cpu().numpy()), n


@pytest.mark.parametrize("where", [0, 700, 4999])
@pytest.mark.parametrize("bad", [-2, 64, 2 ** 31 - 1, -2 ** 31])
def test_sort_pairs_bad_ids(q, where, bad):
    """Ids out of range are counted nowhere and n_active says so."""
    for T in (5000, 900):
        idx = np.random.default_rng(1).integers(0, 64, (T, 1)).astype(np.int32)
        idx[where % T] = bad
        o = _sort(q, idx, 64)
        off, perm, pos, active = i8ref.sort_pairs(idx, 64)
        assert o["n_active"][0] == -1
        assert np.array_equal(o["off"], off) and np.array_equal(o["pos"], pos)
        assert np.array_equal(o["perm"][:perm.size], perm)


ROWS = [(1, 1, 1), (1, 8, 6144), (3, 2, 3), (16, 8, 2048), (17, 5, 100), (50, 3, 77), (7, 64, 40), (400, 4, 520), (1000, 8, 8)]


def _route(rng, T, k, dropped=0.2, spare=0):
    """Places of T k pairs in random order among T k + spare rows, some of them empty."""
    pos = rng.permutation(T * k + spare)[:T * k].astype(np.int32)
    pos[rng.random(T * k) < dropped] = -1
    return pos


def _off(t, by):
    """The same values at an address `by` elements past an aligned one."""
    import torch
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    buf[by:] = t.reshape(-1)
    return buf[by:].view(t.shape)


@pytest.mark.parametrize("by", [0, 1])
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,k,H", ROWS)
def test_dispatch(q, dtype, T, k, H, by):
    import torch
    rng = np.random.default_rng(T + k + H)
    pos = _route(rng, T, k, spare=5)
    if T * k > 4:
        pos[0], pos[3] = T * k + 5, 2 ** 31 - 1  # out of range: empty slots
    x = _t(rng.standard_normal((T, H)).astype(np.float32), dtype)
    x[0, 0] = float("nan")
    rows = _off(torch.full((T * k + 5, H), 3.0, dtype=_dt(dtype), device="cuda"), by)
    q.dispatch(_off(x, by), _t(pos), rows)
    want = np.full((T * k + 5, H), 3.0)
    ok = (pos >= 0) & (pos < T * k + 5)
    want[pos[ok]] = _n(x)[np.nonzero(ok)[0] // k]
    assert np.array_equal(_n(rows), want, equal_nan=True)


def _combine64(ys, pos, w, add, T, k):
    ok = (pos >= 0) & (pos < ys.shape[0])
    y = np.where(ok[:, None], ys[np.where(ok, pos, 0)], 0).reshape(T, k, -1)
    terms = y if w is None else y * np.where(ok.reshape(T, k), w, 0)[..., None]
    out, size = terms.sum(1), np.abs(terms).sum(1)
    return (out, size) if add is None else (out + add, size + np.abs(add))


@pytest.mark.parametrize("by", [0, 1])
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("weights,extra", [(True, True), (True, False), (False, False), (False, True)])
@pytest.mark.parametrize("T,k,H", ROWS)
def test_combine(q, dtype, T, k, H, weights, extra, by):
    import torch
    rng = np.random.default_rng(T + k + H)
    pos = _route(rng, T, k, spare=3)
    if T * k > 4:
        pos[1], pos[:k] = T * k + 3, -1  # a token of empty slots, and a place out of range
    ys = _t(rng.standard_normal((T * k + 3, H)).astype(np.float32), dtype)
    used = np.zeros(T * k + 3, bool)
    used[pos[(pos >= 0) & (pos < T * k + 3)]] = True
    ys[_t(~used)] = float("nan")  # rows that no pair has
    w = rng.standard_normal((T, k)).astype(np.float32)
    w[(pos < 0).reshape(T, k)] = np.nan  # weights of empty slots
    add = _t(rng.standard_normal((T, H)).astype(np.float32), dtype) if extra else None
    out = _off(torch.full((T, H), 3.0, dtype=_dt(dtype), device="cuda"), by)
    q.combine(_off(ys, by), _t(pos), out, topk_w=_t(w) if weights else None, add=None if add is None else _off(add, by))
    want, size = _combine64(_n(ys), pos, w if weights else None, None if add is None else _n(add), T, k)
    tol = (k + 2) * U * size  # a rounding for each slot and for the row added, in any order
    assert (np.abs(_n(out) - want) <= tol + _half(dtype) * (np.abs(want) + tol) + _tiny(dtype)).all()


@pytest.mark.parametrize("by", [0, 1])
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,k,H", ROWS)
def test_combine_backward(q, dtype, T, k, H, by):
    import torch
    rng = np.random.default_rng(T + k + H)
    pos = _route(rng, T, k, spare=3)
    if T * k > 4:
        pos[2] = T * k + 3
    ok = (pos >= 0) & (pos < T * k + 3)
    ys = _t(rng.standard_normal((T * k + 3, H)).astype(np.float32), dtype)
    dout = _t(rng.standard_normal((T, H)).astype(np.float32), dtype)
    w = rng.standard_normal((T, k)).astype(np.float32)
    w.reshape(-1)[~ok] = np.nan
    new = lambda: _off(torch.full((T * k + 3, H), 3.0, dtype=_dt(dtype), device="cuda"), by)  # noqa: E731
    dys, dw = new(), torch.full((T, k), 7.0, device="cuda")
    q.combine_backward(_off(dout, by), _off(ys, by), _t(pos), _t(w), dys, dw)
    g = _n(dout)[np.arange(T * k) // k]
    want = np.full((T * k + 3, H), 3.0)
    want[pos[ok]] = (g * w.reshape(-1, 1))[ok]
    # the product in fp32, then the type's rounding
    assert (np.abs(_n(dys) - want) <= (U + _half(dtype) * (1 + U)) * np.abs(want) + _tiny(dtype)).all()
    terms = g[ok] * _n(ys)[pos[ok]]
    got = _n(dw).reshape(-1)
    # H terms in fp32, in any order: at most H - 1 additions and a product deep
    assert (np.abs(got[ok] - terms.sum(1)) <= H * U * np.abs(terms).sum(1)).all()
    assert (got[~ok] == 0).all()
    # either alone
    only, dw2 = new(), torch.full((T, k), 7.0, device="cuda")
    q.combine_backward(_off(dout, by), None, _t(pos), _t(w), only)
    q.combine_backward(_off(dout, by), _off(ys, by), _t(pos), _t(w), None, dw2)
    assert torch.equal(only, dys) and torch.equal(dw2, dw)


@pytest.mark.parametrize("dtype", DT)
def test_gradients_by_differences(q, dtype):
    """On small whole numbers every sum is exact, and combine and dispatch are linear: a step's difference
    is the gradient, exactly."""
    import torch
    rng = np.random.default_rng(3)
    T, k, H = 6, 3, 24
    pos = _t(_route(rng, T, k))
    ints = lambda *s: _t(rng.integers(-3, 4, s).astype(np.float32), dtype)  # noqa: E731
    ys, dout, x, drows = ints(T * k, H), ints(T, H), ints(T, H), ints(T * k, H)
    w = _t(rng.integers(-3, 4, (T, k)).astype(np.float32))

    def loss(y, wt):
        out = torch.empty((T, H), dtype=y.dtype, device="cuda")
        q.combine(y, pos, out, topk_w=wt)
        return float((out.double() * dout.double()).sum())

    dys, dw = torch.zeros_like(ys), torch.empty_like(w)
    q.combine_backward(dout, ys, pos, w, dys, dw)
    base = loss(ys, w)
    for i in range(T * k):
        u = w.clone()
        u.view(-1)[i] += 1
        assert loss(ys, u) - base == float(dw.view(-1)[i])
        v = ys.clone()
        v[i, i % H] += 1
        assert loss(v, w) - base == float(dys[i, i % H])

    def laid(a):
        rows = torch.zeros((T * k, H), dtype=a.dtype, device="cuda")
        q.dispatch(a, pos, rows)
        return float((rows.double() * drows.double()).sum())

    dx = torch.empty_like(x)
    q.combine(drows, pos, dx)  # the gradient of dispatch
    base = laid(x)
    for i in range(T):
        v = x.clone()
        v[i, 3 * i] += 1
        assert laid(v) - base == float(dx[i, 3 * i])


def test_no_rows_and_no_tokens(q):
    """Nothing to read: combine gives what is added, and calls of no tokens write nothing."""
    import torch
    pos = torch.zeros(8, dtype=torch.int32, device="cuda")
    none, add = torch.empty((0, 16), device="cuda"), torch.arange(32.0, device="cuda").view(2, 16)
    out, w = torch.full((2, 16), 5.0, device="cuda"), torch.ones((2, 4), device="cuda")
    q.combine(none, pos, out, topk_w=w, add=add)
    assert torch.equal(out, add)
    q.combine(none, pos, out)
    assert (out == 0).all()
    dw = torch.full((2, 4), 5.0, device="cuda")
    q.combine_backward(add, none, pos, w, None, dw)
    assert (dw == 0).all()
    q.dispatch(add, pos, none)
    rows = torch.full((4, 16), 5.0, device="cuda")
    q.dispatch(torch.empty((0, 16), device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), rows)
    q.combine(rows, torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty((0, 16), device="cuda"))
    assert (rows == 5).all()


def test_rows_past_32_bits(q):
    """A row buffer whose last rows start past 2^32 bytes and 2^31 elements."""
    import torch
    H, R, T, k = 8192, 300000, 3, 2
    rows = torch.zeros((R, H), dtype=torch.bfloat16, device="cuda")
    pos = _t(np.array([R - 1, 0, 262143, 262144, R - 2, 5], np.int32))
    x = _t(np.random.default_rng(0).standard_normal((T, H)).astype(np.float32), "bfloat16")
    q.dispatch(x, pos, rows)
    assert torch.equal(rows[pos.long()], x.repeat_interleave(k, 0))
    assert int((rows != 0).any(1).sum()) == 6
    out, w = torch.empty_like(x), torch.full((T, k), 0.5, device="cuda")
    q.combine(rows, pos, out, topk_w=w)
    assert torch.equal(out, x)
    dys = rows
    dw = torch.empty((T, k), device="cuda")
    q.combine_backward(out, rows, pos, w, None, dw)
    assert torch.allclose(dw, (x.float() ** 2).sum(1, keepdim=True).expand(T, k), rtol=H * U, atol=0)
    q.combine_backward(out, None, pos, w, dys)
    assert torch.equal(rows[pos.long()], (x / 2).repeat_interleave(k, 0))


def test_more_elements_than_one_launch(q):
    """Rows of no whole pieces with more than 2^32 elements, and more pairs than a launch has wavefronts for."""
    import torch
    T, H = 131073, 32769
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(0)
    at = [0, 65535, 65536, T - 2, T - 1]
    for i in at:
        x[i] = _t(rng.standard_normal(H).astype(np.float32), "bfloat16")
    pos = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    pos[at] = torch.arange(len(at), dtype=torch.int32, device="cuda").flip(0)
    rows = torch.full((len(at) + 1, H), 3.0, dtype=torch.bfloat16, device="cuda")
    q.dispatch(x, pos, rows)
    assert torch.equal(rows[:-1], x[at].flip(0)) and (rows[-1] == 3).all()
    out = torch.full_like(x, 3.0)
    q.combine(rows, pos, out)
    assert torch.equal(out, x)
    del x, out
    P = 4 * (1 << 23) + 5
    pos = torch.arange(P, dtype=torch.int32, device="cuda").flip(0).contiguous()
    y, w = torch.randn((P, 1), device="cuda"), torch.randn((P, 1), device="cuda")
    dout, dy, dw = torch.randn((P, 1), device="cuda"), torch.empty((P, 1), device="cuda"), torch.empty((P, 1), device="cuda")
    q.combine_backward(dout, y, pos, w, dy, dw)
    assert torch.equal(dw, dout * y.flip(0)) and torch.equal(dy.flip(0), dout * w)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("H", [1, 2, 3, 4, 5, 7, 8, 9, 15, 17, 31, 510, 511, 513, 2047, 4646])
def test_rows_of_no_whole_pieces(q, dtype, H):
    """Row ends beside rows of NaN and guards: each element once, nothing outside. combine adds to out itself."""
    import torch
    T, k = 37, 3
    rng = np.random.default_rng(H)
    pos = (rng.permutation(T * k) * 2 + 1).astype(np.int32)  # every other row
    pos[rng.random(T * k) < 0.2] = -1
    ok = pos >= 0
    R = 2 * T * k + 1
    x = _t(rng.standard_normal((T, H)).astype(np.float32), dtype)
    fenced = lambda n: torch.full((n * H + 16,), 3.0, dtype=_dt(dtype), device="cuda")  # noqa: E731
    inside = lambda b, n: b[8:8 + n * H].view(n, H)  # noqa: E731
    kept = lambda b, n: (b[:8] == 3).all() and (b[8 + n * H:] == 3).all()  # noqa: E731
    rb = fenced(R)
    rows = inside(rb, R)
    q.dispatch(x, _t(pos), rows)
    want = torch.full_like(rows, 3.0)
    want[_t(pos[ok]).long()] = x[_t(np.arange(T * k)[ok] // k)]
    assert torch.equal(rows, want) and kept(rb, R)
    ys = torch.full_like(rows, float("nan"))
    ys[_t(pos[ok]).long()] = _t(rng.standard_normal((int(ok.sum()), H)).astype(np.float32), dtype)
    w = rng.standard_normal((T, k)).astype(np.float32)
    ob = fenced(T)
    out = inside(ob, T)
    out.copy_(x)
    q.combine(ys, _t(pos), out, topk_w=_t(w), add=out)
    want, size = _combine64(_n(ys), pos, w, _n(x), T, k)
    tol = (k + 2) * U * size
    assert (np.abs(_n(out) - want) <= tol + _half(dtype) * (np.abs(want) + tol) + _tiny(dtype)).all() and kept(ob, T)
    db = fenced(R)
    dys, dw = inside(db, R), torch.full((T, k), 7.0, device="cuda")
    q.combine_backward(x, ys, _t(pos), _t(w), dys, dw)
    g = _n(x)[np.arange(T * k) // k]
    want = np.full((R, H), 3.0)
    want[pos[ok]] = (g * w.reshape(-1, 1))[ok]
    assert (np.abs(_n(dys) - want) <= (U + _half(dtype) * (1 + U)) * np.abs(want) + _tiny(dtype)).all() and kept(db, R)
    terms = g[ok] * _n(ys)[pos[ok]]
    got = _n(dw).reshape(-1)
    assert (np.abs(got[ok] - terms.sum(1)) <= H * U * np.abs(terms).sum(1)).all() and (got[~ok] == 0).all()
