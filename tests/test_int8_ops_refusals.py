"""The C entry points of the int8 products, of the pairs' way to their experts and back and of the
route's gradient reject bad calls on the host, before anything is enqueued (CPU only: no call here
reaches a kernel); the binding checks types, shapes and devices; and the 64-bit definitions that the
GPU tests compare against hold against each other."""
import ctypes as C

import numpy as np
import pytest

import i8ref

FAKE = 0x7F0000000000  # never dereferenced: every call below fails validation first
P = C.c_void_p(FAKE)


def at(n):
    return C.c_void_p(FAKE + n)


@pytest.fixture(scope="module")
def q():
    import os
    import quantized_moe_sigmoid_amd as q
    if not os.path.exists(q.LIB_PATH):
        from quantized_moe_sigmoid_amd import build
        build.build()
    return q


def _each(f, good, bad):
    """Every argument of `good` that `bad` names, replaced: the status."""
    for i, v, want in bad:
        args = list(good)
        args[i] = v
        assert f(*args) == want, (i, v)


def test_quantise(q):
    f = q.lib().coli_moe_int8_quantize
    assert f(None, 0, 0, 64, None, None, None) == 0
    _each(f, [P, 0, 4, 64, P, P, None], [
        (0, None, -1), (4, None, -1), (5, None, -1), (1, 3, -1), (1, -1, -1), (2, -1, -1), (3, 0, -1), (3, -16, -1), (3, 40, -2),
        (3, (1 << 17) + 16, -2), (2, 1 << 31, -2), (2, 1 << 40, -2), (0, at(8), -4), (4, at(8), -4), (5, at(2), -4)])


def test_linear(q):
    L = q.lib()
    need = L.coli_moe_int8_linear_workspace_bytes(8, 64, 96)
    assert need > 0 and need % 256 == 0 and L.coli_moe_int8_linear_workspace_bytes(0, 0, 16) > 0
    for bad in ((-1, 64, 96), (8, -1, 96), (8, 64, 0), (8, 64, 72), (8, 64, (1 << 17) + 16), ((1 << 20) + 1, 1, 16),
                (1, (1 << 20) + 1, 16), (1 << 20, 1, 1 << 17), (1, 1 << 20, 1 << 17)):
        assert L.coli_moe_int8_linear_workspace_bytes(*bad) == 0
    f = L.coli_moe_int8_linear
    assert f(None, 0, None, None, None, 0, 64, 96, None, None, 0, None) == 0
    assert f(None, 0, None, None, None, 8, 0, 96, None, None, 0, None) == 0
    _each(f, [P, 0, P, P, None, 8, 64, 96, P, P, need, None], [
        (0, None, -1), (2, None, -1), (3, None, -1), (8, None, -1), (1, 3, -1), (5, -1, -1), (6, -1, -1), (7, 0, -1), (7, 24, -2),
        (9, None, -3), (10, need - 256, -3), (10, 0, -3), (0, at(8), -4), (2, at(8), -4), (3, at(2), -4), (4, at(2), -4),
        (8, at(8), -4), (9, at(16), -4)])


def test_experts(q):
    L = q.lib()
    cfg = q.make_cfg(256, 128, 16, 4, has_shared=True, wbits=8)
    need = L.coli_moe_int8_experts_workspace_bytes(C.byref(cfg), 8)
    assert need > 0 and need % 256 == 0
    assert L.coli_moe_int8_experts_workspace_bytes(C.byref(cfg), 1 << 20) == 0
    assert L.coli_moe_int8_experts_workspace_bytes(None, 8) == 0
    w = q._Weights(P, P, None, None)
    up = [C.byref(cfg), C.byref(w), P, 0, 8, P, P, P, P, P, P, need, None]
    down = [C.byref(cfg), C.byref(w), P, 0, 8, P, P, P, P, P, P, P, P, need, None]
    for kw, want in ((dict(wbits=4), -1), (dict(wbits=8, scale_group=64), -1), (dict(wbits=q.W_MXFP4, scale_group=32), -1),
                     (dict(wbits=3), -1)):
        bad = q.make_cfg(256, 128, 16, 4, has_shared=True, **kw)
        assert L.coli_moe_int8_experts_workspace_bytes(C.byref(bad), 8) == 0
        for f, good in ((L.coli_moe_int8_gate_up, up), (L.coli_moe_int8_down, down)):
            assert f(C.byref(bad), *good[1:]) == want
    no_w = [q._Weights(None, P, None, None), q._Weights(P, None, None, None)]
    for f, good in ((L.coli_moe_int8_gate_up, up), (L.coli_moe_int8_down, down)):
        assert f(*good[:4], 0, *([None] * (len(good) - 7)), 0, None) == 0
        n = len(good)
        ptrs = [2] + list(range(5, n - 3))
        _each(f, good, [(0, None, -1), (1, None, -1), (3, 5, -1), (4, -1, -1), (4, 1 << 20, -2), (1, C.byref(no_w[0]), -1),
                        (1, C.byref(no_w[1]), -1), (n - 3, None, -3), (n - 2, 256, -3), (n - 3, at(128), -4)]
              + [(i, None, -1) for i in ptrs] + [(i, at(2), -4) for i in ptrs])
        _each(f, good, [(2, at(8), -4), (n - 4, at(8), -4), (1, C.byref(q._Weights(at(8), P, None, None)), -4),
                        (1, C.byref(q._Weights(P, at(2), None, None)), -4)])


def test_sort_pairs(q):
    L = q.lib()
    need = L.coli_moe_sort_pairs_workspace_bytes(40000, 64)
    assert need >= 65 * 4 and need % 256 == 0
    assert L.coli_moe_sort_pairs_workspace_bytes(0, 1) > 0
    for bad in ((-1, 64), (1 << 30, 64), (8, 0), (8, 1025), (8, -3)):
        assert L.coli_moe_sort_pairs_workspace_bytes(*bad) == 0
    # enough for a number of pairs: enough for fewer
    sizes = [L.coli_moe_sort_pairs_workspace_bytes(n, 100) for n in (1, 1000, 1024, 1025, 5000, 30000, 32768, 33000, 10 ** 6, 2 ** 30 - 1)]
    assert sizes == sorted(sizes)
    f = L.coli_moe_sort_pairs
    assert f(None, 0, 8, 64, None, None, None, None, None, None, 0, None) == 0
    _each(f, [P, 5000, 8, 64, P, P, P, P, P, P, need, None], [
        (0, None, -1), (1, -1, -1), (2, 0, -1), (3, 0, -1), (1, 1 << 27, -2), (3, 1025, -2), (9, None, -3), (10, 256, -3),
        (9, at(4), -4)] + [(i, None, -1) for i in (4, 5, 6, 7, 8)] + [(i, at(2), -4) for i in (0, 4, 5, 6, 7, 8)])


def test_rows(q):
    L = q.lib()
    f = L.coli_moe_dispatch
    assert f(None, 0, 0, 2, 64, None, 9, None, None) == 0 and f(None, 0, 4, 2, 64, None, 0, None, None) == 0
    _each(f, [P, 1, 4, 2, 64, P, 9, P, None], [
        (0, None, -1), (5, None, -1), (7, None, -1), (1, 9, -1), (2, -1, -1), (3, 0, -1), (4, 0, -1), (6, -1, -1),
        (2, 1 << 29, -2), (6, 1 << 40, -2), (0, at(1), -4), (7, at(1), -4), (5, at(2), -4)])
    assert f(P, 1, 1 << 28, 1, 1 << 13, P, 9, P, None) == -2  # T H
    assert f(at(2), 0, 4, 2, 64, P, 9, P, None) == -4 and f(P, 0, 4, 2, 64, P, 9, at(2), None) == -4
    f = L.coli_moe_combine
    assert f(None, 0, 9, 0, 2, 64, None, None, None, None, None) == 0
    _each(f, [P, 1, 9, 4, 2, 64, P, P, P, P, None], [
        (0, None, -1), (6, None, -1), (9, None, -1), (1, 9, -1), (2, -1, -1), (3, -1, -1), (4, 0, -1), (5, 0, -1),
        (3, 1 << 29, -2), (2, 1 << 40, -2), (0, at(1), -4), (6, at(2), -4), (7, at(2), -4), (8, at(1), -4), (9, at(1), -4)])
    f = L.coli_moe_combine_backward
    assert f(None, None, 0, 9, 0, 2, 64, None, None, None, None, None) == 0
    _each(f, [P, P, 1, 9, 4, 2, 64, P, P, P, P, None], [
        (0, None, -1), (1, None, -1), (7, None, -1), (8, None, -1), (2, 9, -1), (3, -1, -1), (4, -1, -1), (5, 0, -1), (6, 0, -1),
        (4, 1 << 29, -2), (3, 1 << 40, -2), (0, at(1), -4), (1, at(1), -4), (7, at(2), -4), (8, at(2), -4), (9, at(1), -4), (10, at(2), -4)])
    assert f(P, P, 1, 9, 4, 2, 64, P, P, None, None, None) == -1  # nothing wanted


def test_route_gradient(q):
    f = q.lib().coli_moe_route_logits_backward
    r = C.byref(q.make_router(16, 4))
    assert f(r, None, 0, 0, None, None, None, None) == 0
    _each(f, [r, P, 0, 8, P, P, P, None], [
        (0, None, -1), (1, None, -1), (4, None, -1), (5, None, -1), (6, None, -1), (2, 3, -1), (3, -1, -1), (3, 1 << 26, -2),
        (1, at(2), -4), (6, at(2), -4), (4, at(2), -4), (5, at(2), -4)])
    for kw, want in ((dict(n_experts=0, top_k=1), -1), (dict(n_experts=16, top_k=17), -1), (dict(n_experts=2048, top_k=4), -2),
                     (dict(n_experts=1024, top_k=65), -2), (dict(n_experts=16, top_k=4, scale=float("nan")), -1)):
        assert f(C.byref(q.make_router(**kw)), P, 0, 8, P, P, P, None) == want


def test_binding_checks(q):
    """On CPU tensors: types and shapes are looked at before the device, nothing is enqueued."""
    import torch
    f, i = lambda *s: torch.zeros(s), lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    u8, i8 = lambda n: torch.zeros(n, dtype=torch.uint8), lambda *s: torch.zeros(s, dtype=torch.int8)  # noqa: E731
    for call in (lambda: q.int8_quantize(f(2, 32).double(), i8(2, 32), f(2)), lambda: q.dispatch(i(2, 32), i(4), f(4, 32)),
                 lambda: q.combine(f(4, 32), i(4), f(2, 32).double())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: q.int8_quantize(f(2, 32), i8(2, 32), f(2)),  # not on a GPU
                 lambda: q.int8_linear(f(2, 32), i8(8, 32), f(8), f(2, 8), u8(1 << 16)),
                 lambda: q.sort_pairs(i(4, 2), i(17), i(8), i(8), i(16), i(1), u8(1 << 16)),
                 lambda: q.dispatch(f(2, 32), i(4), f(4, 32)), lambda: q.combine(f(4, 32), i(4), f(2, 32)),
                 lambda: q.combine(f(4, 32), i(5), f(2, 32)), lambda: q.dispatch(f(2, 32), i(3), f(4, 32)),  # no whole slots
                 lambda: q.combine_backward(f(2, 32), f(4, 32), i(4), f(2, 2), f(4, 32), f(2, 2)),
                 lambda: q.combine_backward(f(2, 32), None, i(4), f(2, 2), None, f(2, 2)),
                 lambda: q.route_logits_backward(q.make_router(16, 2), f(3, 16), i(3, 2), f(3, 2), f(3, 16))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(q.ColiError):
        q.alloc_int8_linear_workspace(4, 4, 24, "cpu")
    with pytest.raises(q.ColiError):
        q.alloc_sort_pairs_workspace(4, 2000, "cpu")


# ------------------------------------------------------------------ the definitions
def test_definition_of_int8_rows():
    x = np.array([[0, 1, -127, 0.5, -0.5, 126.5, 2.4999], [0, 0, 0, 0, 0, 0, 0], [1, np.inf, 0, 0, 0, 0, 0]], np.float32)
    c, s = i8ref.quantise(x)
    assert c[0].tolist() == [0, 1, -127, 1, -1, 127, 2] and s[0] == 1
    assert not c[1:].any() and s[1] == 0 and np.isnan(s[2])
    rng = np.random.default_rng(0)
    x = rng.standard_normal((20, 500)).astype(np.float32)
    c, s = i8ref.quantise(x)
    # half a step and the two divisions' roundings
    assert (np.abs(c * s[:, None].astype(np.float64) - x) <= s[:, None] * (0.5 + 127 * 2.0 ** -22)).all()
    assert (np.abs(c).max(1) == 127).all()


def test_definition_of_the_route_gradient():
    """The derivative of every weight against differences of the weights, in 64 bits."""
    rng = np.random.default_rng(1)
    z = rng.standard_normal((6, 10))
    z[3, 4] = -np.inf
    idx = np.argsort(-z, 1)[:, :4]
    idx[2, 2] = -1
    g = rng.standard_normal((6, 4))
    for kind in ("sigmoid", "softmax"):
        for renorm in (True, False):
            dz = i8ref.route_grad(z, idx, g, kind, renorm, 2.5)
            for e in range(10):
                h = 2.0 ** -12
                up, down = z.copy(), z.copy()
                up[:, e] += h
                down[:, e] -= h
                d = (i8ref.weights(up, idx, kind, renorm, 2.5) - i8ref.weights(down, idx, kind, renorm, 2.5)) / (2 * h)
                want = (np.where(idx >= 0, g, 0) * d).sum(1)
                assert np.abs(want - dz[:, e]).max() < 1e-6  # h^2 / 6 of third derivatives below 1, times 2.5 sum|g|


def test_definition_of_sorted_pairs():
    off, perm, pos, active = i8ref.sort_pairs(np.array([[2, 0], [-1, 2], [0, 5]]), 4)
    assert off.tolist() == [0, 2, 2, 4, 4] and perm.tolist() == [1, 4, 0, 3]
    assert pos.tolist() == [2, 0, -1, 3, 1, -1] and active.tolist() == [0, 2]


@pytest.mark.parametrize("shape", [dict(hidden=7168, ffn=128), dict(hidden=128, ffn=7168)])
def test_experts_widths_that_offsets_rest_on(q, shape):
    """Rows wider than 7040 are refused: 131070 of 7040 fp32 values are what the kernels' 32-bit offsets reach."""
    need = lambda c: q.lib().coli_moe_int8_experts_workspace_bytes(C.byref(c), 65535)  # noqa: E731
    assert need(q.make_cfg(n_experts=3, top_k=1, has_shared=True, wbits=8, **shape)) == 0
    assert need(q.make_cfg(n_experts=3, top_k=1, has_shared=True, wbits=8, **{n: v - 128 if v > 128 else v for n, v in shape.items()})) > 0
