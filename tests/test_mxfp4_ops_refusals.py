"""The C entry points of the route from logits and of the MXFP4 operators reject bad calls on
the host, before anything is enqueued (CPU only: no call here reaches a kernel); and the 64-bit
definitions that the GPU tests compare against hold against each other."""
import ctypes as C

import numpy as np
import pytest

import mxref

FAKE = 0x7F0000000000  # never dereferenced: every call below fails validation first
P = C.c_void_p(FAKE)
ODD = C.c_void_p(FAKE + 2)


@pytest.fixture(scope="module")
def q():
    import os
    import quantized_moe_sigmoid_amd as q
    if not os.path.exists(q.LIB_PATH):
        from quantized_moe_sigmoid_amd import build
        build.build()
    return q


BAD_ROUTERS = [
    (dict(n_experts=0, top_k=1), -1), (dict(n_experts=16, top_k=0), -1), (dict(n_experts=16, top_k=17), -1),
    (dict(n_experts=16, top_k=4, n_group=3), -1), (dict(n_experts=16, top_k=4, n_group=2, topk_group=3), -1),
    (dict(n_experts=16, top_k=9, n_group=2, topk_group=1), -1), (dict(n_experts=16, top_k=4, group_top=3), -1),
    (dict(n_experts=16, top_k=4, group_top=0), -1), (dict(n_experts=16, top_k=4, scale=float("nan")), -1),
    (dict(n_experts=2048, top_k=4), -2), (dict(n_experts=1024, top_k=65), -2), (dict(n_experts=256, top_k=4, n_group=128, topk_group=4), -2),
]


@pytest.mark.parametrize("kw,want", BAD_ROUTERS)
def test_bad_router(q, kw, want):
    r = q.make_router(**kw)
    assert q.lib().coli_moe_route_logits(C.byref(r), P, 0, 8, None, P, P, None) == want


def test_route_logits_arguments(q):
    f = q.lib().coli_moe_route_logits
    r = C.byref(q.make_router(16, 4))
    assert f(r, None, 0, 0, None, None, None, None) == 0
    assert f(None, P, 0, 8, None, P, P, None) == -1
    assert f(r, P, 3, 8, None, P, P, None) == -1
    assert f(r, P, 0, -1, None, P, P, None) == -1
    for args in ((None, 0, 8, None, P, P), (P, 0, 8, None, None, P), (P, 0, 8, None, P, None)):
        assert f(r, *args, None) == -1
    for args in ((ODD, 0, 8, None, P, P), (C.c_void_p(FAKE + 1), 1, 8, None, P, P), (P, 0, 8, ODD, P, P),
                 (P, 0, 8, None, ODD, P), (P, 0, 8, None, P, ODD)):
        assert f(r, *args, None) == -4
    bad = q.make_router(16, 4)
    bad.score = 2
    assert f(C.byref(bad), P, 0, 8, None, P, P, None) == -1


def test_quantise_arguments(q):
    L = q.lib()
    assert L.coli_moe_mxfp4_quantize(None, 0, 0, 64, None, None, None) == 0
    assert L.coli_moe_mxfp4_quantize(P, 0, 4, 48, P, P, None) == -2
    assert L.coli_moe_mxfp4_quantize(P, 0, 1 << 40, 64, P, P, None) == -2
    assert L.coli_moe_mxfp4_quantize(P, 0, -1, 64, P, P, None) == -1
    assert L.coli_moe_mxfp4_quantize(P, 0, 4, 0, P, P, None) == -1
    assert L.coli_moe_mxfp4_quantize(P, 7, 4, 64, P, P, None) == -1
    assert L.coli_moe_mxfp4_quantize(P, 0, 4, 64, None, P, None) == -1
    assert L.coli_moe_mxfp4_quantize(C.c_void_p(FAKE + 8), 0, 4, 64, P, P, None) == -4
    assert L.coli_moe_mxfp4_quantize(P, 0, 4, 64, C.c_void_p(FAKE + 8), P, None) == -4
    assert L.coli_moe_mxfp4_dequantize(P, P, 4, 48, P, 0, None) == -2
    assert L.coli_moe_mxfp4_dequantize(P, P, 4, 64, None, 0, None) == -1
    assert L.coli_moe_mxfp4_dequantize(P, P, 4, 64, C.c_void_p(FAKE + 4), 0, None) == -4
    assert L.coli_moe_mxfp4_dequantize(P, P, 4, 64, P, -1, None) == -1


def test_linear_arguments(q):
    L = q.lib()
    need = L.coli_moe_mxfp4_linear_workspace_bytes(8, 64, 96)
    assert need > 0 and need % 256 == 0
    for bad in ((-1, 64, 96), (8, -1, 96), (8, 64, 0), (8, 64, 80)):
        assert L.coli_moe_mxfp4_linear_workspace_bytes(*bad) == 0
    sizes = [L.coli_moe_mxfp4_linear_workspace_bytes(M, 200, 416) for M in range(1, 600)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))

    def f(x=P, d=0, c=P, s=P, M=8, N=64, K=96, y=P, ws=P, n=need):
        return L.coli_moe_mxfp4_linear(x, d, c, s, M, N, K, y, ws, n, None)

    assert f(M=0, x=None, ws=None) == 0 and f(N=0, c=None) == 0
    assert f(M=-1) == -1 and f(N=-1) == -1 and f(K=0) == -1 and f(d=3) == -1
    assert f(K=80) == -2 and f(K=1 << 21, n=1 << 60) == -2 and f(M=1 << 21, n=1 << 60) == -2
    assert f(x=None) == -1 and f(c=None) == -1 and f(s=None) == -1 and f(y=None) == -1
    assert f(x=ODD) == -4 and f(c=ODD) == -4 and f(y=ODD) == -4 and f(ws=C.c_void_p(FAKE + 64)) == -4
    assert f(ws=None) == -3 and f(n=need - 1) == -3


def test_experts_arguments(q):
    L = q.lib()
    cfg = q.make_cfg(256, 128, 16, 4, has_shared=True, wbits=q.W_MXFP4, scale_group=32)
    need = L.coli_moe_mxfp4_experts_workspace_bytes(C.byref(cfg), 8)
    assert need > 0
    sizes = [L.coli_moe_mxfp4_experts_workspace_bytes(C.byref(cfg), T) for T in range(1, 2000, 3)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    w = q._Weights(P, P, None, None)

    def gu(c=cfg, w=w, x=P, d=0, T=8, g=(P, P, P, P), h=P, ws=P, n=need):
        return L.coli_moe_mxfp4_gate_up(None if c is None else C.byref(c), C.byref(w), x, d, T, *g, h, ws, n, None)

    def dn(c=cfg, w=w, h=P, d=0, T=8, r=(P, P), g=(P, P, P, P), out=P, ws=P, n=need):
        return L.coli_moe_mxfp4_down(None if c is None else C.byref(c), C.byref(w), h, d, T, *r, *g, out, ws, n, None)

    for f in (gu, dn):
        assert f(T=0, ws=None) == 0
        assert f(c=None) == -1 and f(d=9) == -1 and f(T=-1) == -1 and f(T=20000) == -2
        assert f(c=q.make_cfg(256, 128, 16, 4, wbits=4)) == -1  # not MXFP4
        assert f(c=q.make_cfg(160, 128, 16, 4, wbits=q.W_MXFP4, scale_group=32)) == -2
        assert f(w=q._Weights(None, P, None, None)) == -1 and f(w=q._Weights(P, ODD, None, None)) == -4
        assert f(ws=None) == -3 and f(n=255) == -3 and f(ws=C.c_void_p(FAKE + 128)) == -4
        for i in range(4):
            assert f(g=tuple(None if j == i else P for j in range(4))) == -1
            assert f(g=tuple(ODD if j == i else P for j in range(4))) == -4
    assert gu(x=None) == -1 and gu(h=None) == -1 and gu(x=ODD) == -4 and gu(h=ODD) == -4
    assert dn(h=None) == -1 and dn(out=None) == -1 and dn(h=ODD) == -4 and dn(out=ODD) == -4
    assert dn(r=(None, P)) == -1 and dn(r=(P, ODD)) == -4
    assert L.coli_moe_mxfp4_experts_workspace_bytes(C.byref(q.make_cfg(256, 128, 16, 4)), 8) == 0
    assert L.coli_moe_mxfp4_experts_workspace_bytes(C.byref(cfg), 20000) == 0


def test_definition_of_quantisation():
    """No grid value lies closer than the one chosen, and a block already on its grid is kept."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((20, 64)) * np.exp2(rng.integers(-20, 20, (20, 1)))
    c, s = mxref.quantise(x)
    v = mxref.unpack(c, s)
    grid = np.unique(mxref.E2M1)[None, :] * mxref.e8m0(s).repeat(32, 1).reshape(-1, 1)
    best = np.abs(grid - x.reshape(-1, 1)).min(1)
    assert np.array_equal(np.abs(v - x).reshape(-1), best)
    c2, s2 = mxref.quantise(v)
    assert np.array_equal(mxref.unpack(c2, s2), v)


def test_definition_of_route_against_sort():
    """Without groups the route is a stable descending sort of the keys."""
    rng = np.random.default_rng(2)
    z = rng.integers(-4, 5, (30, 24)).astype(float)
    idx, w = mxref.route(z, 5)
    assert np.array_equal(idx, np.argsort(-z, axis=1, kind="stable")[:, :5])
    assert np.allclose(w.sum(1), 1)


def test_sizes_beyond_one_launch(q):
    """Products and conversions whose blocks of 32 pass what one launch counts are refused, not truncated."""
    L = q.lib()
    assert L.coli_moe_mxfp4_quantize(P, 0, 1 << 31, 32, P, P, None) == -2
    assert L.coli_moe_mxfp4_dequantize(P, P, (1 << 31) - 127, 32, P, 1, None) == -2
    assert L.coli_moe_mxfp4_linear_workspace_bytes(1 << 20, 16, 1 << 20) == 0
    assert L.coli_moe_mxfp4_linear_workspace_bytes(16, 1 << 20, 1 << 20) == 0
    assert L.coli_moe_mxfp4_linear(P, 0, P, P, 1 << 20, 16, 1 << 20, P, P, 1 << 62, None) == -2
    assert L.coli_moe_mxfp4_linear_workspace_bytes(1 << 20, 16, 1 << 15) > 0
    r = C.byref(q.make_router(8, 2))
    assert L.coli_moe_route_logits(r, P, 0, (1 << 26) - 3, None, P, P, None) == -2
