"""The route's gradient against the derivative of every weight in 64 bits, and against differences of
the weights that route_logits gives."""
import numpy as np
import pytest

import i8ref

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


def _back(q, z, idx, g, inplace=False, **kw):
    import torch
    r = q.make_router(z.shape[1], idx.shape[1], **kw)
    dz = z.clone() if inplace else torch.full_like(z, 9.0)
    q.route_logits_backward(r, dz if inplace else z, _t(idx.astype(np.int32)), _t(g.astype(np.float32)), dz)
    return dz


def _near(got, want, dtype, g, scale):
    """fp64 inside (a few steps of 2^-53 times the sizes of at most 1024 terms, far below the output's
    rounding), then one rounding; subnormal results of a type may be off by half their step. The
    definition itself is a difference of two products below scale sum|g| (scores over their sum, and
    1 - score, are at most 1), each with at most 8 roundings of 2^-53: off by 2^-49 of that."""
    import torch
    f = torch.finfo(getattr(torch, dtype))
    own = 2.0 ** -49 * scale * np.nansum(np.abs(g), 1, keepdims=True)
    return np.abs(got - want) <= f.eps / 2 * np.abs(want) * (1 + 2.0 ** -20) + f.tiny * f.eps / 2 + 2.0 ** -40 * np.abs(want).max(1, keepdims=True) + own


CASES = [(1, 1, 1), (1, 256, 8), (5, 8, 8), (61, 64, 8), (33, 60, 6), (9, 200, 3), (130, 512, 4), (7, 1024, 64), (3, 1000, 1)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k", CASES)
def test_formula(q, T, E, k, score, renorm, dtype):
    rng = np.random.default_rng(T + E + k)
    z = _t((2 * rng.standard_normal((T, E))).astype(np.float32), dtype)
    z[0, 0] = 30.0
    idx = np.argsort(-_n(z), 1, kind="stable")[:, :k]
    if E > 4 and T > 2:
        z[1, rng.random(E) < 0.3] = float("-inf")
        z[2] = float("-inf")  # a token without experts
        idx = np.argsort(-_n(z), 1, kind="stable")[:, :k]
        idx[~np.isfinite(np.take_along_axis(_n(z), idx, 1))] = -1
    g = rng.standard_normal((T, k)).astype(np.float32)
    got = _n(_back(q, z, idx, g, score=score, renorm=renorm, scale=2.5))
    want = i8ref.route_grad(_n(z), idx, g.astype(np.float64), score, renorm, 2.5)
    if renorm and k == 1:
        assert (got == 0).all()
    assert _near(got, want, dtype, g, 2.5).all()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_logits_in_place_and_experts_twice(q, score, renorm):
    """dz over z; an expert in two slots gets both slots' gradients; NaN logits are absent experts; the
    weights' gradients of empty slots do not enter."""
    import torch
    rng = np.random.default_rng(0)
    z = rng.standard_normal((6, 40)).astype(np.float32)
    idx = np.argsort(-z, 1)[:, :5]
    idx[1, 3] = idx[1, 0]
    idx[2, 1] = -1
    g = rng.standard_normal((6, 5))
    want = i8ref.route_grad(z, idx, g.astype(np.float32), score, renorm, 1.0)
    g[2, 1] = np.nan
    got = _n(_back(q, _t(z), idx, g, inplace=True, score=score, renorm=renorm))
    assert _near(got, want, "float32", g, 1.0).all()
    worst = np.argmin(z, 1)
    z2 = z.copy()
    z2[np.arange(6), worst] = np.nan
    z3 = z.copy()
    z3[np.arange(6), worst] = -np.inf
    g[2, 1] = 0
    a = _back(q, _t(z2), idx, g, score=score, renorm=renorm)
    assert torch.equal(a, _back(q, _t(z3), idx, g, score=score, renorm=renorm))
    assert (_n(a)[np.arange(6), worst] == 0).all()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_far_logits(q, score, renorm):
    """Scores near 0 and 1, and logits of +inf, which move nothing."""
    z = np.array([[-100.0, -101, -300, 0], [50, 49, 48, 0], [-700, -701, -702, -800], [1e30, 5, 4, 3], [3e38, -3e38, 1, 2]], np.float32)
    idx = np.array([[0, 1, 3], [0, 1, 2], [0, 1, 2], [0, 1, 2], [0, 3, 2]])
    g = np.random.default_rng(0).standard_normal((5, 3)).astype(np.float32)
    got = _n(_back(q, _t(z), idx, g, score=score, renorm=renorm))
    zd = z.astype(np.float64)
    p = i8ref.scores(zd, score)
    pj = np.take_along_axis(p, idx, 1)
    other = np.exp(-np.logaddexp(0, zd)) if score == "sigmoid" else None  # 1 - p without its cancellation
    want = np.zeros_like(zd)
    for t in range(5):
        gj = g[t].astype(np.float64)
        if renorm:
            s = pj[t].sum()
            n = pj[t] / s if s > 0 else 0 * pj[t]
            gj = gj - (gj * n).sum()
            add = gj * n * (other[t, idx[t]] if score == "sigmoid" else 1)
            want[t, idx[t]] += add
        elif score == "sigmoid":
            want[t, idx[t]] += gj * pj[t] * other[t, idx[t]]
        else:
            dp = np.zeros(4)
            dp[idx[t]] = gj
            want[t] = p[t] * (dp - (gj * pj[t]).sum())
    assert (np.abs(got - want) <= 2.0 ** -23 * np.abs(want) + 2.0 ** -149 + 2.0 ** -45 * np.abs(g).max()).all()
    z[0, 0] = z[1, 3] = np.inf
    inf = _n(_back(q, _t(z), idx, g, score=score, renorm=renorm))
    assert np.isfinite(inf).all() and inf[0, 0] == 0
    if score == "softmax":
        assert (inf[:2] == 0).all()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_differences(q, score, renorm):
    """Central differences of route_logits' weights, experts far enough apart that a step leaves the choice."""
    import torch
    rng = np.random.default_rng(2)
    T, E, k, h = 4, 12, 4, 2.0 ** -6
    z = np.stack([rng.permutation(E) * 0.4 - 2 for _ in range(T)]).astype(np.float32)
    g = rng.standard_normal((T, k)).astype(np.float32)
    r = q.make_router(E, k, score=score, renorm=renorm, scale=1.5)
    idx, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")

    def weights(zz):
        q.route_logits(r, _t(zz.astype(np.float32)), idx, w)
        return idx.cpu().numpy().copy(), _n(w)

    at, _ = weights(z)
    dz = _n(_back(q, _t(z), at, g, score=score, renorm=renorm, scale=1.5))
    # a weight's third derivative by a logit is below 1 (times the scale); weights are rounded to fp32
    tol = 1.5 * np.abs(g).sum(1) * (h * h / 6 + 2.0 ** -24 / h)
    for e in range(E):
        up, down = z.copy(), z.copy()
        up[:, e] += h
        down[:, e] -= h
        (iu, wu), (il, wl) = weights(up), weights(down)
        assert np.array_equal(iu, at) and np.array_equal(il, at)
        assert (np.abs(((wu - wl) * g).sum(1) / (2 * h) - dz[:, e]) <= tol).all()


def test_one_taken_expert_of_a_softmax_over_its_sum(q):
    """A weight that is always 1: exactly no gradient."""
    z = np.random.default_rng(1).standard_normal((50, 64)).astype(np.float32)
    for score in ("sigmoid", "softmax"):
        got = _back(q, _t(z), np.argmax(z, 1)[:, None], np.ones((50, 1), np.float32), score=score, renorm=True, scale=2.5)
        assert (got == 0).all()
