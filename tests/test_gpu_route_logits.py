"""The route from logits against its definition, one token at a time in 64 bits: ids exactly,
weights to one rounding of fp32; scores, groups, bias, masked experts, ties, every slot count."""
import numpy as np
import pytest

import mxref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_moe_sigmoid_amd as q
    q.lib()
    return q


def _run(q, z, k, dtype="float32", bias=None, **kw):
    import torch
    T, E = z.shape
    zt = torch.from_numpy(np.ascontiguousarray(z, np.float32)).cuda().to(getattr(torch, dtype))
    bt = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
    idx = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    names = dict(G="n_group", Gk="topk_group")
    q.route_logits(q.make_router(E, k, **{names.get(a, a): v for a, v in kw.items()}), zt, idx, w, bias=bt)
    ri, rw = mxref.route(zt.double().cpu().numpy(), k, bias=None if bias is None else np.asarray(bias, np.float32), **kw)
    assert np.array_equal(idx.cpu().numpy(), ri)
    # fp64 exp, sum and division are within a few 2^-52, then one rounding to fp32
    assert (np.abs(w.cpu().double().numpy() - rw) <= np.abs(rw) * 2.0 ** -24 * (1 + 2.0 ** -20) + 2.0 ** -149).all()


SHAPES = [  # T, E, k, G, Gk
    (1, 256, 8, 8, 4), (5, 8, 1, 1, 1), (9, 8, 8, 1, 1), (37, 64, 8, 1, 1), (64, 60, 4, 1, 1), (33, 60, 6, 4, 2),
    (50, 160, 6, 8, 3), (129, 256, 8, 8, 4), (20, 256, 8, 1, 1), (17, 120, 7, 2, 1), (13, 24, 5, 8, 3), (11, 40, 3, 8, 8),
    (10, 64, 8, 64, 16), (7, 512, 16, 16, 4), (6, 1024, 64, 32, 8), (8, 320, 33, 1, 1), (3, 1, 1, 1, 1), (65, 248, 8, 4, 1),
]


@pytest.mark.parametrize("T,E,k,G,Gk", SHAPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("group_top", [1, 2])
def test_route(q, T, E, k, G, Gk, score, with_bias, group_top):
    rng = np.random.default_rng(T * E + k)
    z = 1.5 * rng.standard_normal((T, E))
    z[rng.random((T, E)) < 0.1] = -np.inf
    z[rng.random(T) < 0.1] = -np.inf  # tokens with no expert
    bias = 0.05 * rng.standard_normal(E) if with_bias else None
    for renorm, scale in ((True, 2.5), (False, 1.0)):
        _run(q, z, k, bias=bias, G=G, Gk=Gk, score=score, group_top=group_top, renorm=renorm, scale=scale)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,G,Gk", [(300, 256, 8, 8, 4), (301, 64, 8, 1, 1), (111, 60, 4, 2, 1), (200, 128, 8, 8, 4)])
def test_route_16bit_logits(q, T, E, k, G, Gk, score, dtype):
    """16-bit logits tie often: the lower index wins, among experts and among groups."""
    z = 1.5 * np.random.default_rng(E).standard_normal((T, E))
    _run(q, z, k, dtype, G=G, Gk=Gk, score=score)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,G,Gk", [(256, 8, 8, 4), (64, 8, 1, 1), (60, 8, 4, 2)])
def test_route_ties(q, E, k, G, Gk, score):
    """Rows of one value, of few values, of -0 and 0, of the type's lowest value."""
    rng = np.random.default_rng(E)
    rows = [np.zeros(E), np.full(E, -3.0), np.where(rng.random(E) < 0.5, 0.0, -0.0), np.full(E, np.finfo(np.float32).min)]
    rows += [rng.integers(0, 3, E).astype(float) for _ in range(40)]
    z = np.stack(rows)
    _run(q, z, k, G=G, Gk=Gk, score=score)
    _run(q, z, k, bias=np.zeros(E), G=G, Gk=Gk, score=score)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_route_special_values(q, score, group_top):
    """NaN and -inf take an expert away, +inf takes everything of a softmax, huge values do not
    overflow; fewer experts left than slots; a bias of -inf or NaN takes its expert away."""
    E, k, G, Gk = 32, 6, 4, 2
    rng = np.random.default_rng(8)
    z = rng.standard_normal((40, E))
    z[0] = np.nan
    z[1] = -np.inf
    z[2, 3:] = -np.inf
    z[3, ::2] = np.nan
    z[4, 5] = np.inf
    z[5, [5, 6, 20]] = np.inf
    z[6] *= 1e38
    z[7] = -3e38
    z[8, 1:] = -3e38
    z[9] = np.inf
    z[10] -= 800  # sigmoid underflows to 0 for some: weights of 0
    z[11] = -2000 - np.arange(E)  # every sigmoid is 0: renormalised weights are 0
    z[12, 8:16] = -np.inf  # a group with no expert
    z[13, 9:32] = -np.inf  # one group and one expert of another left
    _run(q, z, k, G=G, Gk=Gk, score=score, group_top=group_top, scale=2.5)
    _run(q, z, k, G=1, Gk=1, score=score, renorm=False)
    bias = 0.1 * rng.standard_normal(E)
    bias[4], bias[9], bias[30] = -np.inf, np.nan, 5.0
    _run(q, z, k, bias=bias, G=G, Gk=Gk, score=score, group_top=group_top)


def test_route_unaligned_logits(q):
    """Rows that start at any multiple of the element size."""
    import torch
    T, E, k = 9, 60, 4
    for dtype in (torch.float32, torch.bfloat16):
        buf = torch.randn(T * E + 3, device="cuda").to(dtype)
        z = buf[1:1 + T * E].view(T, E)
        idx, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
        q.route_logits(q.make_router(E, k), z, idx, w)
        ri, _ = mxref.route(z.double().cpu().numpy(), k)
        assert np.array_equal(idx.cpu().numpy(), ri)


def test_route_empty_and_refused(q):
    import torch
    r = q.make_router(16, 4)
    q.route_logits(r, torch.empty((0, 16), device="cuda"), torch.empty((0, 4), dtype=torch.int32, device="cuda"),
                   torch.empty((0, 4), device="cuda"))
    z, i, w = torch.zeros((2, 16), device="cuda"), torch.zeros((2, 4), dtype=torch.int32, device="cuda"), torch.zeros((2, 4), device="cuda")
    with pytest.raises(ValueError):
        q.route_logits(r, z[:, :8].contiguous(), i, w)
    with pytest.raises(ValueError):
        q.route_logits(r, z, i, w, bias=torch.zeros(8, device="cuda"))
    with pytest.raises(TypeError):
        q.route_logits(r, z, i.long(), w)
    with pytest.raises(ValueError):
        q.make_router(16, 4, score="tanh")
    with pytest.raises(q.ColiError) as e:
        q.route_logits(q.make_router(16, 4, 2, 3), z, i, w)
    assert e.value.status == q.COLI_E_INVALID


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("B", [1.0, 64.0, 512.0, 2.0 ** 14, 2.0 ** 22, 2.0 ** 40, 3e38])
@pytest.mark.parametrize("E,m,Gk", [(8, 2, 1), (16, 2, 3), (64, 8, 4)])
def test_route_groups_whose_best_cancel(q, E, m, Gk, B, score):
    """Groups by their two best, whose biases are B and -B: the sum is small, what its two keys were
    rounded by is not. Logits a little apart, so that groups differ by less than that."""
    rng = np.random.default_rng(E + int(np.log2(B)))
    T, G = 400, E // m
    z = 0.5 * rng.standard_normal((T, 1)) + 4e-5 * rng.standard_normal((T, E))
    bias = np.full(E, -np.inf)
    bias[::m], bias[1::m] = B, -B
    if m > 2:
        bias[2::m] = -3e38  # present and never among the two best (but equal to them at the largest B)
    _run(q, z, min(8, 2 * Gk), bias=bias, G=G, Gk=Gk, score=score, group_top=2, scale=2.5)


def test_route_groups_one_of_which_cancels(q):
    """One group's biases cancel, the others have none."""
    rng = np.random.default_rng(12)
    T, E, G = 500, 32, 8
    for B in (64.0, 700.0, 1e5):
        z = 0.3 * rng.standard_normal((T, 1)) + 4e-5 * rng.standard_normal((T, E))
        bias = np.zeros(E)
        bias[8], bias[9], bias[10], bias[11] = B, -B, -4 * B, -4 * B
        _run(q, z, 6, bias=bias, G=G, Gk=3, group_top=2)
        _run(q, z, 6, bias=bias, G=G, Gk=3, group_top=1)
