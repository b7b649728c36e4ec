"""Routes with ids that are neither an expert nor -1: their slots are empty ones for the experts' products, in
batches of every size, whatever lay in the workspace, h and out before. sort_pairs and group say so by n_active
= -1 and leave the valid pairs grouped."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import quantized_moe_sigmoid_amd as q
    q.lib()
    return q


def _route(T, k, E):
    """A route with bad ids, and the same with -1 in their place."""
    rng = np.random.default_rng(T)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    clean = idx.copy()
    bad = rng.random((T, k)) < 0.1
    bad[T // 2] = True  # a token without any expert
    bad[0, 0] = T > 1
    idx[bad] = rng.choice([E, E + 1, -2, -5, 2 ** 31 - 1, -2 ** 31], bad.sum())
    clean[bad] = -1
    return idx, clean


def _grouped(q, how, cfg, idx):
    import torch
    T, k, E = *idx.shape, cfg.n_experts
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    ids = torch.from_numpy(idx).cuda()
    off, perm, active, n = i32(E + 1), i32(T * k), i32(E), i32(1)
    if how == "sort_pairs":
        q.sort_pairs(ids, off, perm, i32(T * k), active, n, q.alloc_sort_pairs_workspace(T * k, E))
    else:
        q.group(cfg, ids, T, i32(E), off, perm, active, n)
    return ids, (off, perm, active, n)


# int8: one kernel for both halves' few rows and one for many; down of up to 16 tokens with its combine in one
@pytest.mark.parametrize("how", ["sort_pairs", "group"])
@pytest.mark.parametrize("fmt", ["int8", "mxfp4"])
@pytest.mark.parametrize("T,E,k", [(1, 16, 4), (5, 16, 4), (16, 64, 8), (40, 16, 4), (40, 200, 3), (200, 16, 4), (90, 130, 20)])
def test_bad_ids_are_empty_slots(q, how, fmt, T, E, k):
    import torch
    H, F = 384, 256
    g = torch.Generator(device="cuda")
    g.manual_seed(T + E)
    if fmt == "int8":
        cfg = q.make_cfg(H, F, E, k, has_shared=True, wbits=8)
        w = q.Weights(torch.randint(-127, 128, (E + 1, 3 * F * H), dtype=torch.int8, device="cuda", generator=g),
                      (0.5 + torch.rand((E + 1, 2 * F + H), device="cuda", generator=g)) / 1000, None, None)
        gate_up, down, alloc = q.int8_gate_up, q.int8_down, q.alloc_int8_experts_workspace
    else:
        cfg = q.make_cfg(H, F, E, k, has_shared=True, wbits=q.W_MXFP4, scale_group=32)
        n = (E + 1) * 3 * F * H
        w = q.Weights(torch.randint(0, 256, (n // 2,), dtype=torch.uint8, device="cuda", generator=g),
                      torch.randint(120, 124, (n // 32,), dtype=torch.uint8, device="cuda", generator=g), None, None)
        gate_up, down, alloc = q.mxfp4_gate_up, q.mxfp4_down, q.alloc_mxfp4_experts_workspace
    x = torch.randn((T, H), device="cuda", generator=g)
    tw = torch.rand((T, k), device="cuda", generator=g)
    idx, clean = _route(T, k, E)

    def run(route, stale):
        ids, group = _grouped(q, how, cfg, route)
        h = torch.full((T * (k + 1), F), stale, device="cuda")
        out, ws = torch.full((T, H), stale, device="cuda"), alloc(cfg, T)
        ws.view(torch.float32).fill_(stale)
        gate_up(cfg, w, x, *group, h, ws)
        there = torch.cat([torch.from_numpy(clean.reshape(-1) >= 0).cuda(), torch.ones(T, dtype=torch.bool, device="cuda")])
        assert (h[~there] == stale).all()
        ws.view(torch.float32).fill_(stale)
        down(cfg, w, h, ids, tw, *group, out, ws)
        return int(group[3].item()), h[there], out

    n, h, out = run(clean, 9.0)
    assert n >= 0
    bad = run(idx, 1e6)
    assert bad[0] == -1
    assert torch.equal(bad[1], h) and torch.equal(bad[2], out)
