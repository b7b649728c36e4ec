"""The int8 operators, the pairs' and the route's gradient in graphs, on other streams, side by side, and
with buffers larger than asked: every result bit for bit that of one eager call."""
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


class _Layer:
    """Every operator once, in the order of a training step around int8 experts, on buffers of its own."""

    def __init__(self, q, T, seed, H=512, F=384, E=24, k=4):
        import torch
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.q, self.T, self.k = q, T, k
        dt = torch.bfloat16
        rand = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        new = lambda *s: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        i8 = lambda *s: torch.randint(-127, 128, s, dtype=torch.int8, device="cuda", generator=g)  # noqa: E731
        self.cfg = q.make_cfg(H, F, E, k, has_shared=True, wbits=8)
        self.router = q.make_router(E, k, scale=2.5)
        self.w = q.Weights(i8(E + 1, 3 * F * H), (0.5 + torch.rand((E + 1, 2 * F + H), device="cuda", generator=g)) / 2000, None, None)
        self.wr, self.sr, self.br = i8(E, H), torch.rand(E, device="cuda", generator=g) / 2000, rand(E)
        self.x, self.dout = rand(T, H).to(dt), rand(T, H).to(dt)
        self.z, self.dz = new(T, E), new(T, E)
        self.idx, self.tw, self.dtw = i32(T, k), torch.zeros((T, k), device="cuda"), torch.zeros((T, k), device="cuda")
        self.off, self.perm, self.pos, self.active, self.n = i32(E + 1), i32(T * k), i32(T * k), i32(E), i32(1)
        self.h, self.out, self.back, self.dx = new(T * (k + 1), F), new(T, H), new(T, H), new(T, H)
        self.rows, self.drows = new(T * k + 7, H), new(T * k + 7, H)
        self.codes, self.scales = torch.zeros((T, H), dtype=torch.int8, device="cuda"), torch.zeros(T, device="cuda")
        self.ws0 = q.alloc_int8_linear_workspace(T, E, H)
        self.ws1 = q.alloc_sort_pairs_workspace(T * k, E)
        self.ws2 = q.alloc_int8_experts_workspace(self.cfg, T)

    def run(self, stream=None):
        q, s = self.q, dict(stream=stream)
        q.int8_linear(self.x, self.wr, self.sr, self.z, self.ws0, bias=self.br, **s)
        q.route_logits(self.router, self.z, self.idx, self.tw, **s)
        q.sort_pairs(self.idx, self.off, self.perm, self.pos, self.active, self.n, self.ws1, **s)
        q.int8_gate_up(self.cfg, self.w, self.x, self.off, self.perm, self.active, self.n, self.h, self.ws2, **s)
        q.int8_down(self.cfg, self.w, self.h, self.idx, self.tw, self.off, self.perm, self.active, self.n, self.out, self.ws2, **s)
        q.dispatch(self.x, self.pos, self.rows, **s)
        q.combine(self.rows, self.pos, self.back, topk_w=self.tw, add=self.out, **s)
        q.combine_backward(self.dout, self.rows, self.pos, self.tw, self.drows, self.dtw, **s)
        q.combine(self.drows, self.pos, self.dx, **s)
        q.route_logits_backward(self.router, self.z, self.idx, self.dtw, self.dz, **s)
        q.int8_quantize(self.dx, self.codes, self.scales, **s)

    def results(self):
        return [t.clone() for t in (self.z, self.idx, self.tw, self.off, self.perm, self.pos, self.active, self.n, self.h, self.out,
                                    self.rows, self.back, self.drows, self.dtw, self.dx, self.dz, self.codes, self.scales)]


def _same(a, b):
    import torch
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T", [1, 13, 400, 10000])
def test_graph_replays(q, T):
    """Captured once, replayed on other inputs with eager work and waits between the replays."""
    import torch
    l = _Layer(q, T, 1)
    l.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        l.run()
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    for i in range(4):
        l.x.copy_(torch.randn(l.x.shape, device="cuda", generator=g))
        l.dout.copy_(torch.randn(l.x.shape, device="cuda", generator=g))
        if i & 1:
            torch.cuda.synchronize()
        l.run()
        want = l.results()
        for t in (l.z, l.idx, l.tw, l.pos, l.h, l.out, l.rows, l.back, l.drows, l.dtw, l.dx, l.dz, l.codes, l.scales):
            t.fill_(3)
        l.rows[T * l.k:].zero_(), l.drows[T * l.k:].zero_()  # rows of no pair stay as they are
        l.ws0.fill_(0xA5), l.ws1.fill_(0xA5), l.ws2.fill_(0xA5)
        graph.replay()
        assert _same(l.results(), want), i


def test_two_graphs_on_one_workspace(q):
    """One after another on one stream."""
    import torch
    a, b = _Layer(q, 300, 1), _Layer(q, 17, 2)
    b.ws0, b.ws1, b.ws2 = a.ws0, a.ws1, a.ws2
    want = []
    for l in (a, b):
        l.run()
        want.append(l.results())
    torch.cuda.synchronize()
    graphs = []
    for l in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            l.run()
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for i in order:
            graphs[i].replay()
    assert _same(a.results(), want[0]) and _same(b.results(), want[1])


def test_streams_side_by_side(q):
    """Two layers at once, each on a stream and buffers of its own, and the stream given or current."""
    import torch
    a, b = _Layer(q, 500, 3), _Layer(q, 16, 4)
    want = []
    for l in (a, b):
        l.run()
        want.append(l.results())
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for l in (a, b):
            for t in (l.z, l.h, l.out, l.back, l.dx, l.dz):
                t.fill_(3)
        torch.cuda.synchronize()
        for _ in range(3):
            a.run(stream=sa)
            with torch.cuda.stream(sb):
                b.run()
        torch.cuda.synchronize()
        assert _same(a.results(), want[0]) and _same(b.results(), want[1])


def test_run_to_run(q):
    import torch
    l = _Layer(q, 2000, 5)
    l.run()
    want = l.results()
    for _ in range(5):
        l.run()
        assert _same(l.results(), want)
    torch.cuda.synchronize()


@pytest.mark.parametrize("T", [1, 16, 300])
def test_nothing_outside_is_written(q, T):
    """Guard bytes around every output and workspace stay."""
    import torch
    l = _Layer(q, T, 6)
    guards = []
    for name in ("z", "dz", "idx", "tw", "dtw", "off", "perm", "pos", "active", "n", "h", "out", "back", "dx", "rows", "drows",
                 "codes", "scales", "ws0", "ws1", "ws2"):
        t = getattr(l, name)
        raw = torch.full((t.numel() * t.element_size() + 2 * 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        inner = raw[4096:4096 + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        inner.copy_(t)
        setattr(l, name, inner)
        guards.append((name, raw, t.numel() * t.element_size()))
    l.run()
    torch.cuda.synchronize()
    for name, raw, n in guards:
        assert (raw[:4096] == 0x5A).all() and (raw[4096 + n:] == 0x5A).all(), name


def test_refused_calls_write_nothing(q):
    """Workspaces too small, views that are not contiguous, tensors on the CPU, other types and shapes."""
    import torch
    l = _Layer(q, 40, 7)
    before = l.results()
    calls = [
        (q.ColiError, lambda: q.int8_linear(l.x, l.wr, l.sr, l.z, l.ws0[:256])),
        (q.ColiError, lambda: q.int8_gate_up(l.cfg, l.w, l.x, l.off, l.perm, l.active, l.n, l.h, l.ws2[:1024])),
        (q.ColiError, lambda: q.int8_linear(l.x, l.wr, l.sr, l.z, l.ws0[1:])),
        (ValueError, lambda: q.int8_linear(l.x.t(), l.wr, l.sr, l.z, l.ws0)),
        (ValueError, lambda: q.int8_linear(l.x, l.wr, l.sr[:-1], l.z, l.ws0)),
        (TypeError, lambda: q.int8_linear(l.x, l.wr.view(torch.uint8), l.sr, l.z, l.ws0)),
        (ValueError, lambda: q.int8_linear(l.x.cpu(), l.wr, l.sr, l.z, l.ws0)),
        (ValueError, lambda: q.int8_down(l.cfg, q.Weights(l.w.experts[:-1], l.w.scales, None, None), l.h, l.idx, l.tw, l.off, l.perm,
                                         l.active, l.n, l.out, l.ws2)),
        (TypeError, lambda: q.combine(l.rows.float(), l.pos, l.back)),
        (ValueError, lambda: q.combine(l.rows, l.pos, l.back, topk_w=l.tw[:, :3])),
        (TypeError, lambda: q.dispatch(l.x, l.pos.long(), l.rows)),
        (ValueError, lambda: q.combine_backward(l.dout, l.rows, l.pos, l.tw, l.drows[:-1], l.dtw)),
        (ValueError, lambda: q.route_logits_backward(l.router, l.z, l.idx, l.dtw, l.dz[:, :8])),
        (ValueError, lambda: q.sort_pairs(l.idx, l.off[:-1], l.perm, l.pos, l.active, l.n, l.ws1)),
        (q.ColiError, lambda: q.combine_backward(l.dout, l.rows, l.pos, l.tw)),
    ]
    for kind, call in calls:
        with pytest.raises(kind):
            call()
    torch.cuda.synchronize()
    assert _same(l.results(), before)
