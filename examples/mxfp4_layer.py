"""One MoE layer whose every product has both operands in MXFP4, from the library's operators:

    logits = mxfp4_linear(x, router)            route = route_logits(logits)
    group(route)  ->  h = mxfp4_gate_up(x)  ->  out = mxfp4_down(h)

with weights quantised once by mxfp4_quantize. Run it on the GPU:

    python examples/mxfp4_layer.py [--tokens 16] [--hidden 2048] [--ffn 1024] [--experts 64] [--top-k 8]

It prints the layer's time, captured in a graph, and its largest distance from the same layer
in torch on the dequantised weights, relative to the output's largest value.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_moe_sigmoid_amd as q  # noqa: E402


def quantise(w):
    """A float matrix [rows][cols] as MXFP4: codes, scales."""
    codes = torch.empty((w.shape[0], w.shape[1] // 2), dtype=torch.uint8, device=w.device)
    scales = torch.empty((w.shape[0], w.shape[1] // 32), dtype=torch.uint8, device=w.device)
    q.mxfp4_quantize(w, codes, scales)
    return codes, scales


def values(codes, scales, dtype=torch.float32):
    out = torch.empty((codes.shape[0], codes.shape[1] * 2), dtype=dtype, device=codes.device)
    q.mxfp4_dequantize(codes, scales, out)
    return out


class Mxfp4Layer:
    """The layer's weights (random, of that architecture), its configuration and its buffers for up to T tokens."""

    def __init__(self, T, hidden, ffn, n_experts, top_k, n_group=1, topk_group=1, shared=True, dtype=torch.bfloat16,
                 device="cuda", seed=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        rand = lambda r, c: torch.randn((r, c), device=device, generator=g) / c ** 0.5  # noqa: E731
        self.T, self.top_k, self.dtype = T, top_k, dtype
        self.cfg = q.make_cfg(hidden, ffn, n_experts, top_k, has_shared=shared, wbits=q.W_MXFP4, scale_group=32)
        self.router = q.make_router(n_experts, top_k, n_group, topk_group, scale=2.5)
        self.bias = 0.05 * torch.randn(n_experts, device=device, generator=g)
        self.wr = quantise(2 * rand(n_experts, hidden))
        # expert blobs: gate [F][H] | up [F][H] | down [H][F]
        parts = [[quantise(rand(ffn, hidden)), quantise(rand(ffn, hidden)), quantise(rand(hidden, ffn))]
                 for _ in range(n_experts + shared)]
        self.weights = q.Weights(torch.stack([torch.cat([m[0].flatten() for m in p]) for p in parts]),
                                 torch.stack([torch.cat([m[1].flatten() for m in p]) for p in parts]), None, None)
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=device)  # noqa: E731
        self.logits = torch.empty((T, n_experts), dtype=dtype, device=device)
        self.idx, self.w = i32(T, top_k), torch.empty((T, top_k), device=device)
        self.cnt, self.off, self.perm, self.active, self.n_active = (
            i32(n_experts), i32(n_experts + 1), i32(T * top_k), i32(n_experts), i32(1))
        self.h = torch.zeros((T * (top_k + shared), ffn), dtype=dtype, device=device)
        self.ws_router = q.alloc_mxfp4_linear_workspace(T, n_experts, hidden, device)
        self.ws = q.alloc_mxfp4_experts_workspace(self.cfg, T, device)

    def __call__(self, x, out):
        """out [T][H] = the layer of x [T][H]; one stream, no allocation, no synchronisation."""
        q.mxfp4_linear(x, *self.wr, self.logits, self.ws_router)
        q.route_logits(self.router, self.logits, self.idx, self.w, bias=self.bias)
        q.group(self.cfg, self.idx, self.T, self.cnt, self.off, self.perm, self.active, self.n_active)
        q.mxfp4_gate_up(self.cfg, self.weights, x, self.off, self.perm, self.active, self.n_active, self.h, self.ws)
        q.mxfp4_down(self.cfg, self.weights, self.h, self.idx, self.w, self.off, self.perm, self.active, self.n_active,
                     out, self.ws)

    def reference(self, x):
        """The same products in torch, in 32 bits, over the route that the last call took."""
        c = self.cfg
        F, H, k = c.ffn, c.hidden, c.top_k
        stored = lambda a: values(*quantise(a.contiguous()))  # noqa: E731  what a product sees of its activations
        xs, out = stored(x), torch.zeros((x.shape[0], H), device=x.device)
        for e in range(c.n_experts + c.has_shared):
            if e < c.n_experts:
                t, j = torch.nonzero(self.idx == e, as_tuple=True)
                share = self.w[t, j]
            else:
                t = torch.arange(x.shape[0], device=x.device)
                share = torch.ones(x.shape[0], device=x.device)
            if not t.numel():
                continue
            codes, scales = self.weights.experts[e].view(3, -1), self.weights.scales[e].view(3, -1)
            gate, up = (values(codes[m].view(F, -1), scales[m].view(F, -1)) for m in (0, 1))
            down = values(codes[2].view(H, -1), scales[2].view(H, -1))
            h = (torch.nn.functional.silu(xs[t] @ gate.t()) * (xs[t] @ up.t())).to(self.dtype)
            out.index_add_(0, t, share[:, None] * (stored(h) @ down.t()))
        return out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, v in (("tokens", 16), ("hidden", 2048), ("ffn", 1024), ("experts", 64), ("top-k", 8)):
        ap.add_argument("--" + name, type=int, default=v)
    a = ap.parse_args(argv)
    layer = Mxfp4Layer(a.tokens, a.hidden, a.ffn, a.experts, a.top_k)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(layer.dtype)
    out = torch.empty_like(x)
    layer(x, out)
    want = layer.reference(x)
    err = ((out.float() - want).abs().max() / want.abs().max()).item()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, out)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for i in range(120):
        if i == 20:
            start.record()
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens, {a.experts} experts of {a.hidden} x {a.ffn}: "
          f"{start.elapsed_time(end) * 10:.1f} us a layer, largest distance {err:.1e}")
    return err


if __name__ == "__main__":
    main()
