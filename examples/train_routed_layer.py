"""A routed layer in training: the library's route, the pairs' way to their experts and back, and the
gradients of all three, around experts that are torch's own products.

    route_logits -> sort_pairs -> dispatch -> experts (torch) -> combine
    combine_backward -> (torch) -> combine without weights, route_logits_backward

    python examples/train_routed_layer.py [--tokens 512] [--hidden 256] [--ffn 128] [--experts 16] [--top-k 4]

It takes a few steps on a random regression and prints, before them, how far the gradients are from
those of the same layer in plain torch.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_moe_sigmoid_amd as q  # noqa: E402


class Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, router, bias):
        T, k = logits.shape[0], router.top_k
        idx = torch.empty((T, k), dtype=torch.int32, device=logits.device)
        w = torch.empty((T, k), device=logits.device)
        q.route_logits(router, logits, idx, w, bias=bias)
        ctx.save_for_backward(logits, idx)
        ctx.router = router
        ctx.mark_non_differentiable(idx)
        return idx, w

    @staticmethod
    def backward(ctx, _, dw):
        logits, idx = ctx.saved_tensors
        dlogits = torch.empty_like(logits)
        q.route_logits_backward(ctx.router, logits, idx, dw.contiguous(), dlogits)
        return dlogits, None, None


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, pos):
        rows = torch.empty((pos.numel(), x.shape[1]), dtype=x.dtype, device=x.device)
        q.dispatch(x, pos, rows)
        ctx.save_for_backward(pos)
        ctx.shape = x.shape
        return rows

    @staticmethod
    def backward(ctx, drows):
        dx = torch.empty(ctx.shape, dtype=drows.dtype, device=drows.device)
        q.combine(drows.contiguous(), ctx.saved_tensors[0], dx)
        return dx, None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, pos, w):
        out = torch.empty((w.shape[0], rows.shape[1]), dtype=rows.dtype, device=rows.device)
        q.combine(rows, pos, out, topk_w=w)
        ctx.save_for_backward(rows, pos, w)
        return out

    @staticmethod
    def backward(ctx, dout):
        rows, pos, w = ctx.saved_tensors
        drows, dw = torch.zeros_like(rows), torch.empty_like(w)
        q.combine_backward(dout.contiguous(), rows, pos, w, drows, dw)
        return drows, None, dw


class RoutedLayer(torch.nn.Module):
    def __init__(self, hidden, ffn, n_experts, top_k, score="sigmoid", device="cuda"):
        super().__init__()
        par = lambda *s: torch.nn.Parameter(torch.randn(s, device=device) / s[-1] ** 0.5)  # noqa: E731
        self.router = q.make_router(n_experts, top_k, score=score, renorm=True, scale=2.5)
        self.gate, self.up = par(n_experts, ffn, hidden), par(n_experts, ffn, hidden)
        self.down, self.to_logits = par(n_experts, hidden, ffn), par(n_experts, hidden)
        self.bias = 0.05 * torch.randn(n_experts, device=device)  # of the choice, not trained

    def expert(self, e, x):
        return (torch.nn.functional.silu(x @ self.gate[e].t()) * (x @ self.up[e].t())) @ self.down[e].t()

    def forward(self, x):
        T, E, k = x.shape[0], self.router.n_experts, self.router.top_k
        idx, w = Route.apply((x @ self.to_logits.t()).contiguous(), self.router, self.bias)
        i32 = lambda n: torch.empty(n, dtype=torch.int32, device=x.device)  # noqa: E731
        off, perm, pos, active, n_active = i32(E + 1), i32(T * k), i32(T * k), i32(E), i32(1)
        q.sort_pairs(idx, off, perm, pos, active, n_active, q.alloc_sort_pairs_workspace(T * k, E, x.device))
        rows = Dispatch.apply(x, pos)
        ends = off.tolist()
        y = torch.cat([self.expert(e, rows[ends[e]:ends[e + 1]]) for e in range(E)])
        return Combine.apply(y, pos, w)

    def plain(self, x):
        """The same in torch's own operations."""
        z = x @ self.to_logits.t()
        p = torch.sigmoid(z) if self.router.score == 0 else torch.softmax(z, 1)
        idx = torch.topk(p + self.bias, self.router.top_k, dim=1).indices
        taken = torch.gather(p, 1, idx)
        w = 2.5 * taken / taken.sum(1, keepdim=True)
        out = torch.zeros_like(x)
        for e in range(self.router.n_experts):
            t, j = torch.nonzero(idx == e, as_tuple=True)
            out = out.index_add(0, t, w[t, j][:, None] * self.expert(e, x[t]))
        return out


def gradients(layer, f, x, target):
    x = x.clone().requires_grad_(True)
    loss = ((f(x) - target) ** 2).sum()
    return torch.autograd.grad(loss, [x, *layer.parameters()])


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, v in (("tokens", 512), ("hidden", 256), ("ffn", 128), ("experts", 16), ("top-k", 4), ("steps", 3)):
        ap.add_argument("--" + name, type=int, default=v)
    ap.add_argument("--score", default="sigmoid", choices=["sigmoid", "softmax"])
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    layer = RoutedLayer(a.hidden, a.ffn, a.experts, a.top_k, a.score)
    x, target = torch.randn((2, a.tokens, a.hidden), device="cuda")
    ours, plain = gradients(layer, layer, x, target), gradients(layer, layer.plain, x, target)
    err = max(float((g - w).norm() / w.norm()) for g, w in zip(ours, plain))
    print(f"largest distance of a gradient from plain torch's, relative: {err:.1e}")
    opt = torch.optim.SGD(layer.parameters(), lr=1e-3)
    for step in range(a.steps):
        loss = ((layer(x) - target) ** 2).mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        print(f"step {step}: loss {loss.item():.4f}")
    return err


if __name__ == "__main__":
    main()
