"""The measured cases of the int8 products with token and channel scales, of the pairs' way to
their experts and back with its gradient, and of the gradient of the route.

Each case runs one operator:
  linear      x W^T + bias, x quantised to int8 with a scale for each row, W int8 with one for each row;
  gate_up     silu(gate) * up of every pair of a route, on the experts' int8 rows;
  down        the pairs' down rows, weighted and summed for each token, with the shared expert's;
  dispatch    the pairs sorted by expert, and the tokens' rows laid out in that order;
  combine     rows in that order back to their tokens, weighted and summed; `grad`: the gradient of
              that, of the rows and of the weights; without weights it is the gradient of dispatch;
  route_grad  the gradient of the route's weights with respect to the logits.
Where `own` is false `run` computes the operator's plain form in torch.

int8 of a row: s = max|x| / 127 in fp32, codes x / s (one fp32 division) rounded to nearest, halves
away from zero. An expert blob is gate [F][H] | up [F][H] | down [H][F], its scales one for each row.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ cases
def linear(M, N, K, dtype, bias=False):
    return dict(op="linear", M=M, N=N, K=K, dtype=dtype, bias=bias)


def experts(op, T, H, F, E, k, shared, dtype, skew=False, dropped=False):
    return dict(op=op, T=T, H=H, F=F, E=E, k=k, shared=shared, dtype=dtype, skew=skew, dropped=dropped)


def pairs(op, T, H, E, k, dtype, skew=False, dropped=False, weights=True, add=False, grad=False):
    return dict(op=op, T=T, H=H, E=E, k=k, dtype=dtype, skew=skew, dropped=dropped, weights=weights, add=add, grad=grad)


def route_grad(T, E, k, score, dtype, renorm=True, scale=1.0, masked=False):
    return dict(op="route_grad", T=T, E=E, k=k, score=score, dtype=dtype, renorm=renorm, scale=scale, masked=masked)


def listed():
    return [
        # one token through a dense feed-forward's first matrix: bound by the weights
        dict(name="linear one token", **linear(1, 12288, 6144, "bf16")),
        # a prompt chunk of a ragged length through the same matrix: bound by the matrix cores
        dict(name="linear prefill", **linear(4093, 12288, 6144, "bf16", True)),
        # the first half of a decode batch's expert FFN, 256 experts and a shared one
        dict(name="gate/up decode", **experts("gate_up", 16, 6144, 2048, 256, 8, True, "bf16")),
        # a prompt chunk over every expert, routed unevenly
        dict(name="gate/up prefill", **experts("gate_up", 2048, 6144, 2048, 256, 8, True, "bf16", skew=True)),
        # the second half of one token's expert FFN, in fp32 as the layer has it
        dict(name="down one token", **experts("down", 1, 6144, 2048, 256, 8, True, "f32")),
        # the second half of the prompt chunk's, with its combine and slots that the route left empty
        dict(name="down prefill", **experts("down", 2048, 6144, 2048, 256, 8, True, "bf16", skew=True, dropped=True)),
        # a decode batch laid out by expert: latency only
        dict(name="dispatch decode", **pairs("dispatch", 16, 6144, 256, 8, "bf16")),
        # the longest chunk that the layer routes at once (T * k near its limit), small experts
        dict(name="dispatch prefill", **pairs("dispatch", 8191, 2048, 64, 8, "bf16", skew=True)),
        # the experts' rows back to a prompt chunk's tokens, the shared expert's added
        dict(name="combine prefill", **pairs("combine", 2048, 6144, 256, 8, "f16", skew=True, dropped=True, add=True)),
        # its gradient in a training step in fp32
        dict(name="combine gradient", **pairs("combine", 4093, 2048, 64, 8, "f32", grad=True)),
        # a few sequences' router in a small training step: latency only
        dict(name="route gradient softmax", **route_grad(61, 64, 8, "softmax", "bf16", renorm=False, masked=True)),
        # the sigmoid router of a long chunk
        dict(name="route gradient sigmoid", **route_grad(8191, 256, 8, "sigmoid", "f32", True, 2.5)),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "gate_up", "down", "dispatch", "combine", "combine", "route_grad"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    skew, dropped = rng.random() < 0.5, rng.random() < 0.3
    if op == "linear":
        return linear(_log(rng, 1, 4093), _log(rng, 16, 12288), 16 * _log(rng, 4, 384), dtype, rng.random() < 0.5)
    E = rng.choice([8, 16, 60, 64, 128, 256])
    k = rng.randint(1, 8)
    if op in ("gate_up", "down"):
        return experts(op, _log(rng, 1, 2048), 128 * rng.randint(2, 48), 128 * rng.randint(1, 16), E, k,
                       rng.random() < 0.5, dtype, skew, dropped)
    if op == "route_grad":
        return route_grad(_log(rng, 1, 8191), E, k, rng.choice(["sigmoid", "softmax"]), dtype, rng.random() < 0.6,
                          rng.choice([1.0, 2.5]), rng.random() < 0.3)
    H = _log(rng, 64, 6144)
    T = _log(rng, 1, min(8191, 8191 * 2048 // H))
    if op == "dispatch":
        return pairs(op, T, H, E, k, dtype, skew, dropped)
    grad = rng.random() < 0.5
    return pairs(op, T // 2 + 1, H, E, k, dtype, skew, dropped, grad or rng.random() < 0.6, not grad and rng.random() < 0.5, grad)


def work(case):
    c, s = case, SIZE[case["dtype"]]
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K * s + N * K + 4 * N * (1 + c["bias"]) + M * N * s, "flops": 2 * M * N * K}
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] == "route_grad":
        return {"bytes": 2 * T * E * s + 8 * T * k, "flops": 8 * T * E}
    H = c["H"]
    kept = T * k * (4 if c["dropped"] else 5) // 5
    if c["op"] == "dispatch":
        return {"bytes": 4 * T * k + 8 * kept + T * H * s + kept * H * s, "flops": T * k}
    if c["op"] == "combine":
        rows = T * (2 if c["add"] else 1) + kept * (2 if c["grad"] else 1)
        return {"bytes": 4 * T * k * (1 + c["weights"] + c["grad"]) + rows * H * s, "flops": kept * H * (3 if c["grad"] else 2)}
    F, rows = c["F"], kept + T * c["shared"]
    hit = E * (1 - (1 - k / E) ** T) + c["shared"]  # distinct experts of an even route, each read once
    if c["op"] == "gate_up":
        return {"bytes": int(hit * 2 * F * (H + 4)) + T * H * s + rows * F * s, "flops": 4 * rows * F * H}
    return {"bytes": int(hit * H * (F + 4)) + rows * F * s + T * H * s, "flops": 2 * rows * F * H}


# ------------------------------------------------------------------ inputs
def _weights(g, n, rows, cols, dev):
    """n matrices of int8 codes, rows of about unit length, and their scales."""
    codes = torch.randint(-127, 128, (n, rows, cols), dtype=torch.int8, device=dev, generator=g)
    scales = (0.5 + torch.rand((n, rows), device=dev, generator=g)) / (73 * math.sqrt(cols))
    return codes, scales


def _routed(g, T, E, k, skew, dropped, dev):
    """A route and its grouping: idx, w [T][k], pairs sorted by (expert, pair), their places, offsets, hit experts."""
    z = torch.randn((T, E), device=dev, generator=g)
    if skew:  # popularity along a Zipf law, in random order
        z = z - 0.5 * torch.log1p(torch.randperm(E, device=dev, generator=g).float())
    top = torch.sort(z, dim=1, descending=True, stable=True)
    idx = top.indices[:, :k].to(torch.int32).contiguous()
    w = torch.softmax(top.values[:, :k], 1) * 2.5
    if dropped:  # slots that an adaptive route or an expert's full capacity leaves empty
        gone = torch.rand((T, k), device=dev, generator=g) < 0.2
        idx = torch.where(gone, torch.full_like(idx, -1), idx)
        w = torch.where(gone, torch.zeros_like(w), w)
    perm, pos, off, active, n_active = _sorted(idx, E)
    return dict(idx=idx, w=w.contiguous(), perm=perm, pos=pos, off=off, active=active, n_active=n_active)


def _sorted(idx, E):
    flat = idx.reshape(-1).long()
    there = flat >= 0
    key = torch.where(there, flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=order.device)
    pos = torch.where(there, pos, torch.full_like(pos, -1)).to(torch.int32)
    perm = torch.where(torch.arange(order.numel(), device=order.device) < there.sum(), order, torch.zeros_like(order))
    cnt = torch.zeros(E + 1, dtype=torch.int64, device=idx.device).index_add_(0, key, torch.ones_like(key))[:E]
    off = torch.zeros(E + 1, dtype=torch.int32, device=idx.device)
    off[1:] = torch.cumsum(cnt, 0).to(torch.int32)
    n_hit = (cnt > 0).sum().to(torch.int32).reshape(1)
    hit = torch.sort((cnt == 0).to(torch.int32), stable=True).indices.to(torch.int32)  # hit experts first
    active = torch.where(torch.arange(E, device=idx.device) < n_hit, hit, torch.zeros_like(hit))
    return perm.to(torch.int32), pos, off, active, n_hit


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c, s = case, {"case": case}
    dt = DTYPES[c["dtype"]]
    rand = lambda *shape: torch.randn(shape, device=dev, generator=g)  # noqa: E731
    new = lambda *shape, dtype=dt: torch.zeros(shape, dtype=dtype, device=dev)  # noqa: E731
    i32 = torch.int32
    if c["op"] == "linear":
        codes, scales = _weights(g, 1, c["N"], c["K"], dev)
        # rows of very different sizes, as tokens have them
        x = rand(c["M"], c["K"]) * torch.exp2(2 * rand(c["M"], 1))
        s.update(x=x.to(dt), codes=codes[0], scales=scales[0], bias=rand(c["N"]) if c["bias"] else None, out=new(c["M"], c["N"]))
    elif c["op"] == "route_grad":
        T, E, k = c["T"], c["E"], c["k"]
        z = (1.5 * rand(T, E)).to(dt)
        if c["masked"]:  # experts that are away for some tokens, and now and then no expert at all
            z = z.masked_fill(torch.rand((T, E), device=dev, generator=g) < 0.1, float("-inf"))
            z = z.masked_fill(torch.rand((T, 1), device=dev, generator=g) < 0.06, float("-inf"))
        top = torch.sort(z.float(), dim=1, descending=True, stable=True)
        idx = torch.where(torch.isneginf(top.values[:, :k]), torch.full_like(top.indices[:, :k], -1), top.indices[:, :k])
        s.update(z=z, idx=idx.to(i32).contiguous(), dw=rand(T, k), dz=new(T, E))
    elif c["op"] in ("dispatch", "combine"):
        T, H, E, k = c["T"], c["H"], c["E"], c["k"]
        s.update(_routed(g, T, E, k, c["skew"], c["dropped"], dev))
        if c["op"] == "dispatch":
            s.update(x=rand(T, H).to(dt), rows=new(T * k, H), o_off=new(E + 1, dtype=i32), o_perm=new(T * k, dtype=i32),
                     o_pos=new(T * k, dtype=i32), o_active=new(E, dtype=i32), o_n=new(1, dtype=i32))
        else:
            s.update(y=rand(T * k, H).to(dt), add=rand(T, H).to(dt) if c["add"] else None)
            if c["grad"]:
                s.update(dout=rand(T, H).to(dt), dy=new(T * k, H), dw=new(T, k, dtype=torch.float32))
            else:
                s.update(out=new(T, H))
    else:
        T, H, F, E, k, S = c["T"], c["H"], c["F"], c["E"], c["k"], int(c["shared"])
        s.update(_routed(g, T, E, k, c["skew"], c["dropped"], dev))
        codes, _ = _weights(g, E + S, 1, 3 * F * H, dev)
        scales = (0.5 + torch.rand((E + S, 2 * F + H), device=dev, generator=g)) / 73
        scales[:, :2 * F] /= math.sqrt(H)
        scales[:, 2 * F:] /= math.sqrt(F)
        s.update(codes=codes.view(E + S, -1), scales=scales)
        rows = T * k + S * T
        if c["op"] == "gate_up":
            s.update(x=rand(T, H).to(dt), h=new(rows, F))
        else:
            gate = rand(rows, F)
            s.update(h=(gate * torch.sigmoid(gate) * rand(rows, F)).to(dt), out=new(T, H))
    if own:  # what a program of the library keeps: its configuration, weights and workspace
        import quantized_moe_sigmoid_amd as q
        if c["op"] == "linear":
            s["ws"] = q.alloc_int8_linear_workspace(c["M"], c["N"], c["K"], dev)
        elif c["op"] == "dispatch":
            s["ws"] = q.alloc_sort_pairs_workspace(c["T"] * c["k"], c["E"], dev)
        elif c["op"] == "route_grad":
            s["router"] = q.make_router(c["E"], c["k"], score=c["score"], renorm=c["renorm"], scale=c["scale"])
        elif c["op"] in ("gate_up", "down"):
            s["cfg"] = q.make_cfg(c["H"], c["F"], c["E"], c["k"], has_shared=c["shared"], wbits=8)
            s["weights"] = q.Weights(s["codes"], s["scales"], None, None)
            s["ws"] = q.alloc_int8_experts_workspace(s["cfg"], c["T"], dev)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"linear": _linear, "gate_up": _gate_up, "down": _down, "dispatch": _dispatch, "combine": _combine,
                "route_grad": _route_grad}[op](s)
    import quantized_moe_sigmoid_amd as q
    if op == "linear":
        q.int8_linear(s["x"], s["codes"], s["scales"], s["out"], s["ws"], bias=s["bias"])
        return {"y": s["out"]}
    if op == "gate_up":
        q.int8_gate_up(s["cfg"], s["weights"], s["x"], s["off"], s["perm"], s["active"], s["n_active"], s["h"], s["ws"])
        return {"h": s["h"]}
    if op == "down":
        q.int8_down(s["cfg"], s["weights"], s["h"], s["idx"], s["w"], s["off"], s["perm"], s["active"], s["n_active"],
                    s["out"], s["ws"])
        return {"out": s["out"]}
    if op == "dispatch":
        q.sort_pairs(s["idx"], s["o_off"], s["o_perm"], s["o_pos"], s["o_active"], s["o_n"], s["ws"])
        q.dispatch(s["x"], s["o_pos"], s["rows"])
        return {"rows": s["rows"], "off": s["o_off"], "perm": s["o_perm"], "pos": s["o_pos"], "active": s["o_active"],
                "n_active": s["o_n"]}
    if op == "combine":
        w = s["w"] if s["case"]["weights"] else None
        if s["case"]["grad"]:
            q.combine_backward(s["dout"], s["y"], s["pos"], w, s["dy"], s["dw"])
            return {"dy": s["dy"], "dw": s["dw"]}
        q.combine(s["y"], s["pos"], s["out"], topk_w=w, add=s["add"])
        return {"out": s["out"]}
    q.route_logits_backward(s["router"], s["z"], s["idx"], s["dw"], s["dz"])
    return {"dz": s["dz"]}


# ------------------------------------------------------------------ plain forms
def _rounded(x):
    """fp32 codes and scales of the rows of x; divisions in 64 bits round to those in 32."""
    x = x.float()
    scale = (x.abs().amax(1).double() / 127).float()
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    v = (x.double() / safe.double()[:, None]).float().double()
    q = torch.sign(v) * torch.floor(v.abs() + 0.5)
    return torch.where(scale[:, None] > 0, q.clamp(-127, 127), torch.zeros_like(q)).float(), scale


def _product(x, sx, codes, scales):
    return (x @ codes.float().t()) * (sx[:, None] * scales[None, :])


def _linear(s):
    y = _product(*_rounded(s["x"]), s["codes"], s["scales"])
    return {"y": (y if s["bias"] is None else y + s["bias"]).to(s["x"].dtype)}


def _groups(s):
    """The hit experts with the pairs that chose them, the shared expert last."""
    c = s["case"]
    ends = s["off"].tolist()
    for e in range(c["E"]):
        if ends[e + 1] > ends[e]:
            yield e, s["perm"][ends[e]:ends[e + 1]].long()
    if c["shared"]:
        yield c["E"], torch.arange(c["T"], device=s["perm"].device) + c["T"] * c["k"]


def _gate_up(s):
    c = s["case"]
    H, F, k, h = c["H"], c["F"], c["k"], torch.zeros_like(s["h"])
    x, sx = _rounded(s["x"])
    for e, rows in _groups(s):
        token = rows // k if e < c["E"] else rows - c["T"] * k
        gu = _product(x[token], sx[token], s["codes"][e, :2 * F * H].view(2 * F, H), s["scales"][e, :2 * F])
        g, u = gu[:, :F], gu[:, F:]
        h[rows] = (g / (1 + torch.exp(-g)) * u).to(h.dtype)
    return {"h": h}


def _down(s):
    c = s["case"]
    T, H, F, k = c["T"], c["H"], c["F"], c["k"]
    h, sh = _rounded(s["h"])
    y = torch.zeros((h.shape[0], H), device=h.device)
    for e, rows in _groups(s):
        y[rows] = _product(h[rows], sh[rows], s["codes"][e, 2 * F * H:].view(H, F), s["scales"][e, 2 * F:])
    out = (s["w"][:, :, None] * y[:T * k].view(T, k, H)).sum(1)
    return {"out": (out + y[T * k:] if c["shared"] else out).to(s["out"].dtype)}


def _dispatch(s):
    perm, pos, off, active, n_active = _sorted(s["idx"], s["case"]["E"])
    there = (pos >= 0).sum()
    row = torch.arange(perm.numel(), device=perm.device)
    rows = torch.where((row < there)[:, None], s["x"][perm.long() // s["case"]["k"]], torch.zeros_like(s["rows"]))
    return {"rows": rows, "off": off, "perm": perm, "pos": pos, "active": active, "n_active": n_active}


def _combine(s):
    c = s["case"]
    T, k = c["T"], c["k"]
    pos = s["pos"].long().view(T, k)
    there = pos >= 0
    y = torch.where(there[..., None], s["y"][pos.clamp(min=0)].float(), torch.zeros((), device=pos.device))
    if c["grad"]:
        dout = s["dout"].float()
        dy = torch.zeros_like(s["dy"])
        dy[pos[there]] = (s["w"][..., None] * dout[:, None, :])[there].to(dy.dtype)
        return {"dy": dy, "dw": (y * dout[:, None, :]).sum(2)}
    out = (s["w"][..., None] * y).sum(1) if c["weights"] else y.sum(1)
    return {"out": (out if s["add"] is None else out + s["add"].float()).to(s["out"].dtype)}


def _route_grad(s):
    """In 64 bits: what is left of a weight's gradient is a difference."""
    c = s["case"]
    z = s["z"].double()
    idx = s["idx"].long()
    there = idx >= 0
    zero = torch.zeros((), dtype=z.dtype, device=z.device)
    if c["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-z))
    else:
        top = z.amax(1, keepdim=True)
        p = torch.where(z > float("-inf"), torch.exp(z - torch.where(top > float("-inf"), top, zero)), zero)
        total = p.sum(1, keepdim=True)
        p = torch.where(total > 0, p / total, zero)
    g = torch.where(there, s["dw"].double(), zero) * c["scale"]
    if c["renorm"]:
        taken = torch.where(there, torch.gather(p, 1, idx.clamp(min=0)), zero)
        total = taken.sum(1, keepdim=True)
        total = torch.where(total > 0, total, torch.ones_like(total))
        share = taken / total
        g = torch.where(there, (g - (g * share).sum(1, keepdim=True)) / total, zero)
    dp = torch.zeros_like(z).scatter_add_(1, idx.clamp(min=0), g)
    if c["score"] == "sigmoid":
        dz = dp * p * (1 - p)
    else:
        dz = p * dp if c["renorm"] else p * (dp - (p * dp).sum(1, keepdim=True))
    return {"dz": dz.to(s["dz"].dtype)}


# ------------------------------------------------------------------ 64 bits, from the definitions
def _codes64(x):
    """The same fp32 divisions, then a code as the number of half steps that a magnitude has passed."""
    x = x.to(torch.float32)
    top = torch.maximum(x.amax(1), -x.amin(1)).to(torch.float64)
    scale = torch.div(top, 127.0).to(torch.float32).to(torch.float64)
    ratio = torch.nan_to_num(x.to(torch.float64) / scale[:, None], nan=0.0, posinf=0.0, neginf=0.0)
    ratio = ratio.to(torch.float32).to(torch.float64)
    steps = torch.div(2 * ratio.abs() + 1, 2, rounding_mode="floor").clamp(max=127)
    return torch.copysign(steps, ratio), scale


def _value64(s, e, first, rows, cols):
    """Rows of expert e's weights from row `first` of its scales on, as numbers."""
    H, F = s["case"]["H"], s["case"]["F"]
    at = first * H if first < 2 * F else 2 * F * H
    w = s["codes"][e][at:at + rows * cols].reshape(rows, cols).to(torch.float64)
    return w * s["scales"][e][first:first + rows, None].to(torch.float64)


def _exact_experts(case, s):
    T, H, F, k = case["T"], case["H"], case["F"], case["k"]
    gate_up = case["op"] == "gate_up"
    a, scale = _codes64(s["x"] if gate_up else s["h"])
    a = a * scale[:, None]
    owner = s["idx"].reshape(-1)
    out = torch.zeros(s["h"].shape if gate_up else (T, H), dtype=torch.float64, device=a.device)
    for e in range(case["E"] + int(case["shared"])):
        mine = torch.nonzero(owner == e).flatten() if e < case["E"] else torch.arange(T * k, T * k + T, device=a.device)
        if not mine.numel():
            continue
        token = torch.div(mine, k, rounding_mode="floor") if e < case["E"] else mine - T * k
        if gate_up:
            gate = torch.matmul(a[token], _value64(s, e, 0, F, H).t())
            up = torch.matmul(a[token], _value64(s, e, F, F, H).t())
            out[mine] = gate * torch.sigmoid(gate) * up
        else:
            y = torch.matmul(a[mine], _value64(s, e, 2 * F, H, F).t())
            out.index_add_(0, token, y if e == case["E"] else y * s["w"].reshape(-1)[mine, None].double())
    return {"h" if gate_up else "out": out}


def _exact_combine(case, s):
    """Over the sorted rows: each belongs to one pair."""
    T, H, k = case["T"], case["H"], case["k"]
    n = int(s["off"][-1])
    pair = s["perm"][:n].long()
    token = torch.div(pair, k, rounding_mode="floor")
    w = s["w"].reshape(-1)[pair].double() if case["weights"] else torch.ones(n, dtype=torch.float64, device=pair.device)
    if case["grad"]:
        dy = torch.zeros((T * k, H), dtype=torch.float64, device=pair.device)
        dw = torch.zeros(T * k, dtype=torch.float64, device=pair.device)
        up = s["dout"].double()[token]
        dy[:n] = up * w[:, None]
        dw[pair] = torch.linalg.vecdot(up, s["y"][:n].double())
        return {"dy": dy, "dw": dw.view(T, k)}
    out = s["add"].double() if case["add"] else torch.zeros((T, H), dtype=torch.float64, device=pair.device)
    return {"out": out.index_add(0, token, s["y"][:n].double() * w[:, None])}


def _exact_route(case, s):
    """By the derivative of each weight with respect to each logit."""
    T, E, k = case["T"], case["E"], case["k"]
    eye = torch.eye(E, dtype=torch.float64, device=s["z"].device)
    out = []
    for lo in range(0, T, 512):
        z = s["z"][lo:lo + 512].double()
        idx, dw = s["idx"][lo:lo + 512].long(), s["dw"][lo:lo + 512].double()
        there = (idx >= 0).double()
        p = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(z, 1))
        one = eye[idx.clamp(min=0)] * there[..., None]                      # [n][k][E]
        pj = (one * p[:, None, :]).sum(2)
        jac = one * torch.sigmoid(-z)[:, None, :] if case["score"] == "sigmoid" else one - p[:, None, :] * there[..., None]
        jac = jac * pj[..., None]                                           # d p_j / d z_e
        if case["renorm"]:
            total = pj.sum(1)[:, None, None]
            total = torch.where(total > 0, total, torch.ones_like(total))
            jac = jac / total - pj[..., None] * jac.sum(1, keepdim=True) / total ** 2
        out.append((dw[..., None] * jac).sum(1) * case["scale"])
    return {"dz": torch.cat(out)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        a, scale = _codes64(s["x"])
        y = torch.matmul(a, s["codes"].double().t()) * scale[:, None] * s["scales"].double()[None, :]
        return {"y": y if s["bias"] is None else y + s["bias"].double()}
    if case["op"] == "route_grad":
        return _exact_route(case, s)
    if case["op"] == "combine":
        return _exact_combine(case, s)
    if case["op"] == "dispatch":
        kept = torch.nonzero(s["idx"].reshape(-1) >= 0).flatten()
        rows = torch.zeros(s["rows"].shape, dtype=torch.float64, device=kept.device)
        rows[s["pos"].long()[kept]] = s["x"].double()[torch.div(kept, case["k"], rounding_mode="floor")]
        return {"rows": rows, "off": None, "perm": None, "pos": None, "active": None, "n_active": None}
    return _exact_experts(case, s)
