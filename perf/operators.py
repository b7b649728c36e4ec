"""The measured cases of the router from logits and the MXFP4 (microscaled 4-bit) operators.

Each case runs one operator: the route of T tokens from their logits, the MXFP4 quantisation
(packed, then unpacked to the values it stands for), the dense product x W^T with both operands
in MXFP4, and the experts' grouped products over a route (gate/up with SiLU*up, down with the
weighted combine). Where `own` is false `run` computes the operator's plain form in torch.

Operands. MXFP4 (OCP MX v1.0): 32 values share one E8M0 byte u = 2^(u - 127); codes are E2M1, byte
j of a 16-byte block = code j | code (j + 16) << 4. Activations are quantised inside the
operators; weights come quantised. An expert blob is gate [F][H] | up [F][H] | down [H][F].
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ cases
def route(T, E, k, score, dtype, G=1, Gk=1, group_top=2, bias=False, renorm=True, scale=1.0, masked=False):
    return dict(op="route", T=T, E=E, k=k, score=score, dtype=dtype, G=G, Gk=Gk, group_top=group_top, bias=bias,
                renorm=renorm, scale=scale, masked=masked)


def experts(op, T, H, F, E, k, shared, dtype, skew=False, dropped=False):
    return dict(op=op, T=T, H=H, F=F, E=E, k=k, shared=shared, dtype=dtype, skew=skew, dropped=dropped)


def listed():
    return [
        # the decode step of one sequence: a group-limited sigmoid router, latency only
        dict(name="route one token", **route(1, 256, 8, "sigmoid", "f32", 8, 4, 2, True, True, 2.5)),
        # a softmax gate over 64 experts whose weights are left as they are, 16-bit logits, some experts masked
        dict(name="route softmax", **route(4093, 64, 8, "softmax", "bf16", renorm=False, masked=True)),
        # the longest prompt chunk the library routes at once (T * k near its limit)
        dict(name="route prefill", **route(8191, 256, 8, "sigmoid", "f32", 8, 4, 2, True, True, 2.5)),
        # the activations of a decode batch
        dict(name="quantise decode", op="quantise", rows=16, cols=6144, dtype="bf16"),
        # a stack of expert rows turned into MXFP4 when a model is loaded
        dict(name="quantise weights", op="quantise", rows=49152, cols=2048, dtype="bf16"),
        # one token through a dense feed-forward's first matrix: bound by the weights
        dict(name="linear one token", op="linear", M=1, N=12288, K=6144, dtype="bf16"),
        # a small ragged batch on odd sizes (vocabulary slices, heads that are no multiple of a tile)
        dict(name="linear ragged", op="linear", M=77, N=2051, K=2080, dtype="f16"),
        # a prompt chunk through the same dense matrix: bound by the matrix cores
        dict(name="linear prefill", op="linear", M=4096, N=12288, K=6144, dtype="bf16"),
        # one token's experts, of 256 and a shared one
        dict(name="gate/up one token", **experts("gate_up", 1, 6144, 2048, 256, 8, True, "bf16")),
        # a prompt chunk over every expert, routed unevenly
        dict(name="gate/up prefill", **experts("gate_up", 2048, 6144, 2048, 256, 8, True, "bf16", skew=True)),
        # the second half of a decode batch's expert FFN, in fp32 as the int8 path has it
        dict(name="down decode", **experts("down", 16, 6144, 2048, 256, 8, True, "f32")),
        # the second half of the prompt chunk's, with its combine
        dict(name="down prefill", **experts("down", 2048, 6144, 2048, 256, 8, True, "bf16", skew=True)),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _drawn(rng)
    return draw(rng) if 3072 in case.values() else case  # 24 * 128 is no size of this library's


def _drawn(rng):
    op = rng.choice(["route", "quantise", "linear", "gate_up", "down"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    if op == "route":
        E = 8 * _log(rng, 1, 32)
        G = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0])
        Gk = rng.randint(1, G)
        k = rng.randint(1, min(8, Gk * E // G))
        return route(_log(rng, 1, 8191), E, k, rng.choice(["sigmoid", "softmax"]), dtype, G, Gk, rng.choice([1, 2]),
                     rng.random() < 0.5, rng.random() < 0.7, rng.choice([1.0, 2.5]), rng.random() < 0.3)
    if op == "quantise":
        cols = 32 * _log(rng, 1, 512)
        return dict(op=op, rows=_log(rng, 1, 49152 * 1024 // cols), cols=cols, dtype=dtype)
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 4096), N=_log(rng, 16, 12288), K=32 * _log(rng, 4, 192), dtype=dtype)
    E = rng.choice([8, 16, 60, 64, 128, 256])
    return experts(op, _log(rng, 1, 2048), 128 * rng.randint(2, 48), 128 * rng.randint(1, 16), E,
                   rng.randint(1, 8), rng.random() < 0.5, dtype, rng.random() < 0.5, rng.random() < 0.25)


def work(case):
    c = case
    if c["op"] == "route":
        n = c["T"] * c["E"]
        return {"bytes": n * SIZE[c["dtype"]] + 8 * c["T"] * c["k"] + 4 * c["E"] * c["bias"], "flops": 4 * n}
    if c["op"] == "quantise":  # read, the packed form, the unpacked values
        n = c["rows"] * c["cols"]
        return {"bytes": 2 * n * SIZE[c["dtype"]] + n * 17 // 32, "flops": 4 * n}
    if c["op"] == "linear":
        M, N, K, s = c["M"], c["N"], c["K"], SIZE[c["dtype"]]
        return {"bytes": M * K * s + N * K * 17 // 32 + M * N * s, "flops": 2 * M * N * K}
    T, H, F, E, k, s = c["T"], c["H"], c["F"], c["E"], c["k"], SIZE[c["dtype"]]
    rows = T * k + T * c["shared"]
    hit = E * (1 - (1 - k / E) ** T) + c["shared"]  # distinct experts of an even route, each read once
    if c["op"] == "gate_up":
        return {"bytes": int(hit * 2 * F * H * 17 / 32) + T * H * s + rows * F * s, "flops": 4 * rows * F * H}
    return {"bytes": int(hit * F * H * 17 / 32) + rows * F * s + T * H * s, "flops": 2 * rows * F * H}


# ------------------------------------------------------------------ inputs
def _weights(g, n, rows, cols, dev):
    """n matrices of random E2M1 codes with scales of a few binades around 2^-6."""
    codes = torch.randint(0, 256, (n, rows, cols // 2), dtype=torch.uint8, device=dev, generator=g)
    scales = torch.randint(119, 124, (n, rows, cols // 32), dtype=torch.uint8, device=dev, generator=g)
    return codes, scales


def _routed(g, T, E, k, skew, dropped, dev):
    """A route and its grouping: idx, w [T][k], pairs sorted by (expert, pair), offsets, hit experts."""
    z = torch.randn((T, E), device=dev, generator=g)
    if skew:  # popularity along a Zipf law, in random order
        z = z - 0.5 * torch.log1p(torch.randperm(E, device=dev, generator=g).float())
    top = torch.sort(z, dim=1, descending=True, stable=True)
    idx = top.indices[:, :k].to(torch.int32).contiguous()
    w = torch.softmax(top.values[:, :k], 1) * 2.5
    if dropped:  # slots that an adaptive route leaves empty
        gone = torch.rand((T, k), device=dev, generator=g) < 0.2
        idx = torch.where(gone, torch.full_like(idx, -1), idx)
        w = torch.where(gone, torch.zeros_like(w), w)
    flat = idx.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    perm = torch.sort(key, stable=True).indices.to(torch.int32)
    cnt = torch.bincount(key, minlength=E + 1)[:E]
    off = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    off[1:] = torch.cumsum(cnt, 0).to(torch.int32)
    hit = torch.sort((cnt == 0).to(torch.int32), stable=True).indices.to(torch.int32)  # hit experts first
    n_hit = (cnt > 0).sum().to(torch.int32).reshape(1)
    return dict(idx=idx, w=w.contiguous(), perm=perm, off=off, active=hit, n_active=n_hit)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c, s = case, {"case": case}
    dt = DTYPES[c["dtype"]]
    rand = lambda *shape: torch.randn(shape, device=dev, generator=g)  # noqa: E731
    new = lambda *shape, dtype=dt: torch.zeros(shape, dtype=dtype, device=dev)  # noqa: E731
    if c["op"] == "route":
        T, E = c["T"], c["E"]
        z = (1.5 * rand(T, E)).to(dt)
        if c["masked"]:  # experts that are away for some tokens, and now and then no expert at all
            z = z.masked_fill(torch.rand((T, E), device=dev, generator=g) < 0.1, float("-inf"))
            z = z.masked_fill(torch.rand((T, 1), device=dev, generator=g) < 0.06, float("-inf"))
        s.update(z=z, bias=0.05 * rand(E) if c["bias"] else None, idx=new(T, c["k"], dtype=torch.int32),
                 w=new(T, c["k"], dtype=torch.float32))
    elif c["op"] == "quantise":
        rows, cols = c["rows"], c["cols"]
        # values whose block maxima spread over many binades, as weights and activations have them
        x = rand(rows, cols) * torch.exp2(3 * rand(rows, cols // 32)).repeat_interleave(32, 1)
        s.update(x=x.to(dt), codes=new(rows, cols // 2, dtype=torch.uint8), scales=new(rows, cols // 32, dtype=torch.uint8),
                 out=new(rows, cols))
    elif c["op"] == "linear":
        codes, scales = _weights(g, 1, c["N"], c["K"], dev)
        s.update(x=rand(c["M"], c["K"]).to(dt), codes=codes[0], scales=scales[0], out=new(c["M"], c["N"]))
    else:
        T, H, F, E, k, S = c["T"], c["H"], c["F"], c["E"], c["k"], int(c["shared"])
        s.update(_routed(g, T, E, k, c["skew"], c["dropped"], dev))
        codes, scales = _weights(g, E + S, 1, 3 * F * H, dev)
        s.update(codes=codes.view(E + S, -1), scales=scales.view(E + S, -1))
        rows = T * k + S * T
        if c["op"] == "gate_up":
            s.update(x=rand(T, H).to(dt), h=new(rows, F))
        else:
            gate = rand(rows, F)
            s.update(h=(gate * torch.sigmoid(gate) * rand(rows, F)).to(dt), out=new(T, H))
    if own:  # what a program of the library keeps: its configuration, weights and workspace
        import quantized_moe_sigmoid_amd as q
        if c["op"] == "route":
            s["router"] = q.make_router(c["E"], c["k"], c["G"], c["Gk"], score=c["score"], group_top=c["group_top"],
                                        renorm=c["renorm"], scale=c["scale"])
        elif c["op"] == "linear":
            s["ws"] = q.alloc_mxfp4_linear_workspace(c["M"], c["N"], c["K"], dev)
        elif c["op"] in ("gate_up", "down"):
            s["cfg"] = q.make_cfg(c["H"], c["F"], c["E"], c["k"], has_shared=c["shared"], wbits=q.W_MXFP4, scale_group=32)
            s["weights"] = q.Weights(s["codes"], s["scales"], None, None)
            s["ws"] = q.alloc_mxfp4_experts_workspace(s["cfg"], c["T"], dev)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"route": _route, "quantise": _quantise, "linear": _linear, "gate_up": _gate_up, "down": _down}[op](s)
    import quantized_moe_sigmoid_amd as q
    if op == "route":
        q.route_logits(s["router"], s["z"], s["idx"], s["w"], bias=s["bias"])
        return {"experts": s["idx"], "weights": s["w"]}
    if op == "quantise":
        q.mxfp4_quantize(s["x"], s["codes"], s["scales"])
        q.mxfp4_dequantize(s["codes"], s["scales"], s["out"])
        return {"values": s["out"]}
    if op == "linear":
        q.mxfp4_linear(s["x"], s["codes"], s["scales"], s["out"], s["ws"])
        return {"y": s["out"]}
    if op == "gate_up":
        q.mxfp4_gate_up(s["cfg"], s["weights"], s["x"], s["off"], s["perm"], s["active"], s["n_active"], s["h"], s["ws"])
        return {"h": s["h"]}
    q.mxfp4_down(s["cfg"], s["weights"], s["h"], s["idx"], s["w"], s["off"], s["perm"], s["active"], s["n_active"],
                 s["out"], s["ws"])
    return {"out": s["out"]}


# ------------------------------------------------------------------ plain forms
def _route(s):
    """In 64 bits: scores next to each other decide who is taken."""
    c = s["case"]
    T, E, G, k = c["T"], c["E"], c["G"], c["k"]
    ninf = float("-inf")
    z = s["z"].double()
    ok = z > ninf
    if c["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-z))
    else:
        m = z.amax(1, keepdim=True)
        p = torch.where(ok, torch.exp(z - m), torch.zeros_like(z))
        p = p / p.sum(1, keepdim=True)
    score = p if s["bias"] is None else p + s["bias"].double()
    order = z if s["bias"] is None else score  # without a bias the scores grow with the logits
    if G > 1:
        # scores grow with the logits here too where a group counts by its best expert alone
        by = order if c["group_top"] == 1 or E == G else score
        by = torch.where(ok, by, torch.full_like(by, ninf)).view(T, G, E // G)
        best = torch.sort(by, dim=2, descending=True).values[:, :, :c["group_top"]]
        some = best[:, :, 0] > ninf
        gs = torch.where(best > ninf, best, torch.zeros_like(best)).sum(2)
        gs = torch.where(some, gs, torch.full_like(gs, ninf))
        kept = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :c["Gk"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=z.device).scatter_(1, kept, True)
        ok = ok & keep.repeat_interleave(E // G, 1)
    top = torch.sort(torch.where(ok, order, torch.full_like(order, ninf)), dim=1, descending=True, stable=True)
    idx = top.indices[:, :k]
    there = torch.gather(ok, 1, idx)
    w = torch.where(there, torch.gather(p, 1, idx), torch.zeros((), dtype=p.dtype, device=p.device))
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return {"experts": torch.where(there, idx, torch.full_like(idx, -1)).to(torch.int32), "weights": (w * c["scale"]).float()}


def _unpack(codes, scales):
    """fp32 values of MXFP4 rows: codes [..., n / 2] and E8M0 bytes [..., n / 32]."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    blocks = codes.view(*codes.shape[:-1], -1, 16)
    both = torch.cat([blocks & 15, blocks >> 4], -1)
    u = scales.to(torch.int32)
    scale = torch.where(u == 0, torch.full_like(u, 0x400000), u << 23).view(torch.float32)
    return (table[both.to(torch.int32)] * scale[..., None]).view(*codes.shape[:-1], -1)


def _rounded(x):
    """fp32 values that x [rows, n] is stored as in MXFP4."""
    b = x.float().view(x.shape[0], -1, 32)
    top = b.abs().amax(2, keepdim=True)
    u = (torch.frexp(top).exponent - 1 - 2 + 127).clamp(0, 254)
    u = torch.where(top == 0, torch.zeros_like(u), u)
    up = ((254 - u) << 23).view(torch.float32)  # 2^(127 - u)
    down = torch.where(u == 0, torch.full_like(u, 0x400000), u << 23).view(torch.float32)
    a = (b * up).abs()
    # halfway values go to the neighbour with an even mantissa, values past 6 to 6
    v = 0.5 * ((a > .25).float() + (a >= .75).float() + (a > 1.25).float() + (a >= 1.75).float())
    v = v + (a > 2.5).float() + (a >= 3.5).float() + 2 * (a > 5).float()
    return (torch.sign(b) * v * down).view(x.shape)


def _quantise(s):
    return {"values": _rounded(s["x"]).to(s["x"].dtype)}


def _linear(s):
    return {"y": (_rounded(s["x"]) @ _unpack(s["codes"], s["scales"]).t()).to(s["x"].dtype)}


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
    H, F, k, P = c["H"], c["F"], c["k"], c["T"] * c["k"]
    x, h = _rounded(s["x"]), torch.zeros_like(s["h"])
    for e, rows in _groups(s):
        w = _unpack(s["codes"][e, :F * H].view(2 * F, -1), s["scales"][e, :F * H // 16].view(2 * F, -1))
        gu = (x[rows // k] if e < c["E"] else x) @ w.t()
        g, u = gu[:, :F], gu[:, F:]
        h[rows] = (g / (1 + torch.exp(-g)) * u).to(h.dtype)
    return {"h": h}


def _down(s):
    c = s["case"]
    T, H, F, k = c["T"], c["H"], c["F"], c["k"]
    h = _rounded(s["h"])
    y = torch.zeros((h.shape[0], H), device=h.device)
    for e, rows in _groups(s):
        w = _unpack(s["codes"][e, F * H:].view(H, -1), s["scales"][e, F * H // 16:].view(H, -1))
        y[rows] = h[rows] @ w.t()
    out = (s["w"][:, :, None] * y[:T * k].view(T, k, H)).sum(1)
    return {"out": (out + y[T * k:] if c["shared"] else out).to(s["out"].dtype)}


# ------------------------------------------------------------------ 64 bits, from the definitions
def _e2m1(code):
    """Sign, two exponent bits (bias 1) and a mantissa bit."""
    m, e = (code & 1).double(), ((code >> 1) & 3).double()
    mag = torch.where(e == 0, m / 2, torch.exp2(e - 1) * (1 + m / 2))
    return torch.where(code > 7, -mag, mag)


def _value64(codes, scales):
    out = torch.empty((codes.shape[0], scales.shape[1], 32), dtype=torch.float64, device=codes.device)
    pairs = codes.view(codes.shape[0], -1, 16)
    out[:, :, :16] = _e2m1(pairs % 16)
    out[:, :, 16:] = _e2m1(pairs // 16)
    return (out * torch.exp2(scales.double() - 127)[:, :, None]).view(codes.shape[0], -1)


def _stored64(x):
    """Each block over its power of two, rounded half to even on E2M1's spacing: 1/2 below 2, 1 below 4, 2 above."""
    b = x.double().view(x.shape[0], -1, 32)
    top = b.abs().amax(2, keepdim=True)
    e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
    e = torch.where(torch.exp2(e) > top, e - 1, torch.where(torch.exp2(e + 1) <= top, e + 1, e))
    scale = torch.exp2(torch.clamp(e - 2, min=-127))
    v = b / scale
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
    v = torch.clamp(torch.round(v / step) * step, -6, 6)
    return torch.where(top > 0, v * scale, torch.zeros_like(v)).view(x.shape)


def _route64(s):
    """The choice as ranks: an expert's place is how many come before it."""
    c = s["case"]
    T, E, G, k = c["T"], c["E"], c["G"], c["k"]
    w = torch.zeros((T, k), dtype=torch.float64, device=s["z"].device)
    idx = torch.full((T, k), -1, dtype=torch.int32, device=w.device)
    at = torch.arange(E, device=w.device)
    for lo in range(0, T, 512):
        z = s["z"][lo:lo + 512].double()
        n = z.shape[0]
        p = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(z, 1))
        key = z if s["bias"] is None else p + s["bias"].double()
        ok = ~torch.isneginf(z)
        if G > 1:
            by = key if c["group_top"] == 1 or E == G else p + (0 if s["bias"] is None else s["bias"].double())
            by = by.masked_fill(~ok, float("-inf")).view(n, G, E // G)
            many = min(c["group_top"], E // G)
            best = torch.topk(by, many, dim=2).values
            gs = best[:, :, 0].clone()
            if many > 1:
                gs += torch.nan_to_num(best[:, :, 1], neginf=0.0)
            q = torch.arange(G, device=w.device)
            before = (gs[:, None, :] > gs[:, :, None]) | ((gs[:, None, :] == gs[:, :, None]) & (q[None, None, :] < q[None, :, None]))
            ok &= (before.sum(2) < c["Gk"]).repeat_interleave(E // G, 1)
        key = key.masked_fill(~ok, float("-inf"))
        before = (key[:, None, :] > key[:, :, None]) | ((key[:, None, :] == key[:, :, None]) & (at[None, None, :] < at[None, :, None]))
        rank = before.sum(2)
        row, expert = torch.nonzero(ok & (rank < k), as_tuple=True)
        idx[lo + row, rank[row, expert]] = expert.to(torch.int32)
        w[lo + row, rank[row, expert]] = p[row, expert]
    if c["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True))
    return {"experts": idx, "weights": w * c["scale"]}


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "route":
        return _route64(s)
    if c["op"] == "quantise":
        step = max(1, (1 << 25) // c["cols"])
        return {"values": torch.cat([_stored64(s["x"][r:r + step]) for r in range(0, c["rows"], step)])}
    if c["op"] == "linear":
        return {"y": torch.matmul(_stored64(s["x"]), _value64(s["codes"], s["scales"]).t())}
    T, H, F, k = c["T"], c["H"], c["F"], c["k"]
    a = _stored64(s["x"] if c["op"] == "gate_up" else s["h"])
    owner = s["idx"].reshape(-1)
    out = torch.zeros((T, H) if c["op"] == "down" else s["h"].shape, dtype=torch.float64, device=a.device)
    for e in range(c["E"] + int(c["shared"])):
        pairs = torch.nonzero(owner == e).flatten() if e < c["E"] else torch.arange(T * k, T * k + T, device=a.device)
        if not pairs.numel():
            continue
        token = pairs // k if e < c["E"] else pairs - T * k
        codes, scales = s["codes"][e].view(3, -1), s["scales"][e].view(3, -1)
        if c["op"] == "gate_up":
            g, u = (torch.matmul(a[token], _value64(codes[i].view(F, -1), scales[i].view(F, -1)).t()) for i in (0, 1))
            out[pairs] = g * torch.sigmoid(g) * u
        else:
            y = torch.matmul(a[pairs], _value64(codes[2].view(H, -1), scales[2].view(H, -1)).t())
            out.index_add_(0, token, y if e == c["E"] else y * s["w"].reshape(-1)[pairs, None].double())
    return {"out" if c["op"] == "down" else "h": out}
