"""Cases, plain forms and 64-bit definitions of the expert-layer and dense-epilogue operators.

Operators: routing to experts (`route`, `route_backward`), dispatch and
combine of the routed rows (`group`, `combine`, `combine_backward`), the
experts' block-FP8 products (`experts`) and the block-FP8 product with bias,
activation and residual in its epilogue (`linear`, `linear_backward`).

The plain forms are elementary torch operations in 32 bits; the routing
scores, whose order decides which experts are chosen, are in 64.
"""

import math

import torch

own = False

F8 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # A serving step of 64 tokens through a router of 256 experts in 8 groups, sigmoid scores with a balance bias.
        {"name": "route_decode", "op": "route", "tokens": 64, "experts": 256, "top_k": 8, "score": "sigmoid", "bias": True,
         "n_groups": 8, "top_groups": 4, "group_top": 2, "renormalize": True, "scale": 2.5, "dtype": "f32"},
        # The same router over a prefill of 16384 tokens.
        {"name": "route_prefill", "op": "route", "tokens": 16384, "experts": 256, "top_k": 8, "score": "sigmoid", "bias": True,
         "n_groups": 8, "top_groups": 4, "group_top": 2, "renormalize": True, "scale": 2.5, "dtype": "f32"},
        # Training a softmax router of 128 experts without renormalisation: a dense gradient for every logit.
        {"name": "route_backward", "op": "route_backward", "tokens": 8192, "experts": 128, "top_k": 8, "score": "softmax",
         "renormalize": False, "scale": 1.0, "dtype": "bf16"},
        # The expert order of a prefill's pairs (token, expert), all experts on this GPU.
        {"name": "group_prefill", "op": "group", "tokens": 16384, "top_k": 8, "experts": 256, "first": 0, "local": 256},
        # The experts' rows summed back into a prefill's tokens, onto the residual stream.
        {"name": "combine_prefill", "op": "combine", "tokens": 4096, "top_k": 8, "hidden": 7168, "residual": True, "dtype": "bf16"},
        # Its gradients in training, an odd token count.
        {"name": "combine_backward", "op": "combine_backward", "tokens": 2049, "top_k": 6, "hidden": 4096, "dtype": "bf16"},
        # A serving step's gate and up products on this GPU's 32 experts: about two rows each, bound by the weights.
        {"name": "experts_decode", "op": "experts", "tokens": 64, "rows": 64, "experts": 32, "n": 4096, "k": 7168, "gather": True,
         "bias": False, "act": "silu", "gated": True, "dtype": "bf16"},
        # The down product of a short, ragged batch: rows already in expert order.
        {"name": "experts_ragged", "op": "experts", "tokens": 1999, "rows": 1999, "experts": 32, "n": 7168, "k": 2048, "gather": False,
         "bias": True, "act": "none", "gated": False, "dtype": "bf16"},
        # Gate and up products of a prefill: 16384 rows gathered from 8192 tokens.
        {"name": "experts_prefill", "op": "experts", "tokens": 8192, "rows": 16384, "experts": 32, "n": 4096, "k": 7168, "gather": True,
         "bias": False, "act": "silu", "gated": True, "dtype": "bf16"},
        # A serving step's dense down projection onto the residual stream.
        {"name": "linear_decode", "op": "linear", "m": 16, "n": 7168, "k": 18432, "bias": "bf16", "act": "none", "residual": True,
         "pre": False, "dtype": "bf16"},
        # The dense up projection of a training step, which keeps the value before the activation.
        {"name": "linear_prefill", "op": "linear", "m": 4096, "n": 18432, "k": 7168, "bias": "f32", "act": "gelu_tanh", "residual": False,
         "pre": True, "dtype": "bf16"},
        # Gradients of that epilogue: before the activation, and of the bias.
        {"name": "linear_backward", "op": "linear_backward", "m": 4096, "n": 11008, "act": "gelu_tanh", "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "group", "combine", "combine_backward", "experts", "experts", "linear", "linear",
                     "linear_backward"])
    dt = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("route", "route_backward"):
        experts = rng.choice([8, 16, 40, 64, 100, 128, 160, 256])
        n_groups = rng.choice([g for g in (1, 1, 4, 8) if experts % g == 0 and experts // g >= 2])
        top_groups = rng.randint(1, n_groups)
        c = {"op": op, "tokens": _log(rng, 1, 16384), "experts": experts, "top_k": rng.randint(1, min(10, top_groups * experts // n_groups)),
             "score": rng.choice(["sigmoid", "softmax"]), "renormalize": rng.random() < 0.6, "scale": rng.choice([1.0, 2.5]), "dtype": dt}
        if op == "route":
            c |= {"bias": rng.random() < 0.5, "n_groups": n_groups, "top_groups": top_groups, "group_top": rng.choice([1, 2])}
        return c
    if op == "group":
        experts = rng.choice([8, 60, 128, 256])
        local = rng.choice([experts, experts // 4])
        return {"op": op, "tokens": _log(rng, 1, 16384), "top_k": rng.randint(1, 8), "experts": experts,
                "first": rng.randint(0, experts - local), "local": local}
    if op in ("combine", "combine_backward"):
        c = {"op": op, "tokens": _log(rng, 1, 4096), "top_k": rng.randint(1, 8), "hidden": _log(rng, 64, 5120 if dt != "f32" else 2560), "dtype": dt}
        return c | ({"residual": rng.random() < 0.5} if op == "combine" else {})
    if op == "experts":
        gated = rng.random() < 0.5
        rows = _log(rng, 1, 8192)
        gather = rng.random() < 0.5
        return {"op": op, "tokens": _log(rng, max(1, rows // 8), rows) if gather else rows, "rows": rows, "experts": rng.choice([1, 4, 8, 24, 32]),
                "n": 256 * rng.randint(1, 16) if gated else _log(rng, 64, 4096), "k": 128 * _log(rng, 1, 56), "gather": gather,
                "bias": rng.random() < 0.5, "act": rng.choice(["none", "silu", "gelu", "gelu_tanh", "relu"]), "gated": gated,
                "dtype": rng.choice(["bf16", "bf16", "f16"])}
    if op == "linear":
        return {"op": op, "m": _log(rng, 1, 4096), "n": _log(rng, 32, 11008), "k": 128 * _log(rng, 1, 56), "bias": rng.choice(["", "f32", "bf16"]),
                "act": rng.choice(["none", "silu", "gelu", "gelu_tanh", "relu"]), "residual": rng.random() < 0.5, "pre": rng.random() < 0.3,
                "dtype": rng.choice(["bf16", "bf16", "f16"])}
    return {"op": op, "m": _log(rng, 1, 4096), "n": _log(rng, 64, 8192), "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu"]), "dtype": dt}


# ---------------------------------------------------------------- inputs
def _quantized(x, rows):
    """E4M3 codes and f32 scales of x [..., r, k] in blocks of `rows` x 128 (edge blocks may be partial in r)."""
    *lead, r, k = x.shape
    pad = -r % rows
    xp = torch.nn.functional.pad(x, (0, 0, 0, pad)) if pad else x
    b = xp.reshape(*lead, (r + pad) // rows, rows, k // 128, 128)
    s = b.abs().amax((-3, -1)) / 448.0
    s = torch.where(s == 0, 1.0, s)
    e = (b / s[..., :, None, :, None]).to(F8).view(torch.uint8).reshape(*lead, r + pad, k)
    return e[..., :r, :].contiguous(), s.contiguous()


def _routing(tokens, experts, top_k, rnd):
    """Distinct expert ids per token, drawn with an uneven load, as a router gives them."""
    load = 0.5 * rnd(experts)
    return torch.topk(load + rnd(tokens, experts), top_k, dim=1).indices.to(torch.int32)


def _positions(ids, experts, first, local):
    """Offsets and the position in expert order of each pair (-1 for an expert of another GPU)."""
    flat = ids.reshape(-1).long() - first
    key = torch.where((flat >= 0) & (flat < local), flat, local)
    order = torch.argsort(key, stable=True)
    rank = torch.empty_like(order)
    rank[order] = torch.arange(order.numel(), device=order.device)
    counts = (key[None, :] == torch.arange(local, device=key.device)[:, None]).sum(1)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    pos = torch.where(key < local, rank, -1).reshape(ids.shape)
    return order, offsets.to(torch.int32), pos.to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    rnd = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    op = case["op"]
    dt = DTYPES.get(case.get("dtype"))
    s = {"case": case}
    if op in ("route", "route_backward"):
        t, e = case["tokens"], case["experts"]
        s["logits"] = (1.5 * rnd(t, e)).to(dt)
        if op == "route":
            s["bias"] = 0.05 * rnd(e) if case["bias"] else None
        else:
            s["ids"] = torch.topk(s["logits"].float(), case["top_k"], dim=1).indices.to(torch.int32)
            s["dweights"] = rnd(t, case["top_k"])
    elif op == "group":
        s["ids"] = _routing(case["tokens"], case["experts"], case["top_k"], rnd)
    elif op in ("combine", "combine_backward"):
        t, k, h = case["tokens"], case["top_k"], case["hidden"]
        s["pos"] = torch.randperm(t * k, generator=g, device=dev).to(torch.int32).reshape(t, k)
        w = torch.rand((t, k), generator=g, device=dev) + 0.05
        s["weights"] = w / w.sum(1, keepdim=True)
        s["y"] = rnd(t * k, h).to(dt)
        if op == "combine":
            s["residual"] = rnd(t, h).to(dt) if case["residual"] else None
        else:
            s["dout"] = rnd(t, h).to(dt)
    elif op == "experts":
        p, e, n, k = case["rows"], case["experts"], case["n"], case["k"]
        of = torch.multinomial(torch.softmax(0.4 * rnd(e), 0), p, replacement=True, generator=g)
        counts = torch.bincount(of, minlength=e)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["most"] = int(counts.max())
        s["rows"] = torch.randint(0, case["tokens"], (p,), generator=g, device=dev).to(torch.int32) if case["gather"] else None
        s["a"], s["a_scale"] = _quantized(rnd(case["tokens"], k), 1)
        s["w"], s["w_scale"] = _quantized(rnd(e, n, k).mul_(k ** -0.5), 128)
        s["bias"] = 0.2 * rnd(e, n) if case["bias"] else None
    elif op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["a_scale"] = _quantized(rnd(m, k), 1)
        s["w"], s["w_scale"] = _quantized(rnd(n, k).mul_(k ** -0.5), 128)
        s["bias"] = (0.2 * rnd(n)).to(DTYPES[case["bias"]]) if case["bias"] else None
        s["residual"] = rnd(m, n).to(dt) if case["residual"] else None
    else:
        s["dy"] = rnd(case["m"], case["n"]).to(dt)
        s["pre"] = (1.5 * rnd(case["m"], case["n"])).to(dt)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import dequantize_absmax_reduce_b200 as bq
    c, api = s["case"], bq.api
    op = c["op"]
    if op == "route":
        return api.moe_route(s["logits"], c["top_k"], bias=s["bias"], score=c["score"], n_groups=c["n_groups"], top_groups=c["top_groups"],
                             group_top=c["group_top"], renormalize=c["renormalize"], scale=c["scale"])
    if op == "route_backward":
        return api.moe_route_backward(s["logits"], s["ids"], s["dweights"], score=c["score"], renormalize=c["renormalize"], scale=c["scale"])
    if op == "group":
        return api.moe_group(s["ids"], c["local"], first_expert=c["first"])
    if op == "combine":
        return api.moe_combine(s["y"], s["pos"], s["weights"], residual=s["residual"])
    if op == "combine_backward":
        return api.moe_combine_backward(s["dout"], s["y"], s["pos"], s["weights"])
    if op == "experts":
        return api.fp8_grouped_gemm(s["a"], s["a_scale"], s["offsets"], s["w"], s["w_scale"], rows=s["rows"], bias=s["bias"], act=c["act"],
                                    gated=c["gated"], out_dtype=DTYPES[c["dtype"]])
    if op == "linear":
        return api.fp8_block_gemm_epilogue(s["a"], s["a_scale"], s["w"], s["w_scale"], bias=s["bias"], act=c["act"], residual=s["residual"],
                                           out_dtype=DTYPES[c["dtype"]], save_pre=c["pre"])
    return api.gemm_epilogue_backward(s["dy"], s["pre"], c["act"])


# ---------------------------------------------------------------- plain forms
def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "silu":
        return z * _sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if act == "silu":
        g = _sigmoid(z)
        return g * (1.0 + z * (1.0 - g))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        a = math.sqrt(2.0 / math.pi)
        th = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * a * (1.0 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _softmax(x):
    top = x.amax(-1, keepdim=True)
    p = torch.exp(torch.where(x == top, 0.0, x - top))
    return p / p.sum(-1, keepdim=True)


def _decoded(e, s, rows):
    """f32 values of E4M3 codes [..., r, k] with scales per `rows` x 128."""
    wide = s.repeat_interleave(128, -1)
    if rows > 1:
        wide = wide.repeat_interleave(rows, -2)[..., :e.shape[-2], :]
    return e.view(F8).float() * wide


def _plain(s):
    c = s["case"]
    op = c["op"]
    dt = DTYPES.get(c.get("dtype"))
    if op == "route":
        lowest = -math.inf
        x = s["logits"].double()
        bad = torch.isnan(x)
        x = torch.where(bad, lowest, x)
        score = _sigmoid(x) if c["score"] == "sigmoid" else _softmax(x)
        v = x if s["bias"] is None else score + s["bias"].double()
        v = torch.where(torch.isnan(v) | (x == lowest), lowest, v)
        by_group = v.reshape(x.shape[0], c["n_groups"], -1)
        best = torch.sort(by_group, dim=-1, descending=True).values[..., :c["group_top"]]
        value = torch.where((best == lowest).all(-1), lowest, torch.where(best == lowest, 0.0, best).sum(-1))
        order = torch.sort(value, dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        kept = torch.zeros_like(value, dtype=torch.bool).scatter_(1, order, True)
        v = torch.where(kept[..., None], by_group, lowest).reshape(x.shape)
        top = torch.sort(v, dim=-1, descending=True, stable=True)
        ids = top.indices[:, :c["top_k"]]
        there = top.values[:, :c["top_k"]] > lowest
        w = torch.where(there, score.gather(1, ids), 0.0)
        if c["renormalize"]:
            w = w / w.sum(-1, keepdim=True).clamp_min(1e-300)
        w = torch.where(bad.any(-1, keepdim=True), math.nan, w * c["scale"])
        return torch.where(there, ids, -1).to(torch.int32), w.float()
    if op == "route_backward":
        x, g = s["logits"].float(), s["dweights"]
        at = s["ids"].long()
        score = _sigmoid(x) if c["score"] == "sigmoid" else _softmax(x)
        chosen = score.gather(1, at)
        if c["renormalize"]:
            d = chosen.sum(-1, keepdim=True)
            gs = c["scale"] * (g - (g * chosen).sum(-1, keepdim=True) / d) / d
        else:
            gs = c["scale"] * g
        full = torch.zeros_like(x).scatter_add_(1, at, gs)
        if c["score"] == "sigmoid":
            return (full * score * (1.0 - score)).to(dt)
        return (score * (full - (gs * chosen).sum(-1, keepdim=True))).to(dt)
    if op == "group":
        order, offsets, pos = _positions(s["ids"], c["experts"], c["first"], c["local"])
        rows = torch.where(torch.arange(order.numel(), device=order.device) < offsets[-1], order // c["top_k"], -1)
        return offsets, rows.to(torch.int32), pos
    if op == "combine":
        y = (s["y"][s["pos"].long()].float() * s["weights"][..., None]).sum(1)
        return (y if s["residual"] is None else y + s["residual"].float()).to(dt)
    if op == "combine_backward":
        at, dout = s["pos"].long(), s["dout"].float()
        dy = torch.empty_like(s["y"])
        dy[at.reshape(-1)] = (dout[:, None, :] * s["weights"][..., None]).to(dt).reshape(-1, dout.shape[1])
        return dy, (s["y"][at].float() * dout[:, None, :]).sum(-1)
    if op == "experts":
        off = s["offsets"].long()
        slot = torch.arange(max(1, s["most"]), device=off.device)
        p = torch.arange(c["rows"], device=off.device)
        at = (off[:-1, None] + slot).clamp_max(c["rows"] - 1)
        if s["rows"] is not None:
            at = s["rows"].long()[at]
        z = torch.bmm(_decoded(s["a"], s["a_scale"], 1)[at], _decoded(s["w"], s["w_scale"], 128).transpose(1, 2))
        e = torch.searchsorted(off, p, right=True) - 1
        z = z[e, p - off[e]]
        if s["bias"] is not None:
            z = z + s["bias"][e]
        if c["gated"]:
            half = c["n"] // 2
            return (_act(z[:, :half], c["act"]) * z[:, half:]).to(dt)
        return _act(z, c["act"]).to(dt)
    if op == "linear":
        z = _decoded(s["a"], s["a_scale"], 1) @ _decoded(s["w"], s["w_scale"], 128).t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        out = _act(z, c["act"])
        if s["residual"] is not None:
            out = out + s["residual"].float()
        return (out.to(dt), z.to(dt)) if c["pre"] else out.to(dt)
    dz = s["dy"].float() * _act_slope(s["pre"].float(), c["act"])
    return dz.to(dt), dz.sum(0)


# ---------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = torch.float64
    tanh_a = math.sqrt(2.0 / math.pi)

    def act(z):
        return {"none": lambda: z, "relu": lambda: z.clamp_min(0), "silu": lambda: z / (1 + torch.exp(-z)),
                "gelu": lambda: z * 0.5 * torch.erfc(-z / math.sqrt(2.0)),
                "gelu_tanh": lambda: z / (1 + torch.exp(-2 * tanh_a * (z + 0.044715 * z ** 3)))}[case["act"]]()

    def value(e, sc, rows):
        v = e.view(F8).to(f)
        for b in range(v.shape[-1] // 128):
            cols = sc[..., b].to(f).repeat_interleave(rows, 0)[:v.shape[0]]
            v[:, 128 * b:128 * (b + 1)] *= cols[:, None]
        return v

    if op == "route":
        x = s["logits"].to(f)
        score = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, -1)
        v = x.clone() if s["bias"] is None else score + s["bias"].to(f)
        size = case["experts"] // case["n_groups"]
        if case["n_groups"] > 1:
            groups = torch.stack([torch.topk(v[:, j * size:(j + 1) * size], min(size, case["group_top"])).values.sum(1)
                                  for j in range(case["n_groups"])], 1)
            for j in range(case["n_groups"]):
                ahead = (groups > groups[:, j:j + 1]).sum(1) + (groups[:, :j] == groups[:, j:j + 1]).sum(1)
                v[:, j * size:(j + 1) * size].masked_fill_((ahead >= case["top_groups"])[:, None], -math.inf)
        ids = []
        for _ in range(case["top_k"]):
            best = (v == v.amax(1, keepdim=True)).to(torch.int32).argmax(1, keepdim=True)  # the first of equal ones
            ids.append(best)
            v = v.scatter(1, best, -math.inf)
        ids = torch.cat(ids, 1)
        w = torch.gather(score, 1, ids)
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        return ids, w * case["scale"]
    if op == "route_backward":
        x = s["logits"].to(f).requires_grad_(True)
        score = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, -1)
        w = torch.gather(score, 1, s["ids"].long())
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        (case["scale"] * w * s["dweights"].to(f)).sum().backward()
        return x.grad
    if op == "group":
        return None
    if op == "combine":
        out = torch.zeros((case["tokens"], case["hidden"]), dtype=f, device="cuda") if s["residual"] is None else s["residual"].to(f)
        for j in range(case["top_k"]):
            out += s["weights"][:, j:j + 1].to(f) * s["y"][s["pos"][:, j].long()].to(f)
        return out
    if op == "combine_backward":
        dy = torch.zeros(s["y"].shape, dtype=f, device="cuda")
        dw = []
        for j in range(case["top_k"]):
            at = s["pos"][:, j].long()
            dy[at] = s["weights"][:, j:j + 1].to(f) * s["dout"].to(f)
            dw.append((s["y"][at].to(f) * s["dout"].to(f)).sum(1))
        return dy, torch.stack(dw, 1)
    if op == "experts":
        off = s["offsets"].tolist()
        parts = []
        for e in range(case["experts"]):
            if off[e] == off[e + 1]:
                continue
            here = slice(off[e], off[e + 1]) if s["rows"] is None else s["rows"][off[e]:off[e + 1]].long()
            z = value(s["a"][here], s["a_scale"][here], 1) @ value(s["w"][e], s["w_scale"][e], 128).t()
            if s["bias"] is not None:
                z = z + s["bias"][e].to(f)
            parts.append(act(z[:, :case["n"] // 2]) * z[:, case["n"] // 2:] if case["gated"] else act(z))
        return torch.cat(parts)
    if op == "linear":
        z = value(s["a"], s["a_scale"], 1) @ value(s["w"], s["w_scale"], 128).t()
        if s["bias"] is not None:
            z = z + s["bias"].to(f)
        out = act(z)
        if s["residual"] is not None:
            out = out + s["residual"].to(f)
        return (out, z) if case["pre"] else out
    z = s["pre"].to(f).requires_grad_(True)
    dz, = torch.autograd.grad(act(z), z, s["dy"].to(f))
    return dz, dz.sum(0)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    es = SIZE.get(case.get("dtype"), 0)
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        return {"bytes": t * e * es + t * k * 8 + (4 * e if case["bias"] else 0), "flops": 6 * t * e}
    if op == "route_backward":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        dense = case["score"] == "softmax" and not case["renormalize"]
        return {"bytes": t * e * es + (t * e * es if dense else t * k * es) + t * k * 8, "flops": 6 * t * e}
    if op == "group":
        n = case["tokens"] * case["top_k"]
        return {"bytes": 12 * n + 4 * (case["local"] + 1), "flops": 0}
    if op in ("combine", "combine_backward"):
        t, k, h = case["tokens"], case["top_k"], case["hidden"]
        if op == "combine":
            return {"bytes": es * t * h * (k + 1 + (1 if case["residual"] else 0)) + 8 * t * k, "flops": 2 * t * k * h}
        return {"bytes": es * t * h * (2 * k + 1) + 12 * t * k, "flops": 3 * t * k * h}
    if op == "experts":
        p, e, n, k = case["rows"], case["experts"], case["n"], case["k"]
        busy = e * (1.0 - (1.0 - 1.0 / e) ** p)      # experts that an even load reaches
        width = n // 2 if case["gated"] else n
        wk = n * k + 4 * math.ceil(n / 128) * (k // 128) + (4 * n if case["bias"] else 0)
        return {"bytes": min(p, case["tokens"]) * (k + k // 32) + busy * wk + p * width * es + (4 * p if case["gather"] else 0),
                "flops": 2 * p * n * k}
    m, n = case["m"], case["n"]
    if op == "linear":
        k = case["k"]
        out = m * n * es * (1 + (1 if case["residual"] else 0) + (1 if case["pre"] else 0))
        return {"bytes": m * (k + k // 32) + n * k + 4 * math.ceil(n / 128) * (k // 128) + SIZE.get(case["bias"], 0) * n + out,
                "flops": 2 * m * n * k}
    return {"bytes": 3 * m * n * es + 4 * n, "flops": 8 * m * n}
