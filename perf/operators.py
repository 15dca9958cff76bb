"""Cases of the training operators around the optimizer step: 8-bit activation
checkpoints (pack and unpack, SwiGLU through them, weight gradients out of
them) and routing to experts (forward with its dispatch lists, backward with
the balance bias step).

``run`` computes a case in plain torch operations, or through the package when
``own`` is true.  ``exact`` computes it in 64 bits from the definitions.

A checkpoint stores a row in blocks of 32 columns: one byte b per block, worth
2^(b - 127), and one 8-bit code per value (e4m3, or a whole number in
[-127, 127]).  The exponent is the smallest one, not below -111, that keeps the
block's largest magnitude within the codes' range.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 32
LARGEST = {"e4m3": 448.0, "int8": 127.0}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one row of the 192-wide model in fp32: the call's own cost
        {"name": "checkpoint one row", "kind": "checkpoint", "tokens": 1, "cols": 192, "dtype": "f32", "format": "int8"},
        # the attention input of a 1024-wide layer over a batch of 16 sequences of 2048
        {"name": "checkpoint batch", "kind": "checkpoint", "tokens": 32768, "cols": 1024, "dtype": "bf16", "format": "e4m3"},
        # the small model's MLP width in fp32, an odd number of tokens
        {"name": "swiglu small", "kind": "swiglu", "tokens": 1999, "cols": 768, "dtype": "f32", "format": "int8"},
        # gate and up of the 1024 x 2816 MLP over 16384 tokens, forward and backward
        {"name": "swiglu layer", "kind": "swiglu", "tokens": 16384, "cols": 2816, "dtype": "bf16", "format": "e4m3"},
        # the small model's MLP matrix: few output tiles, a long sum over tokens
        {"name": "wgrad small matrix", "kind": "wgrad", "tokens": 8192, "outs": 192, "cols": 768, "dtype": "bf16",
         "format": "int8", "out": "f32", "transposed": False},
        # the 1024 x 2816 projections of the 430M set over 16384 tokens
        {"name": "wgrad layer", "kind": "wgrad", "tokens": 16384, "outs": 2816, "cols": 1024, "dtype": "bf16",
         "format": "e4m3", "out": "bf16", "transposed": False},
        # a few hundred tokens over 8 experts, odd widths, some experts idle, fp16
        {"name": "wgrad experts few tokens", "kind": "experts", "tokens": 301, "outs": 333, "cols": 517, "experts": 8,
         "top_k": 2, "skew": 2.0, "dtype": "f16", "format": "int8", "out": "f32", "transposed": False},
        # the MoE block's up projections, 64 of 2048 x 1408, six experts a token
        {"name": "wgrad experts block", "kind": "experts", "tokens": 8192, "outs": 1408, "cols": 2048, "experts": 64,
         "top_k": 6, "skew": 0.3, "dtype": "bf16", "format": "e4m3", "out": "bf16", "transposed": True},
        # a handful of tokens: the latency of a routing call
        {"name": "route few tokens", "kind": "route", "tokens": 5, "experts": 64, "top_k": 6, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "renormalize": True, "scale": 1.0, "padding": 0.0, "dtype": "bf16"},
        # a padded batch over 256 experts in 8 groups with a balance bias
        {"name": "route batch groups", "kind": "route", "tokens": 16384, "experts": 256, "top_k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "renormalize": True, "scale": 2.5, "padding": 0.04, "dtype": "f32"},
        # backward of a small routing call with renormalised weights
        {"name": "route backward small", "kind": "route_backward", "tokens": 130, "experts": 64, "top_k": 6, "score": "sigmoid",
         "renormalize": True, "scale": 1.0, "padding": 0.1, "dtype": "f32"},
        # backward through the softmax over all 64 experts of the MoE block
        {"name": "route backward batch", "kind": "route_backward", "tokens": 32768, "experts": 64, "top_k": 6, "score": "softmax",
         "renormalize": False, "scale": 1.0, "padding": 0.02, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(("checkpoint", "swiglu", "wgrad", "experts", "route", "route_backward"))
    dtype = rng.choice(("f32", "bf16", "f16"))
    fmt = rng.choice(("e4m3", "int8"))
    if kind in ("checkpoint", "swiglu"):
        cols = _log(rng, 17, 4500)
        return {"kind": kind, "tokens": _log(rng, 1, min(32768, (32 << 20) // cols)), "cols": cols, "dtype": dtype, "format": fmt}
    if kind in ("wgrad", "experts"):
        case = {"kind": kind, "outs": _log(rng, 40, 2900), "cols": _log(rng, 40, 2900), "dtype": rng.choice(("bf16", "f16")),
                "format": fmt, "out": rng.choice(("f32", "bf16", "f16")), "transposed": rng.random() < 0.5}
        most = (45 << 30) // (case["outs"] * case["cols"])
        if kind == "wgrad":
            return {**case, "tokens": _log(rng, 1, min(32768, most))}
        top_k = rng.randint(1, 6)
        experts = _log(rng, max(4, top_k), max(8, min(64, (200 << 20) // (case["outs"] * case["cols"]))))
        return {**case, "experts": experts, "top_k": top_k, "skew": round(rng.uniform(0.0, 2.5), 3),
                "tokens": _log(rng, 3, min(8192, most // top_k))}
    groups = rng.choice((1, 1, 4, 8))
    experts = groups * _log(rng, 8, 256 // groups)
    score = rng.choice(("softmax", "sigmoid"))
    case = {"kind": kind, "tokens": _log(rng, 1, (4 << 20) // experts), "experts": experts, "top_k": rng.randint(1, 8), "score": score,
            "renormalize": rng.random() < 0.6, "scale": rng.choice((1.0, 2.5)), "padding": rng.choice((0.0, 0.05, 0.3)), "dtype": dtype}
    if kind == "route":
        case.update(bias=rng.random() < 0.6, groups=groups, top_groups=rng.randint(1, groups))
    return case


# ---------------------------------------------------------------- inputs

def _activations(tokens, cols, dtype, gen):
    """Normal values with a few channels far above the others, as activations have."""
    x = torch.randn(tokens, cols, generator=gen, device="cuda")
    channel = torch.exp(0.8 * torch.randn(cols, generator=gen, device="cuda"))
    return (x * channel).to(dtype)


def _choose(logits, top_k):
    return torch.topk(logits, top_k, dim=1).indices


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    kind, tokens = case["kind"], case["tokens"]
    dtype = DTYPES[case["dtype"]]
    state = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if kind == "checkpoint":
        state["x"] = _activations(tokens, case["cols"], dtype, gen)
    elif kind == "swiglu":
        # gate and up are the halves of one projection's output
        both = _activations(tokens, 2 * case["cols"], dtype, gen)
        state["gate"], state["up"] = both[:, :case["cols"]], both[:, case["cols"]:]
        state["grad_h"] = (0.01 * normal(tokens, case["cols"])).to(dtype)
    elif kind in ("wgrad", "experts"):
        x = _activations(tokens, case["cols"], dtype, gen)
        state["codes"], state["scales"] = _pack(x, case["format"])
        slots = tokens
        if kind == "experts":
            lean = case["skew"] * normal(case["experts"])
            chosen = _choose(normal(tokens, case["experts"]) + lean, case["top_k"]).reshape(-1)
            slots = chosen.numel()
            sizes = torch.bincount(chosen, minlength=case["experts"])
            state["rows"] = (torch.argsort(chosen, stable=True) // case["top_k"]).to(torch.int32)
            state["offsets"] = torch.nn.functional.pad(torch.cumsum(sizes, 0), (1, 0)).to(torch.int32)
            state["sizes"] = sizes.tolist()
        state["grad_y"] = (0.01 * normal(slots, case["outs"])).to(dtype)
    else:
        experts = case["experts"]
        state["logits"] = (1.5 * normal(tokens, experts)).to(dtype)
        # padded batches: the last positions of some sequences hold no token
        state["mask"] = (torch.rand(tokens, generator=gen, device="cuda") >= case["padding"]) if case["padding"] else None
        if kind == "route":
            state["bias"] = 0.05 * normal(experts) if case["bias"] else None
        else:
            chosen = _choose(state["logits"].float() + 0.05 * normal(experts), case["top_k"])
            if state["mask"] is not None:
                chosen = torch.where(state["mask"][:, None], chosen, -1)
            state["experts"] = chosen.to(torch.int32).contiguous()
            state["grad_weights"] = 0.1 * normal(tokens, case["top_k"])
            state["bias"] = 0.05 * normal(experts)
            state["counts"] = torch.bincount(chosen.reshape(-1) + 1, minlength=experts + 1)[1:].to(torch.int32)
    return state


# ---------------------------------------------------------------- plain forms

def _pack(x, fmt):
    """Codes (a byte a value, rows filled up to 16) and exponent bytes of x's rows."""
    tokens, cols = x.shape
    blocks = -(-cols // BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, blocks * BLOCK - cols)).view(tokens, blocks, BLOCK)
    top = v.abs().amax(dim=2, keepdim=True)
    fraction, exponent = torch.frexp(top)
    largest = 0.875 if fmt == "e4m3" else 127.0 / 128.0
    exponent = (exponent - (9 if fmt == "e4m3" else 7) + (fraction > largest)).clamp(min=-111)
    exponent = torch.where(top == 0, -111, exponent)
    v = torch.ldexp(v, -exponent)
    if fmt == "int8":
        codes = torch.round(v).to(torch.int8).view(torch.uint8)
    else:
        codes = v.to(torch.float8_e4m3fn).view(torch.uint8)
    codes = codes.reshape(tokens, blocks * BLOCK)[:, :-(-cols // 16) * 16].contiguous()
    return codes, (exponent.squeeze(2) + 127).to(torch.uint8)


def _unpack(codes, scales, cols, fmt):
    tokens, blocks = scales.shape
    v = codes[:, :cols].contiguous()
    v = (v.view(torch.int8) if fmt == "int8" else v.view(torch.float8_e4m3fn)).float()
    step = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127)
    return v * step.repeat_interleave(BLOCK, dim=1)[:, :cols]


def _plain_swiglu(state, case):
    gate, up, fmt = state["gate"], state["up"], case["format"]
    dtype = gate.dtype
    h = (gate.float() * torch.sigmoid(gate.float()) * up.float()).to(dtype)
    g, u = (_unpack(*_pack(t, fmt), case["cols"], fmt) for t in (gate, up))
    s = torch.sigmoid(g)
    d = state["grad_h"].float()
    return {"h": h, "grad_gate": (d * u * s * (1 + g * (1 - s))).to(dtype), "grad_up": (d * g * s).to(dtype),
            "h_again": (g * s * u).to(dtype)}


def _plain_wgrad(state, case):
    x = _unpack(state["codes"], state["scales"], case["cols"], case["format"])
    if case["dtype"] == "f16":
        x = x.clamp(-65504.0, 65504.0).half().float()
    dy = state["grad_y"].float()
    if case["kind"] == "wgrad":
        return (x.t() @ dy if case["transposed"] else dy.t() @ x).to(DTYPES[case["out"]])
    parts = zip(dy.split(state["sizes"]), x[state["rows"].long()].split(state["sizes"]))
    # one large product an expert, as a program without a grouped product runs them
    return torch.stack([(b.t() @ a if case["transposed"] else a.t() @ b) for a, b in parts]).to(DTYPES[case["out"]])


def _scores(logits, score):
    return torch.softmax(logits, dim=1) if score == "softmax" else torch.sigmoid(logits)


def _plain_route(state, case):
    tokens, experts, top_k = case["tokens"], case["experts"], case["top_k"]
    logits = state["logits"].double()
    s = _scores(logits, case["score"])
    choice = s if state["bias"] is None else s + state["bias"].double()
    order_by = logits if state["bias"] is None else choice
    groups, keep = case["groups"], case["top_groups"]
    if keep < groups:
        size = experts // groups
        best = torch.topk(choice.view(tokens, groups, size), min(2, size), dim=2).values.sum(dim=2)
        ranked = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :keep]
        kept = torch.zeros(tokens, groups, dtype=torch.bool, device=s.device).scatter_(1, ranked, True)
        order_by = order_by.masked_fill(~kept.repeat_interleave(size, dim=1), -math.inf)
    ids = torch.sort(order_by, dim=1, descending=True, stable=True).indices[:, :top_k]
    dead = torch.isneginf(order_by.gather(1, ids))
    if state["mask"] is not None:
        dead = dead | ~state["mask"][:, None]
    w = s.gather(1, ids).masked_fill(dead, 0.0)
    if case["renormalize"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    ids = ids.masked_fill(dead, -1)
    flat = ids.reshape(-1)
    counts = torch.bincount(flat + 1, minlength=experts + 1)[1:]
    order = torch.argsort(torch.where(flat < 0, experts, flat), stable=True)
    order = torch.where(torch.arange(order.numel(), device=order.device) < counts.sum(), order, -1)
    return {"experts": ids.to(torch.int32), "weights": (w * case["scale"]).float(), "counts": counts.to(torch.int32),
            "offsets": torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0)).to(torch.int32),
            "order": order.to(torch.int32), "rows": torch.div(order, top_k, rounding_mode="floor").to(torch.int32)}


def _plain_route_backward(state, case):
    ids, dw = state["experts"].long(), state["grad_weights"]
    live = ids >= 0
    ids = ids.clamp(min=0)
    s = _scores(state["logits"].float(), case["score"])
    picked = s.gather(1, ids) * live
    ds = dw * live
    if case["renormalize"]:
        total = picked.sum(dim=1, keepdim=True)
        ds = torch.where(total > 0, (ds - (ds * picked).sum(dim=1, keepdim=True) / total) / total, 0.0) * live
    ds = torch.zeros_like(s).scatter_add_(1, ids, ds * case["scale"])
    if case["score"] == "softmax":
        grad = s * (ds - (ds * s).sum(dim=1, keepdim=True))
    else:
        grad = s * (1 - s) * ds
    counts = state["counts"].long()
    state["bias"].add_(torch.sign(counts.sum() - case["experts"] * counts).float(), alpha=0.001)
    return {"grad_logits": grad.to(state["logits"].dtype), "bias": state["bias"]}


def run(state):
    case = state["case"]
    kind = case["kind"]
    if own:
        return _run_own(state, case, kind)
    if kind == "checkpoint":
        return _unpack(*_pack(state["x"], case["format"]), case["cols"], case["format"]).to(state["x"].dtype)
    if kind == "swiglu":
        return _plain_swiglu(state, case)
    if kind in ("wgrad", "experts"):
        return _plain_wgrad(state, case)
    return (_plain_route if kind == "route" else _plain_route_backward)(state, case)


# ---------------------------------------------------------------- the package's operators

def _run_own(state, case, kind):
    import newton_schulz_matrix_momentum_amd as nsm
    if kind == "checkpoint":
        return nsm.checkpoint_unpack(nsm.checkpoint_pack(state["x"], format=case["format"]), dtype=state["x"].dtype)
    if kind == "swiglu":
        h, gate, up = nsm.checkpoint_swiglu(state["gate"], state["up"], format=case["format"])
        grad_gate, grad_up, again = nsm.checkpoint_swiglu_backward(state["grad_h"], gate, up)
        return {"h": h, "grad_gate": grad_gate, "grad_up": grad_up, "h_again": again}
    if kind in ("wgrad", "experts"):
        saved = nsm.Checkpoint(state["codes"], state["scales"], case["cols"], case["format"])
        return nsm.checkpoint_wgrad(state["grad_y"], saved, out_dtype=DTYPES[case["out"]], transposed=case["transposed"],
                                    offsets=state.get("offsets"), rows=state.get("rows"))
    if kind == "route":
        r = nsm.route(state["logits"], case["top_k"], bias=state["bias"], score=case["score"], groups=case["groups"],
                      top_groups=case["top_groups"], renormalize=case["renormalize"], scale=case["scale"], token_mask=state["mask"])
        return {"experts": r.experts, "weights": r.weights, "counts": r.counts, "offsets": r.offsets, "order": r.order, "rows": r.rows}
    grad = nsm.route_backward(state["grad_weights"], state["logits"], state["experts"], score=case["score"],
                              renormalize=case["renormalize"], scale=case["scale"])
    nsm.balance_step(state["bias"], state["counts"], rate=0.001)
    return {"grad_logits": grad, "bias": state["bias"]}


# ---------------------------------------------------------------- work

def work(case):
    kind, tokens = case["kind"], case["tokens"]
    es = BYTES[case["dtype"]]
    code = 1 + 1 / BLOCK
    if kind == "checkpoint":
        n = tokens * case["cols"]
        return {"bytes": n * (2 * es + 2 * code), "flops": 4 * n}
    if kind == "swiglu":
        n = tokens * case["cols"]
        return {"bytes": n * (7 * es + 4 * code), "flops": 30 * n}
    if kind in ("wgrad", "experts"):
        slots = tokens * case.get("top_k", 1)
        matrix = case["outs"] * case["cols"]
        lists = 4 * (slots + case["experts"] + 1) if kind == "experts" else 0
        return {"bytes": slots * case["outs"] * es + tokens * case["cols"] * code + case.get("experts", 1) * matrix * BYTES[case["out"]] + lists,
                "flops": 2 * slots * matrix}
    experts, slots = case["experts"], tokens * case["top_k"]
    padded = tokens if case["padding"] else 0
    if kind == "route":
        return {"bytes": tokens * experts * es + 16 * slots + padded + 8 * experts + (4 * experts if case["bias"] else 0),
                "flops": 20 * tokens * experts}
    # renormalised softmax weights and sigmoid scores need the chosen logits alone
    dense = case["score"] == "softmax" and not case["renormalize"]
    read = tokens * experts * es if dense else slots * es
    return {"bytes": read + tokens * experts * es + 8 * slots + 12 * experts, "flops": 20 * tokens * experts}


# ---------------------------------------------------------------- 64 bits, from the definitions

def _value_table(fmt):
    """The value of each of the 256 codes."""
    values = []
    for c in range(256):
        if fmt == "int8":
            values.append(float(c - 256 if c > 127 else c))
        else:
            sign, field, low = -1.0 if c & 128 else 1.0, (c >> 3) & 15, c & 7
            values.append(sign * (math.ldexp(8 + low, field - 10) if field else math.ldexp(low, -9)))
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def _read_back(x, fmt):
    """What a checkpoint of x stands for: each block on the grid of its own exponent."""
    tokens, cols = x.shape
    x = x.double()
    blocks = [x[:, i:i + BLOCK] for i in range(0, cols, BLOCK)]
    out = []
    for v in blocks:
        ratio = v.abs().amax(dim=1, keepdim=True) / LARGEST[fmt]
        e = torch.ceil(torch.log2(ratio.clamp(min=2.0 ** -200)))
        e = torch.where(ratio > torch.exp2(e), e + 1, e)           # where the logarithm rounded across a power
        e = torch.where(ratio <= torch.exp2(e - 1), e - 1, e).clamp(min=-111)
        y = v * torch.exp2(-e)
        if fmt == "int8":
            grid = torch.ones_like(y)
        else:
            level = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20)))
            level = torch.where(y.abs() >= torch.exp2(level + 1), level + 1, level).clamp(min=-6)
            grid = torch.exp2(level - 3)
        out.append(torch.round(y / grid) * grid * torch.exp2(e))
    return torch.cat(out, dim=1)


def exact(case, seed):
    state = prepare(case, seed)
    kind = case["kind"]
    if kind == "checkpoint":
        return _read_back(state["x"], case["format"])
    if kind == "swiglu":
        g, u = state["gate"].double(), state["up"].double()
        h = g * u / (1 + torch.exp(-g))
        g, u = (_read_back(t, case["format"]) for t in (state["gate"], state["up"]))
        d, s = state["grad_h"].double(), 1 / (1 + torch.exp(-g))
        return {"h": h, "grad_gate": d * u * (s + g * s / (1 + torch.exp(g))), "grad_up": d * g * s, "h_again": g * u * s}
    if kind in ("wgrad", "experts"):
        x = _value_table(case["format"])[state["codes"][:, :case["cols"]].long()]
        column = torch.arange(case["cols"], device="cuda") // BLOCK
        x = x * torch.exp2(state["scales"].double() - 127)[:, column]
        d = state["grad_y"].double()
        if kind == "wgrad":
            return x.t() @ d if case["transposed"] else d.t() @ x
        out, at = [], 0
        for n in state["sizes"]:
            a, b = d[at:at + n], x[state["rows"][at:at + n].long()]
            out.append(b.t() @ a if case["transposed"] else a.t() @ b)
            at += n
        return torch.stack(out)
    logits = state["logits"].double()
    if case["score"] == "softmax":
        s = torch.exp(logits - torch.logsumexp(logits, dim=1, keepdim=True))
    else:
        s = 1 / (1 + torch.exp(-logits))
    live = torch.ones(case["tokens"], 1, dtype=torch.bool, device="cuda") if state["mask"] is None else state["mask"][:, None]
    if kind == "route":
        c = s if state["bias"] is None else s + state["bias"].double()
        by = c if state["bias"] is not None else logits
        groups = case["groups"]
        if case["top_groups"] < groups:
            top = c.view(case["tokens"], groups, -1).sort(dim=2, descending=True).values[:, :, :2].sum(dim=2)
            # a group stays where fewer than top_groups others come before it
            index = torch.arange(groups, device="cuda")
            ahead = (top[:, None, :] > top[:, :, None]) | ((top[:, None, :] == top[:, :, None]) & (index[None, :] < index[:, None]))
            stays = ahead.sum(dim=2) < case["top_groups"]
            by = torch.where(stays.repeat_interleave(case["experts"] // groups, dim=1), by, -math.inf)
        w = s.gather(1, by.sort(dim=1, descending=True, stable=True).indices[:, :case["top_k"]])
        if case["renormalize"]:
            w = w / w.sum(dim=1, keepdim=True)
        return {"experts": None, "weights": torch.where(live, case["scale"] * w, 0.0), "counts": None, "offsets": None,
                "order": None, "rows": None}
    ids, dw = state["experts"].long().clamp(min=0), state["grad_weights"].double()
    p = s.gather(1, ids)
    if case["renormalize"]:
        z = p.sum(dim=1, keepdim=True)
        ds = case["scale"] * (dw / z - (dw * p).sum(dim=1, keepdim=True) / z ** 2)
    else:
        ds = case["scale"] * dw
    grad = torch.zeros_like(s)
    if case["score"] == "softmax":
        grad.scatter_add_(1, ids, p * ds)
        grad -= s * (ds * p).sum(dim=1, keepdim=True)
    else:
        grad.scatter_add_(1, ids, p * (1 - p) * ds)
    counts = state["counts"].double()
    return {"grad_logits": torch.where(live, grad, 0.0), "bias": state["bias"].double() + 0.001 * torch.sign(counts.mean() - counts)}
