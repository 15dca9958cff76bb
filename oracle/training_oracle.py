"""fp64 definitions of the training operators (include/muon.h), in plain numpy.

Written from the formulas, sharing no code with the library: 8-bit
checkpoints, SwiGLU through them, weight gradients, routing to experts with
its gradient, and the balance step.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 32
LARGEST = {"e4m3": 448.0, "int8": 127.0}


def code_values(fmt):
    """The value of each of the 256 code bytes (e4m3's two NaN codes as NaN)."""
    out = np.empty(256)
    for c in range(256):
        if fmt == "int8":
            out[c] = c - 256 if c >= 128 else c
            continue
        sign, field, low = (-1.0 if c >= 128 else 1.0), (c >> 3) & 15, c & 7
        if field == 15 and low == 7:
            out[c] = math.nan
        else:
            out[c] = sign * (math.ldexp(low, -9) if field == 0 else math.ldexp(8 + low, field - 10))
    return out


def _block_exponent(top, fmt):
    """Smallest e >= -111 with top <= Q 2^e, limited so that Q 2^e stays below 2^128."""
    q = LARGEST[fmt]
    e = -111
    if top > 0.0:
        e = max(e, math.frexp(top / q)[1] - 1)
        while top > math.ldexp(q, e):
            e += 1
    return min(e, 119 if fmt == "e4m3" else 121)


def _round_code(y, fmt):
    """y (|y| <= Q) to the nearest code value, ties to the even code."""
    if fmt == "int8":
        return np.rint(y)
    _, exponent = np.frexp(y)
    step = np.ldexp(1.0, np.maximum(exponent - 1, -6) - 3)
    return np.rint(y / step) * step


def checkpoint(x, fmt):
    """(values the checkpoint stands for, exponent bytes) of a 2-D float array."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    out = np.empty_like(x)
    scales = np.empty((rows, blocks), dtype=np.uint8)
    for r in range(rows):
        for b in range(blocks):
            v = x[r, b * BLOCK:(b + 1) * BLOCK]
            if not np.isfinite(v).all():
                scales[r, b] = 255
                out[r, b * BLOCK:(b + 1) * BLOCK] = math.nan
                continue
            e = _block_exponent(float(np.abs(v).max()), fmt)
            q = LARGEST[fmt]
            out[r, b * BLOCK:(b + 1) * BLOCK] = np.ldexp(_round_code(np.clip(np.ldexp(v, -e), -q, q), fmt), e)
            scales[r, b] = e + 127
    return out, scales


def values(codes, scales, cols, fmt):
    """What stored codes and exponent bytes stand for."""
    q = code_values(fmt)[np.asarray(codes)[:, :cols]]
    s = np.ldexp(1.0, np.asarray(scales).astype(np.int64) - 127)
    s[np.asarray(scales) == 255] = math.nan
    return q * np.repeat(s, BLOCK, axis=1)[:, :cols]


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(x, dtype=np.float64)))


def swiglu(gate, up):
    return gate * sigmoid(gate) * up


def swiglu_backward(grad_h, gate, up):
    """(grad_gate, grad_up, h)."""
    s = sigmoid(gate)
    return grad_h * up * s * (1.0 + gate * (1.0 - s)), grad_h * gate * s, gate * s * up


def wgrad(grad_y, x, offsets=None, rows=None, transposed=False):
    """Weight gradient, or the stack of the experts' ones."""
    grad_y, x = np.asarray(grad_y, dtype=np.float64), np.asarray(x, dtype=np.float64)
    slots = grad_y.shape[0]

    def one(lo, hi):
        total = np.zeros((grad_y.shape[1], x.shape[1]))
        for i in range(lo, hi):
            r = i if rows is None else int(rows[i])
            if 0 <= r < x.shape[0]:
                total += np.outer(grad_y[i], x[r])
        return total.T if transposed else total

    if offsets is None:
        return one(0, slots)
    out = []
    for e in range(len(offsets) - 1):
        lo = min(max(int(offsets[e]), 0), slots)
        out.append(one(lo, min(max(int(offsets[e + 1]), lo), slots)))
    return np.stack(out)


def _scores(row, score):
    if score == "sigmoid":
        return sigmoid(row)
    if np.isnan(row).any():
        return np.full_like(row, math.nan)
    top = row.max()
    if top == -math.inf:
        return np.zeros_like(row)
    with np.errstate(invalid="ignore"):
        z = np.exp(row - top)
    return z / z.sum()


def _best(choice, n):
    """Indices of the n best choices that can be taken, best first, the lowest index among equals."""
    order = sorted(range(len(choice)), key=lambda i: (-choice[i], i))
    return [i for i in order if choice[i] > -math.inf][:n]


def route(logits, top_k, bias=None, score="softmax", groups=1, top_groups=1, group_top=2, renormalize=True, scale=1.0,
          token_mask=None):
    """dict of experts, weights, counts, offsets, order, rows."""
    logits = np.asarray(logits, dtype=np.float64)
    tokens, experts = logits.shape
    ids = np.full((tokens, top_k), -1, dtype=np.int64)
    weights = np.zeros((tokens, top_k))
    for t in range(tokens):
        if token_mask is not None and not token_mask[t]:
            continue
        row = logits[t]
        s = _scores(row, score)
        if np.isnan(s).any():
            weights[t] = math.nan
            continue
        choice = s if bias is None else s + np.asarray(bias, dtype=np.float64)
        choice = np.where(np.isneginf(row) | np.isnan(choice), -math.inf, choice)
        by = row.copy() if bias is None else choice.copy()
        if top_groups < groups:
            size = experts // groups
            score_of = []
            for g in range(groups):
                best = sorted(choice[g * size:(g + 1) * size], reverse=True)[:group_top]
                total = sum(best)
                score_of.append(-math.inf if math.isnan(total) else total)
            kept = sorted(range(groups), key=lambda g: (-score_of[g], g))[:top_groups]
            for g in range(groups):
                if g not in kept:
                    by[g * size:(g + 1) * size] = -math.inf
        taken = _best(by, top_k)
        w = np.array([s[i] for i in taken])
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else 0 * w
        ids[t, :len(taken)] = taken
        weights[t, :len(taken)] = scale * w
    flat = ids.reshape(-1)
    counts = np.array([(flat == e).sum() for e in range(experts)], dtype=np.int64)
    order = np.concatenate([np.flatnonzero(flat == e) for e in range(experts)] + [np.full((flat < 0).sum(), -1)]).astype(np.int64)
    return {"experts": ids, "weights": weights, "counts": counts, "offsets": np.concatenate([[0], np.cumsum(counts)]),
            "order": order, "rows": np.where(order < 0, -1, order // top_k)}


def route_weights(row, ids, score, renormalize, scale):
    """The weights of one token's taken experts as a function of its logits (for differences)."""
    s = _scores(np.asarray(row, dtype=np.float64), score)
    w = np.array([s[i] if i >= 0 else 0.0 for i in ids])
    if renormalize:
        w = w / w.sum() if w.sum() > 0 else 0 * w
    return scale * w


def route_backward(grad_weights, logits, ids, score="softmax", renormalize=True, scale=1.0):
    logits = np.asarray(logits, dtype=np.float64)
    grad = np.zeros_like(logits)
    experts = logits.shape[1]
    for t in range(logits.shape[0]):
        live = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < experts]
        if not live:
            continue
        s = _scores(logits[t], score)
        p = np.array([s[ids[t, j]] for j in live])
        dw = np.array([float(grad_weights[t, j]) for j in live])
        if renormalize:
            z = p.sum()
            ds = (dw - (dw * p).sum() / z) / z if z > 0 else 0 * dw
        else:
            ds = dw
        full = np.zeros(experts)
        for j, d in zip(live, scale * ds):
            full[ids[t, j]] += d
        grad[t] = s * (1 - s) * full if score == "sigmoid" else s * (full - (full * s).sum())
    return grad


def balance(bias, counts, rate):
    counts = np.asarray(counts).astype(object)      # exact whole numbers
    total = counts.sum(axis=-1, keepdims=True)
    sign = np.sign((total - counts.shape[-1] * counts).astype(object)).astype(np.float64)
    return np.asarray(bias, dtype=np.float64) + rate * sign
