"""Float64 CPU oracle of the row operators (routing with expert groups, row quantisation to int8,
the int8 product over experts, the weighted blend).

TEST INFRASTRUCTURE ONLY, like ``moe_ref``: it shares no code, table or constant with the CUDA
library and is written row by row from the definitions in the C header.
"""
from __future__ import annotations

import math
from typing import Dict, Optional

import numpy as np

from . import moe_ref

F32_MAX = float(np.finfo(np.float32).max)


def score(l: float, routing: str) -> float:
    """sigmoid(l) or sqrt(softplus(l)), without overflow for any finite l."""
    if routing == "sigmoid":
        return 1.0 / (1.0 + math.exp(-l)) if l >= 0 else math.exp(l) / (1.0 + math.exp(l))
    return math.sqrt(max(l, 0.0) + math.log1p(math.exp(-abs(l))))


def log_score(l: float, routing: str) -> float:
    """log of ``score``, for logits whose score underflows."""
    if routing == "sigmoid":
        return -(max(-l, 0.0) + math.log1p(math.exp(-abs(l))))
    return 0.5 * (math.log(max(l, 0.0) + math.log1p(math.exp(-abs(l)))) if l > -30.0 else l)


def route_row(logits, *, top_k: int, norm: bool, routing: str = "softmax", raw: bool = False, bias=None,
              rsf: float = 1.0, groups: int = 1, topk_groups: int = 1, group_score: str = "max"):
    """(ids, weights) of one row: top_k entries, -1 and 0 where no expert is left."""
    E = len(logits)
    l = [min(float(v), F32_MAX) for v in logits]
    b = [0.0] * E if bias is None else [float(v) for v in bias]
    live = [v > -math.inf and w > -math.inf for v, w in zip(l, b)]      # NaN compares false
    if not any(live):
        return [-1] * top_k, [0.0] * top_k
    if routing == "softmax":
        top = max(v for v, ok in zip(l, live) if ok)
        e = [math.exp(v - top) if ok else 0.0 for v, ok in zip(l, live)]
        s = [v / sum(e) for v in e]
        logs = [v - top if ok else -math.inf for v, ok in zip(l, live)]
    else:
        s = [score(v, routing) if ok else 0.0 for v, ok in zip(l, live)]
        logs = [log_score(v, routing) if ok else -math.inf for v, ok in zip(l, live)]
    key = [x + y for x, y in zip(s, b)] if bias is not None else l
    value = key if (bias is not None or raw) else s
    size = E // groups
    allowed = set(range(E))
    if topk_groups < groups:
        ranked = []
        for g in range(groups):
            of = [e for e in range(g * size, (g + 1) * size) if live[e]]
            if not of:
                continue
            if group_score == "max":
                worth = max(key[e] for e in of)
            else:
                worth = sum(sorted((value[e] for e in of), reverse=True)[:2])
            ranked.append((-worth, g))
        allowed = {e for _, g in sorted(ranked)[:topk_groups]
                   for e in range(g * size, (g + 1) * size)}
    ids = sorted((e for e in range(E) if live[e] and e in allowed), key=lambda e: (-key[e], e))
    ids = ids[:top_k]
    if norm:
        most = max(logs[e] for e in ids) if ids else 0.0
        w = [math.exp(logs[e] - most) for e in ids]
        w = [v / sum(w) for v in w]
    else:
        w = [s[e] for e in ids]
    pad = top_k - len(ids)
    return ids + [-1] * pad, [v * rsf for v in w] + [0.0] * pad


def route(logits: np.ndarray, **kw):
    rows = [route_row(r, **kw) for r in np.asarray(logits, np.float64)]
    k = kw["top_k"]
    return (np.array([r[0] for r in rows], np.int32).reshape(len(rows), k),
            np.array([r[1] for r in rows], np.float64).reshape(len(rows), k))


def group(idx: np.ndarray, num_experts: int) -> Dict[str, np.ndarray]:
    """The grouping of moe_ref, for pairs that have an expert; -1 for what has none."""
    flat = np.asarray(idx).reshape(-1)
    live = [p for p in range(flat.size) if flat[p] >= 0]
    order = sorted(live, key=lambda p: (flat[p], p))
    pairs = np.full(flat.size, -1, np.int32)
    pairs[: len(order)] = order
    place = np.full(flat.size, -1, np.int32)
    place[order] = np.arange(len(order))
    offsets = np.array([sum(1 for p in live if flat[p] < e) for e in range(num_experts + 1)]
                       if flat.size < 4096 else
                       np.searchsorted(np.sort(flat[live]), np.arange(num_experts + 1)), np.int32)
    return {"sorted_pairs": pairs, "expert_offsets": offsets, "token_to_perm": place}


def quantize_rows(x: np.ndarray):
    """(codes, scales) of each row of float32 values."""
    x = np.asarray(x, np.float32)
    codes = np.zeros(x.shape, np.int8)
    scales = np.empty(x.shape[0], np.float32)
    for r, row in enumerate(x):
        if not np.all(np.isfinite(row)):
            scales[r] = np.nan
            continue
        amax = float(np.max(np.abs(row.astype(np.float64))))
        sc = max(np.float32(amax / 127.0), np.float32(2.0 ** -126)) if amax > 0 else np.float32(1)
        scales[r] = sc
        codes[r] = np.clip(np.rint(row.astype(np.float64) / float(sc)), -127, 127)
    return codes, scales


def matmul_int8(x, x_scales, w, w_scales, out, offsets=None, pairs=None, top_k=1,
                pair_weights=None, up=None, up_scales=None, activation="swiglu"):
    """Writes the product's rows into ``out`` (float64); rows without an expert keep theirs.
    Returns |gate * up| beside it, the size that an activation's rounding is relative to."""
    rows = out.shape[0]
    spans = [(0, rows)] if offsets is None else [
        (int(offsets[e]), int(offsets[e + 1])) for e in range(len(offsets) - 1)]
    size = np.zeros_like(out)
    for e, (a, b) in enumerate(spans):
        at = np.arange(a, b)
        if pairs is not None:
            p = np.asarray(pairs)[a:b]
            ok = (p >= 0) & (p // top_k < x.shape[0])
            at, p = at[ok], p[ok]
            src = p // top_k
        else:
            src = at
        if at.size == 0:
            continue
        left = x_scales[src].astype(np.float64)
        if pair_weights is not None:
            left = left * pair_weights[p].astype(np.float64)
        # float64 holds every sum exactly: they stay below 2^31
        def prod(m, s):
            return (x[src].astype(np.float64) @ m[e].astype(np.float64).T) * left[:, None] \
                * s[e].astype(np.float64)[None]
        y = prod(w, w_scales)
        if up is not None:
            u = prod(up, up_scales)
            size[at] = np.abs(y * u)
            y = (moe_ref.silu(y) if activation == "swiglu" else moe_ref.gelu_tanh(y)) * u
        out[at] = y
    return out, size


def combine(y, perm, top_k: int, rows: int, weights=None, shared=None, gate=None):
    """(blend, sum of the terms' magnitudes), both float64 [rows, n]."""
    y = np.asarray(y, np.float64)
    out = np.zeros((rows, y.shape[1]))
    mag = np.zeros_like(out)
    for r in range(rows):
        for s in range(top_k):
            at = int(perm[r * top_k + s])
            if not 0 <= at < y.shape[0]:
                continue
            w = 1.0 if weights is None else float(weights[r, s])
            out[r] += w * y[at]
            mag[r] += abs(w) * np.abs(y[at])
        if shared is not None:
            g = 1.0 if gate is None else float(gate[r])
            out[r] += g * np.asarray(shared[r], np.float64)
            mag[r] += abs(g) * np.abs(np.asarray(shared[r], np.float64))
    return out, mag
