"""Cases for measuring the row operators around the experts: routing with expert groups, row
quantisation to 8-bit integers, the 8-bit product over experts, and the weighted blend.

Every case names its operator in ``op``. ``run`` computes it in plain torch operations, or, when
``own`` is true, by the calls a program makes of this package. Sizes are those of the package's
layer configurations (hidden 2048 and 5120, 16 to 256 experts) and ragged ones between them.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_BIG = float(np.finfo(np.float32).max)
_TINY = 2.0 ** -126


# ---- cases ---------------------------------------------------------------------------------------

def _route(name, rows, experts, top_k, **kw):
    c = dict(name=name, op="route", rows=rows, experts=experts, top_k=top_k, routing="softmax",
             norm=True, bias=False, raw=False, groups=1, topk_groups=1, group_score="max",
             rsf=1.0, dtype="f32", pad=0, masked=0.0)
    c.update(kw)
    return c


def _quantise(name, rows, k, **kw):
    c = dict(name=name, op="quantise", rows=rows, k=k, dtype="bf16", pad=0)
    c.update(kw)
    return c


def _product(name, rows, n, k, **kw):
    c = dict(name=name, op="product", rows=rows, n=n, k=k, experts=1, top_k=1, gather=False,
             act="none", weighted=False, masked=0.0, dtype="bf16", pad=0)
    c.update(kw)
    return c


def _combine(name, rows, n, top_k, **kw):
    c = dict(name=name, op="combine", rows=rows, n=n, top_k=top_k, y_dtype="bf16", dtype="bf16",
             weighted=True, shared="none", masked=0.0)
    c.update(kw)
    return c


def listed():
    return [
        # one token of a 128-expert softmax layer: latency only
        _route("route one token", 1, 128, 8),
        # a prompt through a sigmoid router with a balance bias and the best 4 of 8 groups
        _route("route prompt in groups", 8191, 256, 8, routing="sigmoid", bias=True, groups=8,
               topk_groups=4, group_score="top2", rsf=2.5),
        # a padded batch, bf16 logits in a wider row, softmax weights kept as they are
        _route("route padded batch", 20000, 160, 6, norm=False, groups=8, topk_groups=3, rsf=16.0,
               dtype="bf16", pad=24, masked=0.1),
        # the rows of a decode batch
        _quantise("quantise decode rows", 64, 2048),
        # a prompt's hidden states
        _quantise("quantise prompt", 8192, 5120),
        # one token through a shared expert's down projection: one pass over the weights
        _product("product one token", 1, 5120, 8192),
        # sixteen tokens over 128 experts, gate and up: most experts hold a row or two
        _product("product decode experts", 16, 768, 2048, experts=128, top_k=8, gather=True,
                 act="swiglu"),
        # a prompt through a shared expert's gate and up, an odd number of rows
        _product("product prompt shared", 4099, 8192, 5120, act="swiglu"),
        # a prompt's gate and up over 128 experts, rows gathered by the grouping
        _product("product prompt experts", 8192, 768, 2048, experts=128, top_k=8, gather=True,
                 act="swiglu"),
        # the down projection of the same prompt, rows already in expert order
        _product("product prompt down", 8192, 2048, 768, experts=128, top_k=8),
        # the blend of a decode batch with a gated shared expert
        _combine("combine decode rows", 64, 2048, 8, shared="gated"),
        # the blend of a prompt
        _combine("combine prompt", 8192, 2048, 8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "quantise", "product", "product", "combine"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 3, 4, 8])
        experts = groups * _log(rng, 4, 512 // groups)
        keep = rng.randint(1, groups)
        routing = rng.choice(["softmax", "sigmoid", "sqrtsoftplus"])
        bias = routing != "softmax" and rng.random() < 0.6
        c = _route("", _log(rng, 1, 32768), experts, rng.randint(1, min(16, keep * experts // groups)),
                   routing=routing, norm=rng.random() < 0.6, bias=bias,
                   raw=routing != "softmax" and not bias and rng.random() < 0.4, groups=groups,
                   topk_groups=keep, group_score=rng.choice(["max", "top2"]),
                   rsf=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]),
                   pad=rng.choice([0, 0, 1, 8]), masked=rng.choice([0.0, 0.0, 0.25]))
    elif op == "quantise":
        k = 16 * _log(rng, 4, 512)
        c = _quantise("", _log(rng, 1, max(1, 41_000_000 // k)), k, dtype=rng.choice(["f32", "bf16"]),
                      pad=rng.choice([0, 0, 8]))
    elif op == "product":
        k = 16 * _log(rng, 8, 512)
        n = _log(rng, 64, 8192)
        experts = rng.choice([1, 1, 8, 32, 128])
        if experts > 1:
            n, k = min(n, 2048), min(k, 2048)
        top_k = rng.randint(1, min(8, experts))
        act = rng.choice(["none", "none", "swiglu", "geglu"])
        # the plain form pads every expert to the fullest one: its work stays below the largest
        # listed case's
        most = int(3.0e11 / (2.0 * n * k * top_k * (1 if act == "none" else 2)))
        gather = experts > 1 and rng.random() < 0.5
        c = _product("", _log(rng, 1, max(1, min(8192, most))), n, k, experts=experts, top_k=top_k,
                     gather=gather, act=act, weighted=gather and rng.random() < 0.4,
                     masked=0.2 if experts > 1 and rng.random() < 0.3 else 0.0,
                     dtype=rng.choice(["bf16", "bf16", "f32"]), pad=rng.choice([0, 0, 16]))
    else:
        top_k = rng.randint(1, 8)
        n = _log(rng, 64, 8192)
        c = _combine("", _log(rng, 1, max(1, 128_000_000 // (n * top_k))), n, top_k,
                     y_dtype=rng.choice(["bf16", "bf16", "f32"]), dtype=rng.choice(["bf16", "f32"]),
                     weighted=rng.random() < 0.8, shared=rng.choice(["none", "plain", "gated"]),
                     masked=rng.choice([0.0, 0.2]))
    del c["name"]
    return c


def work(case):
    c = case
    T = c["rows"]
    if c["op"] == "route":
        P = T * c["top_k"]
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": T * c["experts"] * size + P * 16 + (c["experts"] + 1) * 4,
                "flops": 8.0 * T * c["experts"]}
    if c["op"] == "quantise":
        # the values that the codes stand for are what comes back, so they are written too
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": T * c["k"] * (size + 1 + 4) + 4 * T, "flops": 3.0 * T * c["k"]}
    if c["op"] == "product":
        mats = 1 if c["act"] == "none" else 2
        live = T * c["top_k"] * (1.0 - c["masked"])
        E = c["experts"]
        active = E if E == 1 else E * (1.0 - (1.0 - 1.0 / E) ** live)
        out = 2 if c["dtype"] == "bf16" else 4
        x_rows = T if c["gather"] else live
        return {"bytes": active * mats * c["n"] * (c["k"] + 4) + x_rows * (c["k"] + 4)
                + live * c["n"] * out,
                "flops": 2.0 * live * mats * c["n"] * c["k"]}
    y = 2 if c["y_dtype"] == "bf16" else 4
    out = 2 if c["dtype"] == "bf16" else 4
    live = T * c["top_k"] * (1.0 - c["masked"])
    extra = 0 if c["shared"] == "none" else y
    return {"bytes": live * c["n"] * y + T * c["n"] * (out + extra) + T * c["top_k"] * 8,
            "flops": 2.0 * live * c["n"]}


# ---- inputs --------------------------------------------------------------------------------------

def _grouping(idx, experts):
    """Pairs p = row * top_k + slot in order of (expert, p); slots of -1 belong to no expert."""
    flat = idx.reshape(-1).long()
    e = torch.where(flat < 0, torch.full_like(flat, experts), flat)
    order = torch.argsort(e, stable=True)
    at = torch.arange(flat.numel(), device=flat.device)
    counts = torch.zeros(experts + 1, dtype=torch.long, device=flat.device)
    counts.scatter_add_(0, e, torch.ones_like(e))
    ends = torch.cumsum(counts, 0)[:experts]
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    place = torch.empty_like(order).scatter_(0, order, at)
    return (torch.where(at < offsets[-1], order, torch.full_like(order, -1)).int(), offsets.int(),
            torch.where(flat < 0, torch.full_like(place, -1), place).int())


def _choices(c, g):
    """Experts of each row as a trained router leaves them: some are much fuller than others."""
    T, E, k = c["rows"], c["experts"], c["top_k"]
    score = torch.randn(T, E, device="cuda", generator=g) + 0.4 * torch.randn(E, device="cuda",
                                                                             generator=g)
    idx = torch.topk(score, k, dim=1).indices.int()
    off = int(round(T * c["masked"]))
    if off:
        idx[T - off:] = -1
    return idx


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    T = c["rows"]
    s = {"case": c}

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def codes(*shape):
        return (normal(*shape) * 32.0).round_().clamp_(-127, 127).to(torch.int8)

    if c["op"] == "route":
        E = c["experts"]
        wide = torch.zeros(T, E + c["pad"], device="cuda", dtype=_DT[c["dtype"]])
        l = 1.5 * normal(T, E) + 0.5 * normal(E)
        if c["masked"]:
            l[T - int(T * c["masked"]):] = -math.inf      # rows behind the batch's last token
            l[:, E // 2] = -math.inf                      # an expert that is switched off
        wide[:, :E] = l.to(wide.dtype)
        s["wide"] = wide
        s["bias"] = 0.1 * normal(E) if c["bias"] else None
        P = T * c["top_k"]
        i32 = dict(device="cuda", dtype=torch.int32)
        s["out"] = {"idx": torch.empty(T, c["top_k"], **i32),
                    "weights": torch.empty(T, c["top_k"], device="cuda"),
                    "sorted_pairs": torch.empty(P, **i32),
                    "expert_offsets": torch.empty(E + 1, **i32),
                    "token_to_perm": torch.empty(P, **i32)}
    elif c["op"] == "quantise":
        wide = torch.zeros(T, c["k"] + c["pad"], device="cuda", dtype=_DT[c["dtype"]])
        x = normal(T, c["k"]) * torch.exp(0.5 * normal(T, 1))
        x[:, :: 97] *= 12.0                               # the few large channels of hidden states
        wide[:, : c["k"]] = x.to(wide.dtype)
        s["wide"] = wide
        s["codes"] = torch.empty(T, c["k"], device="cuda", dtype=torch.int8)
        s["scales"] = torch.empty(T, device="cuda")
    elif c["op"] == "product":
        E, k, n = c["experts"], c["top_k"], c["n"]
        P = T * k
        if E > 1:
            pairs, offsets, _ = _grouping(_choices(c, g), E)
            s["pairs"], s["offsets"] = pairs, offsets
            s["fullest"] = int((offsets[1:] - offsets[:-1]).max())
        x_rows = T if c["gather"] else P
        s["wide"] = torch.zeros(x_rows, c["k"] + c["pad"], device="cuda", dtype=torch.int8)
        s["wide"][:, : c["k"]] = codes(x_rows, c["k"])
        s["x_scales"] = 0.02 * torch.exp(0.3 * normal(x_rows))
        s["pair_weights"] = torch.rand(P, device="cuda", generator=g) if c["weighted"] else None
        s["w"] = [codes(E, n, c["k"]) for _ in range(1 if c["act"] == "none" else 2)]
        s["w_scales"] = [torch.exp(0.3 * normal(E, n)) / (32.0 * math.sqrt(c["k"])) for _ in s["w"]]
        s["out"] = torch.zeros(P, n, device="cuda", dtype=_DT[c["dtype"]])
    else:
        k, n = c["top_k"], c["n"]
        E = 64
        idx = torch.randint(0, E, (T, k), device="cuda", generator=g, dtype=torch.int32)
        off = int(round(T * c["masked"]))
        if off:
            idx[T - off:] = -1
        s["perm"] = _grouping(idx, E)[2]
        s["y"] = normal(T * k, n).to(_DT[c["y_dtype"]])
        s["weights"] = torch.rand(T, k, device="cuda", generator=g) if c["weighted"] else None
        s["shared"] = None if c["shared"] == "none" else normal(T, n).to(_DT[c["y_dtype"]])
        s["gate"] = torch.rand(T, device="cuda", generator=g) if c["shared"] == "gated" else None
        s["out"] = torch.empty(T, n, device="cuda", dtype=_DT[c["dtype"]])
    return s


# ---- plain forms ---------------------------------------------------------------------------------

def _plain_route(s):
    """Keys are compared in 64 bits: two scores may be closer than 32 bits tell apart."""
    c = s["case"]
    E, k, G = c["experts"], c["top_k"], c["groups"]
    l = s["wide"][:, :E].double().clamp(max=_BIG)
    gone = ~(l > -math.inf)
    l = torch.where(gone, torch.full_like(l, -math.inf), l)
    T = l.shape[0]
    if c["routing"] == "softmax":
        top = l.max(dim=1, keepdim=True).values.clamp(min=-_BIG)
        e = torch.exp(l - top)
        score = e / e.sum(dim=1, keepdim=True).clamp(min=_TINY)
    elif c["routing"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        score = torch.sqrt(l.clamp(min=0.0) + torch.log1p(torch.exp(-l.abs())))
    key = score + s["bias"].double() if c["bias"] else l
    key = torch.where(gone, torch.full_like(key, -math.inf), key)
    if G > 1:
        if c["group_score"] == "max":
            of = key.view(T, G, E // G).max(dim=2).values
        else:
            v = key if (c["bias"] or c["raw"]) else torch.where(gone, key, score)
            two = torch.topk(v.view(T, G, E // G), 2, dim=2).values
            of = two[..., 0] + torch.where(two[..., 1] > -math.inf, two[..., 1],
                                           torch.zeros_like(two[..., 1]))
        best = torch.argsort(of, dim=1, descending=True, stable=True)[:, : c["topk_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, best, True)
        key = key.view(T, G, E // G).masked_fill(~keep[..., None], -math.inf).view(T, E)
    got, idx = torch.sort(key, dim=1, descending=True, stable=True)
    got, idx = got[:, :k], idx[:, :k]
    live = got > -math.inf
    w = torch.where(live, torch.gather(score, 1, idx), torch.zeros_like(got))
    if c["norm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    idx = torch.where(live, idx, torch.full_like(idx, -1)).int()
    pairs, offsets, place = _grouping(idx, E)
    return {"idx": idx, "weights": (w * c["rsf"]).float(), "sorted_pairs": pairs,
            "expert_offsets": offsets, "token_to_perm": place}


def _plain_quantise(s):
    x = s["wide"][:, : s["case"]["k"]].float()
    amax = x.abs().amax(dim=1)
    # divided by a tensor: a division by a number may be a product with its rounded reciprocal
    scale = (amax / torch.full_like(amax, 127.0)).clamp(min=_TINY)
    scale = torch.where(amax > 0, scale, torch.ones_like(amax))
    # the quotient in 64 bits: next to a half it decides the code
    q = torch.round(x.double() / scale.double()[:, None]).clamp(-127, 127).float()
    return {"values": q * scale[:, None], "scales": scale}


def _act(name, gate, up):
    if name == "swiglu":
        return gate / (1.0 + torch.exp(-gate)) * up
    t = torch.tanh(math.sqrt(2.0 / math.pi) * (gate + 0.044715 * gate ** 3))
    return 0.5 * gate * (1.0 + t) * up


def _plain_product(s):
    c = s["case"]
    x, xs = s["wide"][:, : c["k"]], s["x_scales"]
    if c["experts"] == 1:
        ys = [(x.float() @ w[0].float().t()) * ws[0] * xs[:, None]
              for w, ws in zip(s["w"], s["w_scales"])]
        y = ys[0] if c["act"] == "none" else _act(c["act"], *ys)
        return y.to(s["out"].dtype)
    # every expert's rows, padded to the fullest expert: one batched product
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(s["fullest"], device=off.device)
    live = at < off[1:, None]
    at = torch.where(live, at, torch.full_like(at, -1))
    pair = s["pairs"].long()[at.clamp(min=0)]
    row = pair // c["top_k"] if c["gather"] else at.clamp(min=0)
    row = torch.where(live, row, torch.zeros_like(row))
    scale = xs[row]
    if s["pair_weights"] is not None:
        scale = scale * s["pair_weights"][pair.clamp(min=0)]
    xg = x[row].float()
    ys = [torch.bmm(xg, w.float().transpose(1, 2)) * ws[:, None, :] * scale[..., None]
          for w, ws in zip(s["w"], s["w_scales"])]
    y = ys[0] if c["act"] == "none" else _act(c["act"], *ys)
    P, n = s["out"].shape
    # row P takes what the padding computed; rows that no expert owns stay zero
    out = torch.zeros(P + 1, n, device=y.device, dtype=s["out"].dtype)
    out[torch.where(live, at, torch.full_like(at, P)).view(-1)] = y.view(-1, n).to(out.dtype)
    return out[:P]


def _plain_combine(s):
    c = s["case"]
    T, k = c["rows"], c["top_k"]
    perm = s["perm"].long().view(T, k)
    y = s["y"][perm.clamp(min=0)].float()
    w = torch.ones(T, k, device=y.device) if s["weights"] is None else s["weights"]
    w = torch.where(perm < 0, torch.zeros_like(w), w)
    out = (y * w[..., None]).sum(dim=1)
    if s["shared"] is not None:
        out = out + s["shared"].float() * (1.0 if s["gate"] is None else s["gate"][:, None])
    return out.to(_DT[c["dtype"]])


# ---- the package's calls -------------------------------------------------------------------------

def _matrix(B, w, scales):
    m = B.moe_matrix()
    m.format = B.MOE_FMT_INT8
    m.packed = w.data_ptr()
    m.scales = scales.data_ptr()
    m.expert_stride = w.stride(0)
    m.scale_stride = scales.stride(0) * 4
    return m


def _workspace(s, B, nbytes):
    """The workspace that the program keeps beside its inputs, made on the first pass."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(nbytes, 256), dtype=torch.uint8, device="cuda")
        B.moe_workspace_init(s["ws"], s["ws"].numel(), torch.cuda.current_stream())
    return s["ws"]


def _own_run(s):
    from mixture_experts_decode_gemv_b200 import binding as B

    c = s["case"]
    T = c["rows"]
    st = torch.cuda.current_stream()
    if c["op"] == "route":
        if "cfg" not in s:
            s["cfg"] = B.moe_route_cfg(
                num_experts=c["experts"], top_k=c["top_k"], routing=B.ROUTING_CODES[c["routing"]],
                norm_topk_prob=int(c["norm"]), select_on_raw_logits=int(c["raw"]),
                has_expert_bias=int(c["bias"]), routed_scaling_factor=c["rsf"],
                num_groups=c["groups"], topk_groups=c["topk_groups"],
                group_score=B.GROUP_SCORE_CODES[c["group_score"]],
                logits_dtype=B.FORMAT_CODES[c["dtype"]])
            s["ws_bytes"] = B.moe_route_workspace_bytes(s["cfg"], T)
        ws = _workspace(s, B, s["ws_bytes"])
        o = s["out"]
        B.moe_route_rows(s["cfg"], T, s["wide"], s["wide"].stride(0), s["bias"], o["idx"],
                         o["weights"], o["sorted_pairs"], o["expert_offsets"], o["token_to_perm"],
                         ws, ws.numel(), st)
        return o
    if c["op"] == "quantise":
        B.moe_quantize_rows_int8(T, c["k"], B.FORMAT_CODES[c["dtype"]], s["wide"],
                                 s["wide"].stride(0), s["codes"], s["codes"].stride(0),
                                 s["scales"], st)
        return {"values": s["codes"] * s["scales"][:, None], "scales": s["scales"]}
    if c["op"] == "product":
        if "cfg" not in s:
            s["cfg"] = B.moe_matmul_cfg(
                n=c["n"], k=c["k"], num_experts=c["experts"], top_k=c["top_k"],
                activation=B.ACTIVATION_CODES["geglu" if c["act"] == "geglu" else "swiglu"],
                out_dtype=B.FORMAT_CODES[c["dtype"]])
            s["mats"] = [_matrix(B, w, ws) for w, ws in zip(s["w"], s["w_scales"])]
            s["ws_bytes"] = B.moe_matmul_workspace_bytes(s["cfg"], s["out"].shape[0])
        ws = _workspace(s, B, s["ws_bytes"])
        B.moe_matmul_int8(s["cfg"], s["wide"].shape[0], s["wide"], s["wide"].stride(0),
                          s["x_scales"], s["out"].shape[0], s.get("offsets"),
                          s["pairs"] if c["gather"] else None, s["pair_weights"], s["mats"][0],
                          s["mats"][1] if len(s["mats"]) > 1 else None, s["out"],
                          s["out"].stride(0), ws, ws.numel(), st)
        return s["out"]
    B.moe_combine_rows(T, c["n"], c["top_k"], B.FORMAT_CODES[c["y_dtype"]], s["y"], s["y"].stride(0),
                       s["y"].shape[0], s["perm"], s["weights"], s["shared"],
                       c["n"] if s["shared"] is not None else 0, s["gate"],
                       B.FORMAT_CODES[c["dtype"]], s["out"], s["out"].stride(0), st)
    return s["out"]


_PLAIN = {"route": _plain_route, "quantise": _plain_quantise, "product": _plain_product,
          "combine": _plain_combine}


def run(state):
    return _own_run(state) if own else _PLAIN[state["case"]["op"]](state)


# ---- the definitions in 64 bits ------------------------------------------------------------------

def _exact_route(s):
    c = s["case"]
    E, k, G, T = c["experts"], c["top_k"], c["groups"], c["rows"]
    l = s["wide"][:, :E].float().cpu().numpy().astype(np.float64)
    off = np.isneginf(l) | np.isnan(l)
    with np.errstate(all="ignore"):
        if c["routing"] == "softmax":
            e = np.where(off, 0.0, np.exp(l - np.max(np.where(off, -1e30, l), axis=1)[:, None]))
            score = e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300)
        elif c["routing"] == "sigmoid":
            score = np.exp(-np.logaddexp(0.0, -l))
        else:
            score = np.sqrt(np.logaddexp(0.0, l))
    rank = l if s["bias"] is None else score + s["bias"].cpu().numpy().astype(np.float64)
    rank = np.where(off, -np.inf, rank)
    if G > 1:
        by = rank if (c["group_score"] == "max" or c["bias"] or c["raw"]) else np.where(
            off, -np.inf, score)
        top = -np.sort(-by.reshape(T, G, E // G), axis=2)
        of = top[:, :, 0]
        if c["group_score"] == "top2":
            of = of + np.where(np.isneginf(top[:, :, 1]), 0.0, top[:, :, 1])
        place = np.argsort(np.argsort(-of, axis=1, kind="stable"), axis=1, kind="stable")
        rank = np.where(np.repeat(place < c["topk_groups"], E // G, axis=1), rank, -np.inf)
    idx = np.argsort(-rank, axis=1, kind="stable")[:, :k]
    dead = np.isneginf(np.take_along_axis(rank, idx, axis=1))
    w = np.where(dead, 0.0, np.take_along_axis(score, idx, axis=1))
    if c["norm"]:
        total = w.sum(axis=1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    idx = np.where(dead, -1, idx).astype(np.int32)
    flat = idx.reshape(-1)
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable")
    offsets = np.searchsorted(np.sort(np.where(flat < 0, E, flat)), np.arange(E + 1))
    place = np.empty(flat.size, np.int64)
    place[order] = np.arange(flat.size)
    return {"idx": idx, "weights": w * c["rsf"],
            "sorted_pairs": np.where(np.arange(flat.size) < offsets[E], order, -1).astype(np.int32),
            "expert_offsets": offsets.astype(np.int32),
            "token_to_perm": np.where(flat < 0, -1, place).astype(np.int32)}


def _exact_quantise(s):
    x = s["wide"][:, : s["case"]["k"]].float().cpu().numpy().astype(np.float64)
    amax = np.max(np.abs(x), axis=1)
    # the scale is stored in 32 bits, and the codes are those of the stored scale
    scale = np.where(amax > 0, np.maximum((amax / 127.0).astype(np.float32), np.float32(_TINY)),
                     np.float32(1)).astype(np.float64)
    return {"values": np.clip(np.rint(x / scale[:, None]), -127, 127) * scale[:, None],
            "scales": scale}


def _exact_product(s):
    c = s["case"]
    x = s["wide"][:, : c["k"]].double()
    P, n = s["out"].shape
    out = torch.zeros(P, n, device="cuda", dtype=torch.float64)
    off = s["offsets"].tolist() if c["experts"] > 1 else [0, P]
    for e in range(c["experts"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        pair = s["pairs"][a:b].long() if c["experts"] > 1 else torch.arange(a, b, device="cuda")
        row = pair // c["top_k"] if c["gather"] else torch.arange(a, b, device="cuda")
        left = s["x_scales"][row].double()
        if s["pair_weights"] is not None:
            left = left * s["pair_weights"][pair].double()
        ys = [torch.mm(x[row], w[e].double().t()) * torch.outer(left, ws[e].double())
              for w, ws in zip(s["w"], s["w_scales"])]
        if c["act"] == "none":
            out[a:b] = ys[0]
        elif c["act"] == "swiglu":
            out[a:b] = ys[0] * torch.sigmoid(ys[0]) * ys[1]
        else:
            out[a:b] = torch.nn.functional.gelu(ys[0], approximate="tanh") * ys[1]
    return out


def _exact_combine(s):
    c = s["case"]
    T, k, n = c["rows"], c["top_k"], c["n"]
    out = torch.zeros(T, n, device="cuda", dtype=torch.float64)
    perm = s["perm"].long().view(T, k)
    for j in range(k):
        live = perm[:, j] >= 0
        w = 1.0 if s["weights"] is None else s["weights"][live, j].double()[:, None]
        out[live] += s["y"][perm[live, j]].double() * w
    if s["shared"] is not None:
        gate = 1.0 if s["gate"] is None else s["gate"].double()[:, None]
        out += s["shared"].double() * gate
    return out


_EXACT = {"route": _exact_route, "quantise": _exact_quantise, "product": _exact_product,
          "combine": _exact_combine}


def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))
