"""GPU tests of the row operators against their float64 oracle: whole numbers bit-exact, floating
outputs within bounds that count the roundings (each is derived where it is used)."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from mixture_experts_decode_gemv_b200 import binding as B
from oracle import moe_ref, rows_ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, BF16 = B.MOE_FMT_F32, B.MOE_FMT_BF16
DT = {F32: torch.float32, BF16: torch.bfloat16}
EPS = 2.0 ** -24                    # half a step of float32
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def dev(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a)).to("cuda", dtype)


def status(ws):
    return B.moe_get_device_status(ws, ws.numel(), torch.cuda.current_stream())


def workspace(nbytes):
    ws = torch.empty(max(256, nbytes), dtype=torch.uint8, device="cuda")
    B.moe_workspace_init(ws, ws.numel(), torch.cuda.current_stream())
    return ws


# ---- routing -------------------------------------------------------------------------------------

def route_on_gpu(logits, top_k, routing="softmax", norm=True, raw=False, bias=None, rsf=1.0, groups=1,
                 topk_groups=1, group_score="max", grouping=True, ws=None, stream=None):
    """logits: a CUDA tensor [T, E], any row stride. Outputs stand between canary values."""
    T, E = logits.shape
    cfg = B.moe_route_cfg(num_experts=E, top_k=top_k, routing=B.ROUTING_CODES[routing],
                          norm_topk_prob=int(norm), select_on_raw_logits=int(raw),
                          has_expert_bias=int(bias is not None), routed_scaling_factor=rsf,
                          num_groups=groups, topk_groups=topk_groups,
                          group_score=B.GROUP_SCORE_CODES[group_score],
                          logits_dtype=F32 if logits.dtype == torch.float32 else BF16)
    P = T * top_k
    full = {n: torch.full((c + 16,), 77, dtype=d, device="cuda")
            for n, c, d in (("idx", P, torch.int32), ("weights", P, torch.float32),
                            ("sorted_pairs", P, torch.int32), ("expert_offsets", E + 1, torch.int32),
                            ("token_to_perm", P, torch.int32))}
    out = {n: t[8:-8] for n, t in full.items()}
    # canaries keep the 4-byte alignment only: the outputs need no more
    nb = B.moe_route_workspace_bytes(cfg, T)
    if ws is None:
        ws = torch.full((nb + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    g = [out["sorted_pairs"], out["expert_offsets"], out["token_to_perm"]] if grouping else [None] * 3
    B.moe_route_rows(cfg, T, logits, logits.stride(0) if T else E, bias, out["idx"], out["weights"], *g,
                     ws, nb, stream if stream is not None else torch.cuda.current_stream())
    torch.cuda.synchronize()
    for n, t in full.items():
        assert torch.all(t[:8] == 77) and torch.all(t[-8:] == 77), f"{n}: written outside"
        if not grouping and n in ("sorted_pairs", "expert_offsets", "token_to_perm"):
            assert torch.all(t == 77)
    assert torch.all(ws[nb:] == 0xA5)
    got = {n: t.cpu().numpy() for n, t in out.items()}
    got["idx"] = got["idx"].reshape(T, top_k)
    got["weights"] = got["weights"].reshape(T, top_k)
    return got


def check_route(logits, got, grouping=True, **kw):
    l = logits.float().cpu().numpy()
    if kw.get("bias") is not None:
        kw = dict(kw, bias=kw["bias"].cpu().numpy())
    ids, w = rows_ref.route(l, **kw)
    np.testing.assert_array_equal(got["idx"], ids)
    # exp of a difference d carries |d| * EPS from its argument (|d| <= 32 here where the result
    # counts) and a few units of its own; sums, quotients and the scale add under 24 more; the
    # denominator has as much again: under 2 * 64 roundings in all. Below 2^-100 nothing counts.
    rsf = kw.get("rsf", 1.0)
    np.testing.assert_allclose(got["weights"], w, rtol=128 * EPS, atol=2.0 ** -100 * abs(rsf))
    if grouping:
        want = rows_ref.group(ids, l.shape[1])
        for n, v in want.items():
            np.testing.assert_array_equal(got[n], v, err_msg=n)


ROUTES = [
    dict(top_k=8, norm=True), dict(top_k=6, norm=False, rsf=16.0),
    dict(top_k=4, routing="sigmoid", norm=True, with_bias=True),
    dict(top_k=3, routing="sigmoid", norm=False, raw=True),
    dict(top_k=5, routing="sqrtsoftplus", norm=True, with_bias=True, rsf=2.5),
    dict(top_k=1, routing="sqrtsoftplus", norm=False),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("experts", [8, 31, 33, 64, 128, 160, 256, 512])
@pytest.mark.parametrize("opts", ROUTES)
def test_route_without_groups(opts, experts, dtype):
    kw = dict(opts)
    rng = np.random.default_rng(experts)
    l = dev(rng.standard_normal((37, experts)) * 1.5, dtype)
    if kw.pop("with_bias", False):
        kw["bias"] = dev(rng.standard_normal(experts) * 0.1, torch.float32)
    check_route(l, route_on_gpu(l, **kw), **kw)


@pytest.mark.parametrize("score", ["max", "top2"])
@pytest.mark.parametrize("experts,groups,keep", [(256, 8, 4), (160, 8, 3), (64, 2, 1), (96, 3, 2),
                                                 (510, 17, 5), (512, 32, 7), (506, 11, 6), (30, 6, 5),
                                                 (32, 32, 9)])
@pytest.mark.parametrize("opts", ROUTES)
def test_route_with_groups(opts, experts, groups, keep, score):
    kw = dict(opts, groups=groups, topk_groups=keep, group_score=score)
    kw["top_k"] = min(kw["top_k"], keep * experts // groups)
    rng = np.random.default_rng(experts + groups)
    l = dev(rng.standard_normal((33, experts)) * 1.5, torch.float32)
    if kw.pop("with_bias", False):
        kw["bias"] = dev(rng.standard_normal(experts) * 0.1, torch.float32)
    check_route(l, route_on_gpu(l, **kw), **kw)


@pytest.mark.parametrize("rows", [0, 1, 2, 15, 63, 64, 65, 147, 148, 149, 1000, 2369, 6001])
@pytest.mark.parametrize("experts,top_k,groups,keep", [(1, 1, 1, 1), (16, 2, 1, 1), (64, 16, 4, 3)])
def test_route_row_counts(rows, experts, top_k, groups, keep):
    rng = np.random.default_rng(rows)
    kw = dict(top_k=top_k, routing="sigmoid", norm=True, groups=groups, topk_groups=keep)
    l = dev(rng.standard_normal((rows, experts)), torch.float32)
    check_route(l, route_on_gpu(l, **kw), **kw)
    got = route_on_gpu(l, grouping=False, **kw)
    check_route(l, got, grouping=False, **kw)


@pytest.mark.parametrize("rows", [5, 300])
@pytest.mark.parametrize("opts", ROUTES)
def test_route_masked_experts_and_rows(opts, rows):
    kw = dict(opts, groups=4, topk_groups=2, group_score="top2")
    rng = np.random.default_rng(11)
    l = rng.standard_normal((rows, 32)).astype(np.float32)
    l[0] = -np.inf                                    # nothing left
    l[1, 3:] = np.nan                                 # three experts left, in one group
    l[2, 8:16] = -np.inf                              # a whole group
    l[3, ::2] = -np.inf
    l[4, [1, 9, 17]] = np.inf                         # as the largest finite logit
    if rows > 5:
        l[rows // 2:, 1:] = -np.inf                   # one expert left
        l[-3:] = -np.inf
    t = dev(l, torch.float32)
    if kw.pop("with_bias", False):
        b = (rng.standard_normal(32) * 0.1).astype(np.float32)
        b[5] = -np.inf
        b[6] = np.nan
        kw["bias"] = dev(b)
    check_route(t, route_on_gpu(t, **kw), **kw)


@pytest.mark.parametrize("routing", ["softmax", "sigmoid", "sqrtsoftplus"])
@pytest.mark.parametrize("norm", [True, False])
def test_route_extreme_logits(routing, norm):
    l = np.zeros((7, 40), np.float32)
    l[1] = -300.0 - np.arange(40)                     # every score underflows float32
    l[2] = 60.0 + np.arange(40) % 7                   # sigmoid saturates: the logits still rank
    l[3] = -np.finfo(np.float32).max
    l[4] = np.finfo(np.float32).max
    l[5] = np.where(np.arange(40) % 3 == 0, 1e-30, -1e-30)
    l[6] = -90.0 - 0.5 * np.arange(40)                # scores around the smallest normal number
    kw = dict(top_k=6, routing=routing, norm=norm)
    t = dev(l)
    check_route(t, route_on_gpu(t, **kw), **kw)


def test_route_ties_go_to_the_lowest_expert():
    rng = np.random.default_rng(5)
    l = rng.integers(-2, 3, (200, 256)).astype(np.float32)
    zero = torch.zeros(256, device="cuda")
    for kw in (dict(top_k=8, norm=True), dict(top_k=8, routing="sigmoid", norm=True, bias=zero),
               dict(top_k=8, routing="sigmoid", norm=True, bias=zero, groups=8, topk_groups=4,
                    group_score="top2"),
               dict(top_k=8, routing="softmax", norm=True, groups=8, topk_groups=4, group_score="top2")):
        t = dev(l)
        check_route(t, route_on_gpu(t, **kw), **kw)


@pytest.mark.parametrize("routing", ["sigmoid", "sqrtsoftplus"])
@pytest.mark.parametrize("groups,keep", [(1, 1), (8, 4)])
def test_route_keys_closer_than_float32_tells_apart(routing, groups, keep):
    """Biases that lift every key to the same number: what is left between two keys is the rounding
    of the stored bias, up to 2^-25, and 64-bit arithmetic ranks them by it."""
    rng = np.random.default_rng(6)
    base = (rng.standard_normal(128) * 1.5).astype(np.float32)
    s = np.array([rows_ref.score(float(v), routing) for v in base])
    bias = dev((0.5 - s).astype(np.float32))
    l = np.repeat(base[None], 100, axis=0)
    l[::2] += (rng.standard_normal((50, 128)) * 2.0 ** -22).astype(np.float32)
    t = dev(l)
    kw = dict(top_k=8, routing=routing, norm=True, bias=bias, groups=groups, topk_groups=keep,
              group_score="top2")
    check_route(t, route_on_gpu(t, **kw), **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_route_strided_rows_at_odd_addresses(dtype, pad):
    rng = np.random.default_rng(8)
    wide = torch.full((90, 64 + pad), float("nan"), dtype=dtype, device="cuda")
    view = wide.view(-1)[1: 1 + 89 * (64 + pad)].view(89, 64 + pad)[:, :64]
    view.copy_(dev(rng.standard_normal((89, 64)), dtype))
    kw = dict(top_k=8, norm=True)
    check_route(view, route_on_gpu(view, **kw), **kw)


def test_route_past_two_to_the_31_logits():
    """The last rows of a long batch route and group like the same rows alone."""
    rows, E = 4_300_000, 512
    g = torch.Generator(device="cuda").manual_seed(2)
    part = torch.randn(1000, E, device="cuda", generator=g)
    l = part.repeat(rows // 1000, 1)
    kw = dict(top_k=2, routing="softmax", norm=True)
    few, many = route_on_gpu(part, **kw), route_on_gpu(l, **kw)
    n = rows // 1000
    np.testing.assert_array_equal(many["expert_offsets"], few["expert_offsets"] * n)
    np.testing.assert_array_equal(many["idx"].reshape(n, -1), np.repeat(few["idx"].reshape(1, -1), n, axis=0))
    perm, pairs = many["token_to_perm"].astype(np.int64), many["sorted_pairs"]
    np.testing.assert_array_equal(pairs[perm], np.arange(2 * rows))
    flat = many["idx"].reshape(-1)[pairs]             # grouped, and in order within each expert
    assert np.all(np.diff(flat) >= 0) and np.all(np.diff(pairs)[np.diff(flat) == 0] > 0)


def test_route_without_grouping_needs_no_workspace():
    l = torch.randn(100, 40, device="cuda")
    idx, w = torch.empty(100, 3, dtype=torch.int32, device="cuda"), torch.empty(100, 3, device="cuda")
    cfg = B.moe_route_cfg(num_experts=40, top_k=3, routing=0, norm_topk_prob=1, select_on_raw_logits=0,
                          has_expert_bias=0, routed_scaling_factor=1.0, num_groups=1, topk_groups=1, group_score=0,
                          logits_dtype=F32)
    B.moe_route_rows(cfg, 100, l, 40, None, idx, w, stream=torch.cuda.current_stream())
    assert torch.equal(idx.long(), torch.topk(l, 3, dim=1).indices)


def test_route_agrees_with_the_decode_layer():
    """The same experts and grouping as moe_decode_forward chooses for its rows."""
    from mixture_experts_decode_gemv_b200.device_layer import DeviceLayer
    from mixture_experts_decode_gemv_b200.synthetic import LayerConfig, SyntheticLayer
    cfg = LayerConfig(name="rows", hidden=256, num_experts=32, top_k=4, moe_inter=128, fmt="bf16",
                      routing="sigmoid", has_expert_bias=True, norm_topk_prob=True,
                      routed_scaling_factor=1.5, index=901)
    lay = SyntheticLayer(cfg)
    lay.key_fn = moe_ref.selection_key_fn(lay)
    m = 48
    x = lay.x(m)
    layer = DeviceLayer(lay)
    ws, out = layer.new_workspace(m), layer.new_out(m)
    layer.forward(layer.x_to_device(x), out, ws)
    want = layer.read_routing(m, ws)
    wr = moe_ref.bf16_to_f64(lay.router_w()).reshape(32, 256)
    l = dev((moe_ref.decode_activations(x, cfg.x_dtype) @ wr.T).astype(np.float32))
    got = route_on_gpu(l, 4, routing="sigmoid", norm=True, rsf=1.5,
                       bias=dev(np.asarray(lay.expert_bias(), np.float32)))
    for n in ("idx", "sorted_pairs", "expert_offsets", "token_to_perm"):
        np.testing.assert_array_equal(got[n], want[n].reshape(got[n].shape), err_msg=n)
    # logits summed in another order (256 products) and both sides' roundings
    np.testing.assert_allclose(got["weights"], want["w"].reshape(m, 4), rtol=1e-4)


# ---- quantisation --------------------------------------------------------------------------------

def quantise_on_gpu(x, ld_codes=None, offset=0):
    rows, k = x.shape
    ldq = ld_codes or k
    full = torch.full((rows * ldq + 64,), 55, dtype=torch.int8, device="cuda")
    codes = full[16 + offset: 16 + offset + rows * ldq]
    scales = torch.full((rows + 2,), 77.0, device="cuda")
    B.moe_quantize_rows_int8(rows, k, F32 if x.dtype == torch.float32 else BF16, x, x.stride(0), codes,
                             ldq, scales[1:-1], torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert scales[0] == 77 and scales[-1] == 77
    assert torch.all(full[:16 + offset] == 55) and torch.all(full[16 + offset + rows * ldq:] == 55)
    q = codes.view(rows, ldq)
    assert torch.all(q[:, k:] == 55)
    return q[:, :k].cpu().numpy(), scales[1:-1].cpu().numpy()


def check_quantise(x, got):
    codes, scales = rows_ref.quantize_rows(x.float().cpu().numpy())
    np.testing.assert_array_equal(got[1], scales)
    np.testing.assert_array_equal(got[0], codes)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 7), (3, 16), (64, 2048), (5, 2056), (2, 40000), (300, 768),
                                    (1025, 130), (17, 5120), (9, 1000), (4, 8192), (3, 8200), (6, 24)])
def test_quantise_rows(rows, k, dtype):
    rng = np.random.default_rng(k)
    x = dev(rng.standard_normal((rows, k)) * np.exp(2 * rng.standard_normal((rows, 1))), dtype)
    check_quantise(x, quantise_on_gpu(x))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,ldq,offset", [(8, 96, 0), (1, 95, 1), (0, 96, 3), (3, 104, 8), (8, 97, 0)])
def test_quantise_strides_and_alignment(dtype, pad, ldq, offset):
    rng = np.random.default_rng(9)
    wide = torch.full((21 * (95 + pad) + 16,), float("nan"), dtype=dtype, device="cuda")
    view = wide[pad % 8: pad % 8 + 21 * (95 + pad)].view(21, 95 + pad)[:, :95]
    view.copy_(dev(rng.standard_normal((21, 95)), dtype))
    check_quantise(view, quantise_on_gpu(view, ldq, offset))


def test_quantise_values_at_the_borders():
    rng = np.random.default_rng(10)
    f = np.finfo(np.float32)
    rows = [np.zeros(64), np.full(64, f.max), np.full(64, f.tiny), np.full(64, 2.0 ** -149),
            np.arange(64) * 2.0 ** -149, np.arange(64) * f.tiny]
    for e in (0, -60, 60):                            # exact halves of the scale: ties to even
        r = (np.arange(64) - 31.5) * 2.0 ** e
        r[0] = 127.0 * 2.0 ** e
        rows.append(r)
    for _ in range(200):                              # neighbours of a half, for awkward scales
        amax = np.float32(np.exp(rng.standard_normal()))
        sc = np.float32(np.float64(amax) / 127)
        r = ((rng.integers(-127, 127, 64) + 0.5) * np.float64(sc)).astype(np.float32)
        step = rng.integers(-1, 2, 64)
        r = np.where(step > 0, np.nextafter(r, np.float32(np.inf)),
                     np.where(step < 0, np.nextafter(r, np.float32(-np.inf)), r))
        r = np.clip(r, -amax, amax)
        r[0] = amax
        rows.append(r)
    x = np.array(rows, np.float64).astype(np.float32)
    bad = np.repeat(x[6:7], 3, axis=0)
    bad[0, 5], bad[1, 63], bad[2, 0] = np.nan, np.inf, -np.inf
    t = dev(np.concatenate([x, bad]))
    check_quantise(t, quantise_on_gpu(t))
    check_quantise(t.bfloat16(), quantise_on_gpu(t.bfloat16()))


def test_quantise_past_two_to_the_31_elements():
    rows, k = 140_001, 16384
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    tail = torch.randn(3, k, device="cuda", generator=g)
    x[-3:] = tail
    codes = torch.empty(rows, k, dtype=torch.int8, device="cuda")
    scales = torch.empty(rows, device="cuda")
    B.moe_quantize_rows_int8(rows, k, BF16, x, k, codes, k, scales, torch.cuda.current_stream())
    check_quantise(x[-3:], (codes[-3:].cpu().numpy(), scales[-3:].cpu().numpy()))
    assert torch.all(scales[:-3] == 1) and not torch.any(codes[:1000])


# ---- product -------------------------------------------------------------------------------------

def int8_matrix(w, scales):
    m = B.moe_matrix()
    m.format, m.packed, m.scales = B.MOE_FMT_INT8, w.data_ptr(), scales.data_ptr()
    m.expert_stride, m.scale_stride = w.stride(0), scales.stride(0) * 4
    return m


class Product:
    """Seeded operands of one product, on the host and the device."""

    def __init__(self, seed, rows, n, k, sizes=None, top_k=1, gather=False, weighted=False, act=None,
                 out_dtype=BF16, ld_x=None, ld_out=None, extreme=False, slack=0):
        rng = np.random.default_rng(seed)
        self.rows, self.n, self.k, self.top_k, self.act, self.out_dtype = rows, n, k, top_k, act, out_dtype
        E = 1 if sizes is None else len(sizes)
        self.E = E
        self.offsets = None if sizes is None else np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        x_rows = (rows + top_k - 1) // top_k if gather else rows
        self.x_rows = x_rows
        lo, hi = (-128, 128) if extreme else (-127, 128)
        draw = (lambda *s: rng.choice(np.array([-128, 127], np.int8), s)) if extreme else (
            lambda *s: rng.integers(lo, hi, s).astype(np.int8))
        self.x = draw(x_rows, k)
        self.xs = (0.02 * np.exp(0.3 * rng.standard_normal(x_rows))).astype(np.float32)
        self.w = [draw(E, n, k) for _ in range(2 if act else 1)]
        # the products of uniform codes have a deviation of about 73^2 sqrt(k): the gate lies near +-3
        self.ws = [(np.exp(0.3 * rng.standard_normal((E, n))) / (40.0 * math.sqrt(k))).astype(np.float32)
                   for _ in self.w]
        self.pairs = rng.permutation(x_rows * top_k)[:rows].astype(np.int32) if gather else None
        self.pw = rng.uniform(0.1, 1.0, x_rows * top_k).astype(np.float32) if weighted else None
        self.ld_x = ld_x or k
        self.ld_out = ld_out or n
        wide = np.full((x_rows, self.ld_x), 99, np.int8)
        wide[:, :k] = self.x
        self.dx, self.dxs = dev(wide), dev(self.xs)
        # `slack` bytes between experts, so that strides are not the matrices' own size
        self.dw = []
        for w in self.w:
            buf = np.full((E, n * k + slack), 88, np.int8)
            buf[:, : n * k] = w.reshape(E, -1)
            self.dw.append(dev(buf))
        self.dws = [dev(s) for s in self.ws]
        self.doff = None if self.offsets is None else dev(self.offsets)
        self.dpairs = None if self.pairs is None else dev(self.pairs)
        self.dpw = None if self.pw is None else dev(self.pw)
        self.cfg = B.moe_matmul_cfg(n=n, k=k, num_experts=E, top_k=top_k,
                                    activation=B.ACTIVATION_CODES[act or "swiglu"], out_dtype=out_dtype)
        self.mats = [int8_matrix(w, s) for w, s in zip(self.dw, self.dws)]
        self.ws_bytes = B.moe_matmul_workspace_bytes(self.cfg, rows)

    def new_out(self):
        self.full = torch.full((self.rows * self.ld_out + 64,), 7.0, dtype=DT[self.out_dtype],
                               device="cuda")
        return self.full[32: 32 + self.rows * self.ld_out]

    def call(self, out, ws, stream=None):
        B.moe_matmul_int8(self.cfg, self.x_rows, self.dx, self.ld_x, self.dxs, self.rows, self.doff,
                          self.dpairs, self.dpw, self.mats[0], self.mats[1] if self.act else None, out,
                          self.ld_out, ws, ws.numel(),
                          stream if stream is not None else torch.cuda.current_stream())

    def run(self):
        ws = workspace(self.ws_bytes)
        out = self.new_out()
        self.call(out, ws)
        torch.cuda.synchronize()
        assert status(ws) == B.MOE_OK
        assert torch.all(self.full[:32] == 7) and torch.all(self.full[32 + self.rows * self.ld_out:] == 7)
        grid = out.view(self.rows, self.ld_out)
        assert torch.all(grid[:, self.n:] == 7)
        return grid[:, : self.n].double().cpu().numpy()

    def check(self, got):
        want, size = rows_ref.matmul_int8(
            self.x, self.xs, self.w[0], self.ws[0], np.full((self.rows, self.n), 7.0), self.offsets,
            self.pairs, self.top_k, self.pw, *(([self.w[1], self.ws[1]]) if self.act else []),
            **(dict(activation=self.act) if self.act else {}))
        # Plain: the int32 sum is exact; its conversion, the weight on the scale and two products
        # round once each: 4. With an activation the gate's 4 roundings grow by its condition number
        # (silu, gelu: under 1 + |g| where it counts, |g| < 24 here), the exponential adds 2 + 1.2 |g|
        # of twice EPS, tanh's own error (1 + tanh cancels for negative g) counts against |g * u|, and
        # the other factor has 4 + 3: under 256 relative and 8 of |g * u|.
        bound = 4 * EPS * np.abs(want) if self.act is None else 256 * EPS * np.abs(want) + 8 * EPS * size
        bound = bound + HALF[self.out_dtype] * (np.abs(want) + bound) + 2.0 ** -126
        off = np.abs(got - want) > bound
        assert not off.any(), (int(off.sum()), np.argwhere(off)[:4].tolist(),
                               got[off][:4].tolist(), want[off][:4].tolist())


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 100, 127, 128, 129, 255, 256, 257,
                                  300, 513])
@pytest.mark.parametrize("n,k", [(128, 128), (200, 272)])
def test_product_row_counts(rows, n, k):
    p = Product(rows, rows, n, k, out_dtype=F32)
    p.check(p.run())


@pytest.mark.parametrize("act", [None, "swiglu", "geglu"])
@pytest.mark.parametrize("rows,n,k", [(1, 1, 16), (90, 1, 16), (3, 65, 48), (5, 127, 144), (40, 130, 2064), (130, 257, 1008),
                                      (270, 384, 512), (20, 1000, 4096), (600, 100, 128)])
def test_product_odd_sizes(rows, n, k, act):
    for dt in (F32, BF16):
        p = Product(n + k, rows, n, k, act=act, out_dtype=dt)
        p.check(p.run())


GROUPINGS = {
    "some empty": [0, 3, 0, 0, 17, 1, 0, 40],
    "one row each": [1] * 24,
    "one expert has all": [0, 0, 200, 0],
    "uneven": [5, 129, 64, 0, 256, 31, 300, 2],
    "tiles that end full": [128, 256, 0, 128, 64, 16],
}


@pytest.mark.parametrize("act", [None, "swiglu", "geglu"])
@pytest.mark.parametrize("gather,weighted", [(False, False), (True, False), (True, True)])
@pytest.mark.parametrize("sizes", list(GROUPINGS))
def test_product_over_experts(sizes, gather, weighted, act):
    s = GROUPINGS[sizes]
    tail = 5                                          # rows that no expert owns stay as they were
    p = Product(len(s), sum(s) + tail, 144, 208, sizes=s, top_k=3 if gather else 1, gather=gather,
                weighted=weighted, act=act, ld_x=224, ld_out=151, slack=48)
    got = p.run()
    p.check(got)
    assert np.all(got[sum(s):] == 7.0)


def test_product_sums_at_the_ends_of_their_range():
    """Codes of -128 and 127 over the longest k: sums near 2^31."""
    p = Product(1, 3, 40, 131056, extreme=True, out_dtype=F32)
    p.x[0] = -128
    p.w[0][0, 0] = -128
    p.dx, p.dw = dev(p.x), [dev(p.w[0].reshape(1, -1))]
    p.mats = [int8_matrix(p.dw[0], p.dws[0])]
    p.check(p.run())


@pytest.mark.parametrize("experts,rows,n,k,act", [(128, 128, 768, 2048, "swiglu"), (1, 1, 5120, 8192, None),
                                                  (1, 5, 640, 8192, "geglu"), (512, 900, 96, 256, None),
                                                  (32, 2000, 320, 1792, "swiglu"), (1, 777, 1024, 5120, None)])
def test_product_at_the_layers_sizes(experts, rows, n, k, act):
    rng = np.random.default_rng(experts)
    sizes = None
    if experts > 1:
        sizes = np.bincount(rng.integers(0, experts, rows), minlength=experts).tolist()
    p = Product(rows, rows, n, k, sizes=sizes, act=act)
    p.check(p.run())


def test_product_bad_pairs_leave_their_rows():
    p = Product(3, 40, 70, 64, sizes=[20, 20], top_k=2, gather=True)
    p.pairs[[0, 7, 39]] = [-1, 2 * p.x_rows, 2**31 - 1]
    p.dpairs = dev(p.pairs)
    got = p.run()
    p.check(got)
    assert np.all(got[[0, 7, 39]] == 7.0)


@pytest.mark.parametrize("offsets", [[-5, 10, 30], [0, 50, 60], [0, 2**31 - 1, 2**31 - 1], [30, 10, 20],
                                     [12, 12, 12]])
def test_product_bad_offsets_stay_inside(offsets):
    """Offsets outside the rows, or not ascending: nothing outside `out` is touched (the canaries in
    run()), whatever becomes of the rows."""
    p = Product(4, 40, 70, 64, sizes=[20, 20])
    p.doff = dev(np.array(offsets, np.int32))
    p.run()


def test_product_nan_scale_gives_nan_rows():
    p = Product(5, 20, 64, 64)
    p.dxs[3] = float("nan")
    got = p.run()
    assert np.isnan(got[3]).all() and np.isfinite(np.delete(got, 3, axis=0)).all()


@pytest.mark.parametrize("sizes", [[30, 0, 41], [200, 150, 90]])      # single blocks, pairs of blocks
@pytest.mark.parametrize("layout", ["up first", "one matrix twice", "other strides"])
def test_product_gate_and_up_wherever_they_lie(layout, sizes):
    p = Product(11, sum(sizes), 96, 208, sizes=sizes, act="swiglu", out_dtype=F32)
    E, size = len(sizes), 96 * 208
    if layout == "up first":                          # one allocation, up below gate
        both = torch.cat([p.dw[1].view(-1), p.dw[0].view(-1)])
        p.dw = [both[E * size:].view(E, size), both[: E * size].view(E, size)]
    elif layout == "one matrix twice":
        p.w[1], p.dw[1] = p.w[0], p.dw[0]
    else:
        wide = torch.full((E, size + 160), 5, dtype=torch.int8, device="cuda")
        wide[:, :size] = p.dw[1]
        p.dw[1] = wide
    p.mats = [int8_matrix(w, s) for w, s in zip(p.dw, p.dws)]
    p.check(p.run())


@pytest.mark.parametrize("rows,gather", [(20, False), (300, False), (300, True)])
def test_product_wait_that_runs_out(rows, gather):
    """A stage whose operands never all arrive: the call ends, and the workspace says so."""
    p = Product(12, rows, 128, 1024, sizes=[rows], top_k=2 if gather else 1, gather=gather)
    ws, out = workspace(p.ws_bytes), p.new_out()
    try:
        B.moe_debug_barrier_test(1, 2_000_000)
        p.call(out, ws)
        torch.cuda.synchronize()
        assert status(ws) == B.MOE_ERR_DEVICE_TIMEOUT
    finally:
        B.moe_debug_barrier_test(0, 0)
    p.check(p.run())


@pytest.mark.parametrize("rows", [3, 90])
@pytest.mark.parametrize("act", ["swiglu", "geglu"])
def test_product_of_a_shut_gate_is_zero_however_large(rows, act):
    """A gate far below zero times an up as large: their product passes float32, the activation is 0."""
    p = Product(13, rows, 64, 64, act=act, out_dtype=F32)
    p.dx.fill_(1)
    p.dw[0].fill_(-1)
    p.dw[1].fill_(1)
    p.dxs.fill_(1e12)
    for s in p.dws:
        s.fill_(1e12)
    got = p.run()
    assert np.all(got == 0)


def test_product_rows_do_not_depend_on_their_neighbours():
    """A row's bits are the same alone and within any batch."""
    p = Product(6, 300, 160, 528, out_dtype=F32)
    many = p.run()
    for r in (0, 130, 299):
        q = Product(6, 300, 160, 528, out_dtype=F32)
        q.rows = q.x_rows = 1
        q.dx, q.dxs = q.dx[r: r + 1].contiguous(), q.dxs[r: r + 1].contiguous()
        np.testing.assert_array_equal(q.run()[0], many[r])


def test_product_output_past_two_to_the_31_elements():
    rows, n, k = 70_001, 32_768, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(-127, 128, (rows, k), device="cuda", generator=g, dtype=torch.int8)
    w = torch.randint(-127, 128, (1, n, k), device="cuda", generator=g, dtype=torch.int8)
    xs, ws = torch.ones(rows, device="cuda"), torch.ones(1, n, device="cuda")
    out = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    cfg = B.moe_matmul_cfg(n=n, k=k, num_experts=1, top_k=1, activation=0, out_dtype=BF16)
    work = workspace(B.moe_matmul_workspace_bytes(cfg, rows))
    B.moe_matmul_int8(cfg, rows, x, k, xs, rows, None, None, None, int8_matrix(w, ws), None, out, n, work,
                      work.numel(), torch.cuda.current_stream())
    # sums of 16 products of integers are exact in float32
    at = torch.tensor([0, 1, 32_767, 65_535, 65_536, rows - 2, rows - 1], device="cuda")
    want = (x[at].float() @ w[0].float().t()).bfloat16()
    assert torch.equal(out[at], want) and status(work) == B.MOE_OK


def test_product_weights_past_two_to_the_31_bytes():
    E, n, k = 68, 4096, 8192
    w = torch.zeros(E, n, k, dtype=torch.int8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    w[-1] = torch.randint(-127, 128, (n, k), device="cuda", generator=g, dtype=torch.int8)
    x = torch.randint(-127, 128, (150, k), device="cuda", generator=g, dtype=torch.int8)
    xs, ws = torch.ones(150, device="cuda"), torch.ones(E, n, device="cuda")
    for rows in (3, 150):
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[-1] = rows
        out = torch.empty(rows, n, device="cuda")
        cfg = B.moe_matmul_cfg(n=n, k=k, num_experts=E, top_k=1, activation=0, out_dtype=F32)
        work = workspace(B.moe_matmul_workspace_bytes(cfg, rows))
        B.moe_matmul_int8(cfg, rows, x, k, xs, rows, off, None, None, int8_matrix(w, ws), None, out, n, work,
                          work.numel(), torch.cuda.current_stream())
        want = (x[:rows].double() @ w[-1].double().t())
        # one rounding of the exact sum
        assert torch.all((out.double() - want).abs() <= EPS * want.abs())


# ---- blend ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("y_dtype", [F32, BF16])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("rows,n,top_k,pad", [(1, 8, 1, 0), (5, 64, 8, 0), (64, 2048, 8, 0), (3, 7, 2, 0),
                                              (40, 130, 6, 3), (33, 257, 4, 8), (7, 1024, 16, 1), (200, 96, 3, 16)])
def test_combine(rows, n, top_k, pad, y_dtype, out_dtype):
    rng = np.random.default_rng(rows * n)
    P = rows * top_k
    y = torch.full((P, n + pad), float("nan"), dtype=DT[y_dtype], device="cuda")
    y[:, :n] = dev(rng.standard_normal((P, n)), DT[y_dtype])
    perm = rng.permutation(P).astype(np.int32)
    perm[rng.random(P) < 0.2] = -1
    if P > 6:
        perm[5] = P                                   # outside: adds nothing
    if rows > 2:
        perm[top_k: 2 * top_k] = -1                   # a row without experts
    w = rng.uniform(-1, 1, (rows, top_k)).astype(np.float32)
    sh = torch.full((rows, n + pad), float("nan"), dtype=DT[y_dtype], device="cuda")
    sh[:, :n] = dev(rng.standard_normal((rows, n)), DT[y_dtype])
    gate = rng.uniform(0, 1, rows).astype(np.float32)
    yn, shn = y[:, :n].double().cpu().numpy(), sh[:, :n].double().cpu().numpy()
    for ww, ss, gg in ((w, None, None), (None, None, None), (w, sh, None), (w, sh, gate), (None, sh, gate)):
        full = torch.full((rows * (n + pad) + 32,), 7.0, dtype=DT[out_dtype], device="cuda")
        out = full[16:-16]
        B.moe_combine_rows(rows, n, top_k, y_dtype, y, n + pad, P, dev(perm), None if ww is None else dev(ww),
                           ss, n + pad if ss is not None else 0, None if gg is None else dev(gg), out_dtype,
                           out, n + pad, torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert torch.all(full[:16] == 7) and torch.all(full[-16:] == 7)
        grid = out.view(rows, n + pad)
        assert torch.all(grid[:, n:] == 7)
        want, mag = rows_ref.combine(yn, perm, top_k, rows, ww, None if ss is None else shn, gg)
        bound = (top_k + 2) * EPS * mag               # one rounding per term of the running sum
        bound = bound + HALF[out_dtype] * (np.abs(want) + bound) + 2.0 ** -126
        got = grid[:, :n].double().cpu().numpy()
        assert np.all(np.abs(got - want) <= bound), float(np.max(np.abs(got - want) - bound))


def test_combine_skips_rows_it_does_not_name():
    """NaN in rows of y that no slot names stays out of the sums."""
    y = torch.full((8, 32), float("nan"), device="cuda")
    y[3] = 2.0
    out = torch.empty(2, 32, device="cuda")
    B.moe_combine_rows(2, 32, 2, F32, y, 32, 8, dev(np.array([3, -1, -1, -1], np.int32)), None, None, 0, None,
                       F32, out, 32, torch.cuda.current_stream())
    assert torch.all(out[0] == 2) and torch.all(out[1] == 0)


def test_combine_without_any_row_of_y():
    sh = torch.randn(3, 24, device="cuda")
    out = torch.empty(3, 24, device="cuda")
    perm = torch.full((6,), -1, dtype=torch.int32, device="cuda")
    B.moe_combine_rows(3, 24, 2, F32, None, 24, 0, perm, None, sh, 24, None, F32, out, 24, torch.cuda.current_stream())
    assert torch.equal(out, sh)


def test_combine_past_two_to_the_31_elements():
    rows, n = 66_000, 32_776
    y = torch.empty(rows, n, dtype=torch.bfloat16, device="cuda")
    y[-1] = torch.randn(n, device="cuda")
    y[-2] = torch.randn(n, device="cuda")
    perm = torch.tensor([rows - 1, rows - 2], dtype=torch.int32, device="cuda")
    out = torch.empty(1, n, device="cuda")
    B.moe_combine_rows(1, n, 2, BF16, y, n, rows, perm, None, None, 0, None, F32, out, n, torch.cuda.current_stream())
    assert torch.equal(out[0], y[-1].float() + y[-2].float())


def test_combine_more_rows_than_a_grid_axis_holds():
    rows = 70_000
    y = torch.arange(rows, device="cuda", dtype=torch.float32)[:, None].expand(rows, 8).contiguous()
    perm = torch.arange(rows - 1, -1, -1, device="cuda", dtype=torch.int32)
    out = torch.empty(rows, 8, device="cuda")
    B.moe_combine_rows(rows, 8, 1, F32, y, 8, rows, perm, None, None, 0, None, F32, out, 8,
                       torch.cuda.current_stream())
    assert torch.equal(out, y.flip(0))


# ---- together ------------------------------------------------------------------------------------

class Layer:
    """An int8 expert layer built from the row operators, as a program would hold it."""

    def __init__(self, T, h, inter, E, k, seed=0, **route):
        rng = np.random.default_rng(seed)
        self.T, self.h, self.I, self.E, self.k = T, h, inter, E, k
        self.wf = [(rng.standard_normal((E, a, b)) / math.sqrt(b)).astype(np.float32)
                   for a, b in ((inter, h), (inter, h), (h, inter))]
        packed = [[B.moe_quantize_int8(m) for m in w] for w in self.wf]
        self.q = [dev(np.stack([p[0] for p in w])) for w in packed]
        self.s = [dev(np.stack([p[1] for p in w])) for w in packed]
        self.mats = [int8_matrix(a, b) for a, b in zip(self.q, self.s)]
        opts = dict(routing="sigmoid", norm=True, rsf=1.0, groups=4, topk_groups=2, group_score="top2")
        opts.update(route)
        self.opts = opts
        self.bias = dev((rng.standard_normal(E) * 0.1).astype(np.float32))
        self.rcfg = B.moe_route_cfg(
            num_experts=E, top_k=k, routing=B.ROUTING_CODES[opts["routing"]], norm_topk_prob=int(opts["norm"]),
            select_on_raw_logits=0, has_expert_bias=1, routed_scaling_factor=opts["rsf"],
            num_groups=opts["groups"], topk_groups=opts["topk_groups"],
            group_score=B.GROUP_SCORE_CODES[opts["group_score"]], logits_dtype=F32)
        self.gu = B.moe_matmul_cfg(n=inter, k=h, num_experts=E, top_k=k, activation=0, out_dtype=BF16)
        self.dn = B.moe_matmul_cfg(n=h, k=inter, num_experts=E, top_k=k, activation=0, out_dtype=BF16)
        P = T * k
        z = dict(device="cuda")
        self.x = torch.empty(T, h, dtype=torch.bfloat16, **z)
        self.logits = torch.empty(T, E, **z)
        self.idx, self.pairs, self.perm = (torch.empty(P, dtype=torch.int32, **z) for _ in range(3))
        self.off = torch.empty(E + 1, dtype=torch.int32, **z)
        self.w = torch.empty(T, k, **z)
        self.xq, self.xs = torch.empty(T, h, dtype=torch.int8, **z), torch.empty(T, **z)
        self.act = torch.zeros(P, inter, dtype=torch.bfloat16, **z)
        self.aq, self.as_ = torch.empty(P, inter, dtype=torch.int8, **z), torch.empty(P, **z)
        self.y = torch.zeros(P, h, dtype=torch.bfloat16, **z)
        self.out = torch.empty(T, h, dtype=torch.bfloat16, **z)
        self.rws = workspace(B.moe_route_workspace_bytes(self.rcfg, T))
        self.mws = workspace(max(B.moe_matmul_workspace_bytes(self.gu, P),
                                 B.moe_matmul_workspace_bytes(self.dn, P)))
        self.set_inputs(seed)

    def set_inputs(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.x.copy_(torch.randn(self.T, self.h, device="cuda", generator=g))
        self.logits.copy_(torch.randn(self.T, self.E, device="cuda", generator=g))

    def forward(self, stream=None):
        st = stream if stream is not None else torch.cuda.current_stream()
        T, P, h, I = self.T, self.T * self.k, self.h, self.I
        B.moe_route_rows(self.rcfg, T, self.logits, self.E, self.bias, self.idx, self.w, self.pairs, self.off,
                         self.perm, self.rws, self.rws.numel(), st)
        B.moe_quantize_rows_int8(T, h, BF16, self.x, h, self.xq, h, self.xs, st)
        B.moe_matmul_int8(self.gu, T, self.xq, h, self.xs, P, self.off, self.pairs, None, self.mats[0],
                          self.mats[1], self.act, I, self.mws, self.mws.numel(), st)
        B.moe_quantize_rows_int8(P, I, BF16, self.act, I, self.aq, I, self.as_, st)
        B.moe_matmul_int8(self.dn, P, self.aq, I, self.as_, P, self.off, None, None, self.mats[2], None, self.y, h,
                          self.mws, self.mws.numel(), st)
        B.moe_combine_rows(T, h, self.k, BF16, self.y, h, P, self.perm, self.w, None, 0, None, BF16, self.out, h,
                           st)

    def float_reference(self):
        """The layer with the weights and activations unquantised, in float64."""
        ids, w = rows_ref.route(self.logits.cpu().numpy(), top_k=self.k, bias=self.bias.cpu().numpy(), **self.opts)
        x = self.x.double().cpu().numpy()
        out = np.zeros((self.T, self.h))
        for t in range(self.T):
            for e, g in zip(ids[t], w[t]):
                if e >= 0:
                    out[t] += g * moe_ref.swiglu_expert(*(m[e].astype(np.float64) for m in self.wf), x[t])
        return ids, out


@pytest.mark.parametrize("T,h,inter,E,k", [(1, 256, 128, 16, 4), (37, 256, 144, 16, 4), (150, 128, 96, 32, 6)])
def test_layer_of_row_operators(T, h, inter, E, k):
    L = Layer(T, h, inter, E, k, seed=T)
    L.forward()
    torch.cuda.synchronize()
    ids, want = L.float_reference()
    np.testing.assert_array_equal(L.idx.cpu().numpy().reshape(T, k), ids)
    got = L.out.double().cpu().numpy()
    # Rounding to 127 steps of the largest of m normal values errs by about max / 127 / sqrt(12), so
    # by 0.007 to 0.009 of the deviation for x and the weights; the act rows' largest value is
    # some 6 deviations: 0.014. The product of gate and up carries about 3 of the first kind and the
    # down product adds two: sqrt(3 * 2 * 0.009^2 + 0.014^2 + 0.009^2) = 0.028 in the 2-norm, bf16
    # another 0.003. Twice that bounds it.
    assert np.linalg.norm(got - want) <= 0.06 * np.linalg.norm(want)
    assert status(L.mws) == B.MOE_OK


def test_layer_captured_and_replayed():
    L = Layer(70, 256, 128, 16, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.forward(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.forward(torch.cuda.current_stream())
    for seed in (5, 6):
        L.set_inputs(seed)
        L.forward()
        torch.cuda.synchronize()
        want = {n: getattr(L, n).clone() for n in ("out", "idx", "w", "pairs", "off", "perm", "act", "y")}
        for n in want:
            getattr(L, n).zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n, t in want.items():
            assert torch.equal(getattr(L, n), t), n


def test_first_calls_of_a_process_inside_a_capture():
    """Nothing has to be called before a capture: the library's own set-up is no work on a stream."""
    code = """
import sys
sys.path[:0] = [%r, %r]
import torch
from test_row_ops_gpu import Layer
L = Layer(70, 256, 128, 16, 4)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    L.forward(torch.cuda.current_stream())
graph.replay()
torch.cuda.synchronize()
got = L.out.clone()
L.forward()
torch.cuda.synchronize()
assert torch.equal(got, L.out) and bool(L.out.any())
print("captured")
""" % (ROOT, os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_layers_on_two_streams_at_once():
    a, b = Layer(200, 256, 128, 16, 4, seed=1), Layer(90, 256, 128, 16, 4, seed=2)
    want = []
    for L in (a, b):
        L.forward()
        torch.cuda.synchronize()
        want.append(L.out.clone())
        L.out.zero_()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        a.forward(s1)
        b.forward(s2)
    torch.cuda.synchronize()
    assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])


def test_calls_repeat_bit_for_bit():
    p = Product(9, 700, 520, 1040, sizes=[100, 0, 350, 250], act="swiglu")
    first = p.run()
    for _ in range(5):
        np.testing.assert_array_equal(p.run(), first)
