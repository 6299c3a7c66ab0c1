"""CPU tests of the row operators: refusals before any launch, the int8 host helpers, and pins of
their oracle against the decode layer's oracle, closed forms and brute force."""
import ctypes
import itertools
import os
import re

import numpy as np
import pytest
import torch

from mixture_experts_decode_gemv_b200 import binding as B
from mixture_experts_decode_gemv_b200.synthetic import LayerConfig
from oracle import moe_ref, rows_ref

pytestmark = pytest.mark.cpu

FAKE = 0x7F0000000000
NO_GPU = (B.MOE_ERR_CUDA, B.MOE_ERR_UNSUPPORTED_DEVICE)


def route_cfg(**kw):
    c = dict(num_experts=16, top_k=4, routing=0, norm_topk_prob=1, select_on_raw_logits=0,
             has_expert_bias=0, routed_scaling_factor=1.0, num_groups=1, topk_groups=1, group_score=0,
             logits_dtype=B.MOE_FMT_F32)
    c.update(kw)
    return B.moe_route_cfg(**c)


def route(c, rows=4, logits=FAKE, ld=16, bias=None, idx=FAKE, weights=FAKE, pairs=FAKE, offsets=FAKE,
          perm=FAKE, ws=FAKE, wsb=1 << 30):
    return B.lib.moe_route_rows(ctypes.byref(c) if c else None, rows, logits, ld, bias, idx, weights,
                                pairs, offsets, perm, ws, wsb, None)


def test_struct_fields_match_the_header():
    text = open(os.path.join(os.path.dirname(B.LIB_PATH), "..", "include", "moe_decode.h")).read()
    for name, struct in (("moe_route_cfg", B.moe_route_cfg), ("moe_matmul_cfg", B.moe_matmul_cfg)):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, re.S).group(1)
        assert re.findall(r"(?:int32_t|float)\s+(\w+);", body) == [f[0] for f in struct._fields_]
    for limit in ("MOE_ROUTE_MAX_EXPERTS", "MOE_ROUTE_MAX_TOP_K", "MOE_ROUTE_MAX_GROUPS"):
        assert int(re.search(r"#define %s (\d+)" % limit, text).group(1)) == getattr(B, limit)


@pytest.mark.parametrize("change,status", [
    (dict(num_experts=0), "BAD_SHAPE"), (dict(num_experts=513), "BAD_SHAPE"),
    (dict(top_k=0), "BAD_SHAPE"), (dict(top_k=17, num_experts=32), "BAD_SHAPE"),
    (dict(num_groups=0), "BAD_SHAPE"), (dict(num_groups=3), "BAD_SHAPE"),
    (dict(num_experts=66, num_groups=33, topk_groups=33), "BAD_SHAPE"),
    (dict(num_groups=4, topk_groups=5), "BAD_SHAPE"), (dict(num_groups=4, topk_groups=0), "BAD_SHAPE"),
    (dict(num_groups=8, topk_groups=1, top_k=3), "BAD_SHAPE"),
    (dict(routing=3), "BAD_OPTION"), (dict(norm_topk_prob=2), "BAD_OPTION"),
    (dict(select_on_raw_logits=1), "BAD_OPTION"), (dict(has_expert_bias=1), "BAD_OPTION"),
    (dict(routing=1, select_on_raw_logits=1, has_expert_bias=1), "BAD_OPTION"),
    (dict(group_score=2), "BAD_OPTION"), (dict(routed_scaling_factor=float("inf")), "BAD_OPTION"),
    (dict(logits_dtype=B.MOE_FMT_NVFP4), "BAD_FORMAT"),
])
def test_route_cfg_refusals(change, status):
    c = route_cfg(**change)
    want = getattr(B, "MOE_ERR_" + status)
    assert route(c, ld=512) == want
    n = ctypes.c_size_t()
    assert B.lib.moe_route_workspace_bytes(ctypes.byref(c), 4, ctypes.byref(n)) == want


def test_route_call_refusals():
    c = route_cfg()
    assert route(None) == B.MOE_ERR_NULL_POINTER
    assert route(c, rows=-1) == B.MOE_ERR_BAD_SHAPE
    assert route(c, rows=1 << 30) == B.MOE_ERR_BAD_SHAPE          # pairs pass 2^31 - 1
    assert route(c, ld=15) == B.MOE_ERR_BAD_SHAPE
    for name in ("logits", "idx", "weights", "pairs", "offsets", "perm", "ws"):
        assert route(c, **{name: None}) == B.MOE_ERR_NULL_POINTER, name
    for name in ("logits", "idx", "weights", "pairs", "offsets", "perm"):
        assert route(c, **{name: FAKE + 2}) == B.MOE_ERR_MISALIGNED, name
    assert route(c, ws=FAKE + 128) == B.MOE_ERR_MISALIGNED
    assert route(c, wsb=16) == B.MOE_ERR_WORKSPACE
    assert route(c, bias=FAKE) == B.MOE_ERR_BAD_OPTION            # a bias the options do not read
    assert route(route_cfg(routing=1, has_expert_bias=1)) == B.MOE_ERR_NULL_POINTER
    assert route(c, rows=0, logits=None, pairs=None, offsets=None, perm=None, ws=None) == B.MOE_OK
    if not torch.cuda.is_available():
        assert route(c) in NO_GPU
        assert route(c, pairs=None, offsets=None, perm=None, ws=None) in NO_GPU


def test_route_workspace_never_shrinks_with_rows():
    c = route_cfg(num_experts=512, top_k=8)
    sizes = [B.moe_route_workspace_bytes(c, r) for r in (0, 1, 63, 64, 65, 100, 1000, 10**5, 10**8)]
    assert sizes == sorted(sizes) and all(s % 256 == 0 for s in sizes)


def matrix(fmt=B.MOE_FMT_INT8, n=64, k=64, packed=FAKE, scales=FAKE, stride=None, sstride=None):
    m = B.moe_matrix()
    m.format, m.packed, m.scales = fmt, packed, scales
    m.expert_stride = n * k if stride is None else stride
    m.scale_stride = n * 4 if sstride is None else sstride
    return m


def matmul(c=None, x_rows=8, x=FAKE, ld=64, xs=FAKE, rows=8, offsets=FAKE, pairs=None, pw=None, w=None,
           up=None, out=FAKE, ldo=64, ws=FAKE, wsb=1 << 30, **kw):
    base = dict(n=64, k=64, num_experts=4, top_k=2, activation=0, out_dtype=B.MOE_FMT_BF16)
    base.update(kw)
    c = c or B.moe_matmul_cfg(**base)
    w = matrix() if w is None else w
    return B.lib.moe_matmul_int8(ctypes.byref(c), x_rows, x, ld, xs, rows, offsets, pairs, pw,
                                 ctypes.byref(w), ctypes.byref(up) if up is not None else None, out,
                                 ldo, ws, wsb, None)


def test_matmul_refusals():
    bad = [
        (dict(n=0), "BAD_SHAPE"), (dict(k=0), "BAD_SHAPE"), (dict(k=24), "BAD_FORMAT"),
        (dict(k=131072, ld=131072), "BAD_SHAPE"), (dict(num_experts=0), "BAD_SHAPE"),
        (dict(num_experts=513), "BAD_SHAPE"), (dict(top_k=0), "BAD_SHAPE"), (dict(top_k=17), "BAD_SHAPE"),
        (dict(activation=2), "BAD_OPTION"), (dict(out_dtype=B.MOE_FMT_INT8), "BAD_FORMAT"),
        (dict(rows=-1), "BAD_SHAPE"), (dict(rows=1 << 31), "BAD_SHAPE"), (dict(x_rows=-1), "BAD_SHAPE"),
        (dict(x_rows=7), "BAD_SHAPE"), (dict(ld=48), "BAD_SHAPE"), (dict(ldo=63), "BAD_SHAPE"),
        (dict(ld=72), "MISALIGNED"), (dict(x=FAKE + 8), "MISALIGNED"), (dict(xs=FAKE + 2), "MISALIGNED"),
        (dict(offsets=FAKE + 2), "MISALIGNED"), (dict(pairs=FAKE + 1), "MISALIGNED"),
        (dict(out=FAKE + 1), "MISALIGNED"), (dict(ws=FAKE + 16), "MISALIGNED"),
        (dict(offsets=None), "NULL_POINTER"), (dict(x=None), "NULL_POINTER"),
        (dict(xs=None), "NULL_POINTER"), (dict(out=None), "NULL_POINTER"), (dict(ws=None), "NULL_POINTER"),
        (dict(wsb=0), "WORKSPACE"), (dict(pw=FAKE), "BAD_OPTION"),
        (dict(w=matrix(fmt=B.MOE_FMT_FP8_E4M3)), "BAD_FORMAT"), (dict(w=matrix(packed=None)), "NULL_POINTER"),
        (dict(w=matrix(scales=None)), "NULL_POINTER"), (dict(w=matrix(packed=FAKE + 8)), "MISALIGNED"),
        (dict(w=matrix(stride=64 * 64 + 8)), "MISALIGNED"), (dict(w=matrix(stride=64 * 48)), "BAD_SHAPE"),
        (dict(w=matrix(sstride=250)), "MISALIGNED"), (dict(w=matrix(sstride=128)), "BAD_SHAPE"),
        (dict(up=matrix(fmt=B.MOE_FMT_BF16)), "BAD_FORMAT"),
    ]
    for kw, status in bad:
        assert matmul(**kw) == getattr(B, "MOE_ERR_" + status), (kw, status)
    assert matmul(rows=0) == B.MOE_OK
    if not torch.cuda.is_available():
        for kw in (dict(), dict(up=matrix()), dict(pairs=FAKE, pw=FAKE, x_rows=4),
                   dict(num_experts=1, offsets=None)):
            assert matmul(**kw) in NO_GPU, kw


def test_quantise_and_combine_refusals():
    def quant(rows=4, k=8, dt=0, x=FAKE, ld=8, q=FAKE, ldq=8, s=FAKE):
        return B.lib.moe_quantize_rows_int8(rows, k, dt, x, ld, q, ldq, s, None)
    assert quant(rows=-1) == quant(k=0) == quant(ld=7) == quant(ldq=7) == B.MOE_ERR_BAD_SHAPE
    assert quant(rows=1 << 31) == B.MOE_ERR_BAD_SHAPE
    assert quant(dt=2) == B.MOE_ERR_BAD_FORMAT
    assert quant(x=None) == quant(q=None) == quant(s=None) == B.MOE_ERR_NULL_POINTER
    assert quant(x=FAKE + 2) == quant(s=FAKE + 1) == B.MOE_ERR_MISALIGNED
    assert quant(rows=0, x=None) == B.MOE_OK

    def comb(rows=4, n=8, k=2, ydt=1, y=FAKE, ldy=8, yrows=8, perm=FAKE, w=FAKE, sh=None, ldsh=0,
             gate=None, odt=1, out=FAKE, ldo=8):
        return B.lib.moe_combine_rows(rows, n, k, ydt, y, ldy, yrows, perm, w, sh, ldsh, gate, odt, out,
                                      ldo, None)
    for kw in (dict(rows=-1), dict(n=0), dict(k=0), dict(k=17), dict(yrows=-1), dict(ldy=7),
               dict(ldo=7), dict(sh=FAKE, ldsh=7), dict(rows=1 << 30, k=4)):
        assert comb(**kw) == B.MOE_ERR_BAD_SHAPE, kw
    assert comb(ydt=3) == comb(odt=6) == B.MOE_ERR_BAD_FORMAT
    assert comb(gate=FAKE) == B.MOE_ERR_BAD_OPTION
    assert comb(y=None) == comb(perm=None) == comb(out=None) == B.MOE_ERR_NULL_POINTER
    for kw in (dict(y=FAKE + 1), dict(perm=FAKE + 2), dict(w=FAKE + 2), dict(out=FAKE + 1),
               dict(sh=FAKE + 1, ldsh=8), dict(sh=FAKE, ldsh=8, gate=FAKE + 2)):
        assert comb(**kw) == B.MOE_ERR_MISALIGNED, kw
    assert comb(rows=0, y=None) == B.MOE_OK
    if not torch.cuda.is_available():
        assert quant() in NO_GPU and comb() in NO_GPU


def test_decode_layer_refuses_int8_weights():
    from mixture_experts_decode_gemv_b200.device_layer import make_cfg
    c = make_cfg(LayerConfig(name="v", hidden=64, num_experts=4, top_k=2, moe_inter=64))
    t = B.moe_expert_table(matrix(), matrix(), matrix())
    n = ctypes.c_int32()
    assert B.lib.moe_decode_launches(ctypes.byref(c), 1, ctypes.byref(t), None,
                                     ctypes.byref(n)) == B.MOE_ERR_BAD_FORMAT


def test_int8_host_quantiser_and_decoder():
    rng = np.random.default_rng(7)
    w = (rng.standard_normal((9, 64)) * 10.0 ** rng.integers(-3, 3, (9, 1))).astype(np.float32)
    w[2] = 0.0
    w[3, 5] = np.inf
    w[4] *= np.float32(2.0 ** -140)                   # below the smallest scale
    w[5, :] = np.arange(64) - 31.5                    # halves of its own scale
    w[5, 0] = 127.0
    packed, scales = B.moe_quantize_int8(w)
    codes, sc = rows_ref.quantize_rows(w)
    np.testing.assert_array_equal(packed, codes)
    np.testing.assert_array_equal(scales, sc)
    assert scales[2] == 1.0 and np.isnan(scales[3]) and not packed[3].any()
    ok = [r for r in range(9) if r != 3]
    # half a step of the stored scale
    assert np.all(np.abs(packed[ok].astype(np.float64) * scales[ok, None] - w[ok])
                  <= 0.5 * scales[ok, None].astype(np.float64) * (1 + 2.0 ** -22))
    dec = B.moe_dequantize(B.MOE_FMT_INT8, packed, scales, None, None, 9, 64)
    np.testing.assert_array_equal(dec[ok], packed[ok].astype(np.float32) * scales[ok, None])
    assert B.moe_packed_bytes(B.MOE_FMT_INT8, 10, 64) == (640, 40, 0)
    with pytest.raises(B.MoeError):
        B.moe_packed_bytes(B.MOE_FMT_INT8, 10, 40)


# ---- pins of the oracle --------------------------------------------------------------------------

@pytest.mark.parametrize("routing,raw,bias", [("softmax", False, False), ("sigmoid", False, True),
                                              ("sigmoid", True, False), ("sqrtsoftplus", False, True)])
def test_oracle_without_groups_is_the_decode_layers(routing, raw, bias):
    rng = np.random.default_rng(3)
    cfg = LayerConfig(name="r", hidden=64, num_experts=24, top_k=5, moe_inter=64, routing=routing,
                      norm_topk_prob=True, select_on_raw_logits=raw, has_expert_bias=bias,
                      routed_scaling_factor=2.5)
    l = rng.standard_normal((20, 24))
    b = rng.standard_normal(24) * 0.2 if bias else None
    ids, w = rows_ref.route(l, top_k=5, routing=routing, norm=True, raw=raw, bias=b, rsf=2.5)
    for r in range(20):
        want_ids, want_w = moe_ref.route_row(l[r], cfg, b)
        assert list(ids[r]) == list(want_ids)
        np.testing.assert_allclose(w[r], want_w, rtol=1e-12)
    g = rows_ref.group(ids, 24)
    want = moe_ref.group_by_expert(ids, 24)
    for name, key in (("sorted_pairs", "sorted_pairs"), ("expert_offsets", "expert_offsets"),
                      ("token_to_perm", "token_to_perm")):
        np.testing.assert_array_equal(g[name], np.asarray(want[key]))


def test_oracle_groups_against_every_subset():
    """The kept groups are those of the best total among all subsets (distinct scores)."""
    rng = np.random.default_rng(4)
    for _ in range(20):
        l = rng.standard_normal(12)
        s = 1.0 / (1.0 + np.exp(-l))
        worth = np.sort(s.reshape(4, 3), axis=1)[:, 1:].sum(axis=1)
        best = max(itertools.combinations(range(4), 2), key=lambda c: worth[list(c)].sum())
        pool = [e for e in range(12) if e // 3 in best]
        want = sorted(pool, key=lambda e: -l[e])[:4]
        ids, w = rows_ref.route_row(l, top_k=4, routing="sigmoid", norm=False, groups=4, topk_groups=2,
                                    group_score="top2")
        assert ids == want
        np.testing.assert_allclose(w, s[want], rtol=1e-12)


def test_oracle_masks_and_underflow():
    ids, w = rows_ref.route_row([-np.inf, np.nan, 1.0, -np.inf], top_k=3, routing="softmax", norm=False)
    assert ids == [2, -1, -1] and w == [1.0, 0.0, 0.0]
    ids, w = rows_ref.route_row([-np.inf] * 4, top_k=2, routing="sigmoid", norm=True)
    assert ids == [-1, -1] and w == [0.0, 0.0]
    ids, w = rows_ref.route_row([-2000.0, -2001.0], top_k=2, routing="sigmoid", norm=True)
    np.testing.assert_allclose(w, [1 / (1 + np.exp(-1)), 1 - 1 / (1 + np.exp(-1))], rtol=1e-12)
    ids, w = rows_ref.route_row([-2000.0, -2002.0], top_k=2, routing="sqrtsoftplus", norm=True)
    np.testing.assert_allclose(w, [1 / (1 + np.exp(-1)), 1 - 1 / (1 + np.exp(-1))], rtol=1e-12)
    assert rows_ref.route_row([np.inf, 3.0], top_k=2, routing="softmax", norm=False)[1] == [1.0, 0.0]


def test_oracle_product_and_blend_by_hand():
    x = np.array([[1, -2], [3, 4]], np.int8)
    w = np.array([[[1, 1]], [[2, -1]]], np.int8)
    xs, ws = np.array([0.5, 2.0], np.float32), np.array([[2.0], [4.0]], np.float32)
    out, _ = rows_ref.matmul_int8(x, xs, w, ws, np.full((5, 1), 9.0), offsets=[0, 2, 4],
                                  pairs=[0, 3, 1, 2, -1], top_k=2)
    # pairs 0, 3 -> rows 0, 1 (expert 0); pairs 1, 2 -> rows 0, 1 (expert 1)
    np.testing.assert_array_equal(out[:, 0], [-1 * 0.5 * 2, 7 * 2 * 2, 4 * 0.5 * 4, 2 * 2 * 4, 9.0])
    got, mag = rows_ref.combine(out, [0, 2, -1, 1], 2, 2, weights=np.array([[1, 0.5], [7, 0.25]]),
                                shared=np.array([[1.0], [2.0]]), gate=np.array([3.0, 0.5]))
    np.testing.assert_array_equal(got[:, 0], [-1 + 4 + 3, 7 + 1])
    np.testing.assert_array_equal(mag[:, 0], [1 + 4 + 3, 7 + 1])
