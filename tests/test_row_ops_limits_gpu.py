"""GPU tests of the row operators at the limits of their arguments: values at the ends of float32, lengths
at the ends of 32 bits, and the batch sizes where the choice of a launch changes."""
import numpy as np
import pytest
import torch

from mixture_experts_decode_gemv_b200 import binding as B
from oracle import rows_ref
from test_row_ops_gpu import (BF16, DT, F32, Layer, Product, check_quantise, check_route, dev, int8_matrix, quantise_on_gpu,
                              route_on_gpu, status, workspace)

pytestmark = pytest.mark.gpu

F32_MAX = float(np.finfo(np.float32).max)
BF16_MAX = float(torch.finfo(torch.bfloat16).max)


def rows_at_the_ends(E, G, big, seed):
    """Rows whose groups hold logits near +-big: alone, beside ordinary ones, and beside masked ones."""
    rng = np.random.default_rng(seed)
    size = E // G
    l = rng.standard_normal((40, E)) * 1.5
    of = np.arange(E) // size
    l[0] = -big                                       # every pair of a group sums to -2 big
    l[1, of == 0] = -big                              # a group switched off by the lowest finite number ...
    l[2] = -np.inf
    l[2, of == 1] = -big                              # ... and needed, as nothing else is left but
    l[2, G // 2 * size] = 0.5                         # one expert
    l[3] = -np.inf
    l[3, of >= G - 2] = -big
    l[4] = big
    l[5, of % 2 == 1] = np.inf                        # as the largest finite logit
    l[6, ::size] = 0.9 * big                          # sums past the largest number, the highest in the last group
    l[6, 1::size] = big * np.linspace(0.3, 0.99, G)
    l[7, ::size] = big                                # equal sums past it: the lower groups
    l[7, 1::size] = big
    l[8, ::size] = big                                # big - big
    l[8, 1::size] = -big
    l[8, 2::size] = -big
    l[9] = np.where(rng.random(E) < 0.5, -big, l[9])
    for r in range(10, 30):                           # sums on both sides of the border
        l[r] = rng.uniform(-1.0, 1.0, E) * big
    for r in range(30, 40):
        l[r] = np.where(rng.random(E) < 0.7, -np.inf, rng.choice([-big, 0.75 * -big, 0.5 * -big], E))
    return l


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,G,keep", [(32, 4, 2), (256, 8, 4), (510, 17, 5), (512, 32, 7)])
@pytest.mark.parametrize("routing", ["sigmoid", "sqrtsoftplus"])
def test_route_group_sums_past_float32(routing, E, G, keep, dtype):
    """Groups are ranked by their sums as 64 bits hold them, and one with a finite logit is never masked."""
    t = dev(rows_at_the_ends(E, G, F32_MAX if dtype == torch.float32 else BF16_MAX, E), dtype)
    for score in ("top2", "max"):
        kw = dict(top_k=6, routing=routing, norm=True, raw=True, groups=G, topk_groups=keep, group_score=score)
        check_route(t, route_on_gpu(t, **kw), **kw)


@pytest.mark.parametrize("E,G,keep", [(32, 4, 2), (256, 8, 4), (512, 32, 7)])
@pytest.mark.parametrize("routing", ["sigmoid", "sqrtsoftplus"])
def test_route_biases_at_the_ends_of_float32(routing, E, G, keep):
    rng = np.random.default_rng(E)
    size = E // G
    l = rng.standard_normal((24, E)) * 1.5
    l[4:8, size:] = -np.inf                           # only the first group is left
    l[8:16] = np.where(rng.random((8, E)) < 0.8, -np.inf, l[8:16])
    t = dev(l, torch.float32)
    biases = []
    b = rng.standard_normal(E) * 0.1
    b[:size] = -F32_MAX                               # the first group switched off
    biases.append(b)
    b = rng.standard_normal(E) * 0.1
    b[::size], b[1::size] = 0.9 * F32_MAX, F32_MAX * np.linspace(0.3, 0.99, G)
    biases.append(b)
    biases.append(np.full(E, -F32_MAX))
    biases.append(np.where(np.arange(E) % size < 2, np.inf, 0.1 * rng.standard_normal(E)))
    for b in biases:
        for score in ("top2", "max"):
            kw = dict(top_k=6, routing=routing, norm=True, bias=dev(b.astype(np.float32)), groups=G, topk_groups=keep,
                      group_score=score)
            check_route(t, route_on_gpu(t, **kw), **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,G,keep", [(16, 1, 1), (160, 8, 3), (256, 1, 1), (510, 17, 5)])
def test_route_zeros_of_both_signs_tie(E, G, keep, dtype):
    rng = np.random.default_rng(E)
    l = np.where(rng.random((50, E)) < 0.5, 0.0, -0.0)
    l[25:] = np.where(rng.random((25, E)) < 0.9, l[25:], rng.integers(-1, 2, (25, E)))
    t = dev(l, dtype)
    assert bool(torch.signbit(t).any()) and not bool(torch.signbit(t).all())
    zero = torch.zeros(E, device="cuda")
    for kw in (dict(routing="softmax"), dict(routing="sigmoid", raw=True), dict(routing="sqrtsoftplus", bias=zero),
               dict(routing="sigmoid", bias=-zero)):
        for score in ("max", "top2"):
            kw = dict(kw, top_k=6, norm=True, groups=G, topk_groups=keep, group_score=score)
            check_route(t, route_on_gpu(t, **kw), **kw)


def test_quantise_the_longest_row():
    """A row of 2^31 - 1 elements: positions one step behind its end do not fit 31 bits."""
    k = 2**31 - 1
    x = torch.zeros(1, k, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 127, 128, 2**30, k - 129, k - 128, k - 2, k - 1], device="cuda")
    v = torch.tensor([127.0, -1.0, 2.5, 3.5, -64.0, 5.0, -127.0, 100.0], device="cuda")     # the scale is 1
    x[0, at] = v.bfloat16()
    full = torch.full((k + 512,), 55, dtype=torch.int8, device="cuda")
    scales = torch.full((3,), 77.0, device="cuda")
    B.moe_quantize_rows_int8(1, k, BF16, x, k, full[256:256 + k], k, scales[1:2], torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert scales.tolist() == [77.0, 1.0, 77.0]
    assert torch.all(full[:256] == 55) and torch.all(full[256 + k:] == 55)
    codes = full[256:256 + k]
    assert codes[at].tolist() == [127, -1, 2, 4, -64, 5, -127, 100]     # halves to even
    codes[at] = 0
    assert not torch.any(codes)


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("rows", [1, 7, 64])
def test_product_exchanges_the_sums_of_many_tiles(rows, act):
    """A long k split over clusters that take several tiles each: the blocks' sums change hands tile after tile in
    the same shared memory."""
    p = Product(rows, rows, 20480 if act is None else 10240, 8192, act=act, out_dtype=F32)
    first = p.run()
    p.check(first)
    for _ in range(20):
        np.testing.assert_array_equal(p.run(), first)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_combine_the_longest_row(dtype):
    n = 2**31 - 1
    y = torch.zeros(1, n, dtype=DT[dtype], device="cuda")
    at = torch.tensor([0, 1, 2**28, 2**30 + 1, n - 9, n - 8, n - 2, n - 1], device="cuda")
    y[0, at] = torch.arange(1, 9, device="cuda").to(DT[dtype])
    perm = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = torch.full((1,), 2.0, device="cuda")
    full = torch.full((n + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
    B.moe_combine_rows(1, n, 1, dtype, y, n, 1, perm, w, None, 0, None, BF16, full[64:64 + n], n,
                       torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.all(full[:64] == 7) and torch.all(full[64 + n:] == 7)
    out = full[64:64 + n]
    assert torch.equal(out[at].float(), 2.0 * torch.arange(1, 9, device="cuda"))
    out[at] = 0
    assert not torch.any(out)


@pytest.mark.parametrize("n", [2**31 - 1, 2**31 - 100, 2**31 - 200])
def test_product_of_almost_two_to_the_31_channels(n):
    k, rows = 16, 2
    w = torch.zeros(n * k, dtype=torch.int8, device="cuda").view(1, n, k)
    ws = torch.ones(1, n, device="cuda")
    at = torch.cat([torch.arange(300), 2**30 + torch.arange(300), n - 300 + torch.arange(300)]).cuda()
    g = torch.Generator(device="cuda").manual_seed(7)
    w[0, at] = torch.randint(-127, 128, (900, k), device="cuda", generator=g, dtype=torch.int8)
    x = torch.randint(-127, 128, (rows, k), device="cuda", generator=g, dtype=torch.int8)
    xs = torch.ones(rows, device="cuda")
    full = torch.full((rows * n + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
    cfg = B.moe_matmul_cfg(n=n, k=k, num_experts=1, top_k=1, activation=0, out_dtype=BF16)
    work = workspace(B.moe_matmul_workspace_bytes(cfg, rows))
    B.moe_matmul_int8(cfg, rows, x, k, xs, rows, None, None, None, int8_matrix(w, ws), None, full[64:], n, work,
                      work.numel(), torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert status(work) == B.MOE_OK
    assert torch.all(full[:64] == 7) and torch.all(full[64 + rows * n:] == 7)
    for r in range(rows):
        out = full[64 + r * n:64 + (r + 1) * n]
        # sums of 16 products of integers are exact in float32
        assert torch.equal(out[at], (w[0, at].float() @ x[r].float()).bfloat16())
        out[at] = 0
        assert not torch.any(out)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("norm", [False, True])
def test_route_roots_of_scores_below_float32(norm, dtype):
    """sqrt(softplus(l)) is a normal number down to l = -174, where e^l has long left float32."""
    l = np.stack([-87.0 - 0.5 * np.arange(64), -16.0 - 0.05 * np.arange(64), -100.0 - np.arange(64),
                  np.where(np.arange(64) % 9 == 0, -16.5, -110.0 + 0.25 * np.arange(64)),
                  np.random.default_rng(1).uniform(-120.0, -90.0, 64)])
    t = dev(l, dtype)
    zero = torch.zeros(64, device="cuda")
    for kw in (dict(), dict(raw=True, groups=8, topk_groups=3, group_score="top2"), dict(bias=zero),
               dict(groups=8, topk_groups=3, group_score="top2"),
               dict(bias=zero, groups=8, topk_groups=3, group_score="top2")):
        kw = dict(kw, top_k=16, routing="sqrtsoftplus", norm=norm)
        check_route(t, route_on_gpu(t, **kw), **kw)


@pytest.mark.parametrize("routing", ["sigmoid", "sqrtsoftplus"])
@pytest.mark.parametrize("E,G,keep", [(256, 1, 1), (320, 4, 2), (512, 8, 4), (510, 17, 5), (512, 32, 7)])
def test_route_close_keys_among_large_biases(routing, E, G, keep):
    """Keys that only 64 bits tell apart, beside experts whose biases are far from them on either side."""
    rng = np.random.default_rng(E + G)
    base = (rng.standard_normal(E) * 1.5).astype(np.float32)
    s = np.array([rows_ref.score(float(v), routing) for v in base])
    l = np.repeat(base[None], 40, axis=0)
    l[::2] += (rng.standard_normal((20, E)) * 2.0 ** -22).astype(np.float32)
    t = dev(l)
    flat = (0.5 - s).astype(np.float32)
    for at, far in ((E // 3, -1e9), (E // 3, -3e4), (E // 3, 1e4), (E - 1, 2.0 ** 20), (0, -2.0 ** 120)):
        b = flat.copy()
        b[at] = far
        b[(at + 5) % E] = far                         # the score is lost in the rounding of this sum
        for score in ("max", "top2"):
            kw = dict(top_k=8, routing=routing, norm=True, bias=dev(b), groups=G, topk_groups=keep, group_score=score)
            check_route(t, route_on_gpu(t, **kw), **kw)


def route_time(l, **kw):
    """Microseconds of one call of the routing without a host between the calls: the best of several graphs' replays."""
    T, E = l.shape
    bias = kw.get("bias")
    cfg = B.moe_route_cfg(num_experts=E, top_k=8, routing=B.ROUTING_CODES["sigmoid"], norm_topk_prob=1,
                          select_on_raw_logits=int(bias is None), has_expert_bias=int(bias is not None),
                          routed_scaling_factor=1.0, num_groups=8, topk_groups=4, group_score=B.MOE_GROUP_TOP2,
                          logits_dtype=F32)
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, pairs, perm, off = (torch.empty(n, **i32) for n in (T * 8, T * 8, T * 8, E + 1))
    w = torch.empty(T * 8, device="cuda")
    ws = torch.empty(B.moe_route_workspace_bytes(cfg, T), dtype=torch.uint8, device="cuda")
    def call():
        B.moe_route_rows(cfg, T, l, E, bias, idx, w, pairs, off, perm, ws, ws.numel(), torch.cuda.current_stream())
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(20):
            call()
    best = float("inf")
    for _ in range(8):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3 / 20)
    return best


def test_route_time_does_not_hang_on_one_far_value():
    """An expert switched off by a large finite bias, or by a logit of the lowest finite number, leaves the other experts'
    keys as far apart as they were: the rows are still settled in 32 bits."""
    g = torch.Generator(device="cuda").manual_seed(1)
    l = torch.randn(8191, 256, device="cuda", generator=g)
    bias = 0.1 * torch.randn(256, device="cuda", generator=g)
    far = bias.clone()
    far[100] = -1e9
    lowest = l.clone()
    lowest[:, 100] = -F32_MAX
    times = [route_time(l, bias=bias), route_time(l, bias=far), route_time(l), route_time(lowest)]
    print("us:", times)
    assert times[1] < 1.3 * times[0] and times[3] < 1.3 * times[2], times


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,G,keep", [(16, 1, 1), (31, 1, 1), (256, 1, 1), (256, 8, 8), (256, 8, 4), (510, 17, 9), (512, 1, 1)])
def test_route_saturated_scores_rank_beyond_float32(E, G, keep, dtype):
    """sigmoid(30) and sigmoid(31) are both 1 in 32 bits. Many equal logits come before the one that 64 bits rank first."""
    rng = np.random.default_rng(E)
    e = np.arange(E)
    l = np.full((24, E), 30.0)
    l[0, E - 1] = 31
    l[1, E // 2:] = 35
    l[2] = rng.integers(25, 37, E)
    l[3] = np.where(e < 2, 30, rng.integers(28, 34, E))
    l[4] = np.where(e == E - 2, 36, -30)
    l[5] = e % 3 + 30
    l[7] = np.where(e % 5 == 4, 33, 30)
    for r in range(8, 24):
        l[r] = np.where(rng.random(E) < 0.8, 30, rng.integers(29, 32, E))
    t = dev(l, dtype)
    step = np.where(e % 7 == 6, 0.5, 0.25).astype(np.float32)
    for b in (np.zeros(E, np.float32), np.full(E, 0.25, np.float32), step, -step, 1e6 * step):
        for k in (1, 3, 8, 15):
            kw = dict(top_k=k, routing="sigmoid", norm=True, bias=dev(b), groups=G, topk_groups=keep, group_score="top2")
            check_route(t, route_on_gpu(t, **kw), **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [8 * g for g in (1, 32, 33, 64, 65, 96, 97, 127, 128, 129, 256, 257, 384, 385, 640, 641, 1024, 1025,
                                              1536, 1537, 2560, 2561, 4096, 4097)])
def test_quantise_around_every_change_of_the_launch(k, dtype):
    rng = np.random.default_rng(k)
    x = dev(rng.standard_normal((5, k)), dtype)
    x[3, -1] = 40.0
    check_quantise(x, quantise_on_gpu(x))


@pytest.mark.parametrize("rows", [16, 17, 24, 25, 1183, 1184, 1185, 1193])
@pytest.mark.parametrize("E,G,keep", [(64, 4, 3), (512, 1, 1)])
def test_route_row_counts_where_the_launch_changes(rows, E, G, keep):
    """One launch up to 16 rows; blocks of eight rows up to 148 of them (1184 rows), longer blocks beyond."""
    rng = np.random.default_rng(rows)
    l = rng.standard_normal((rows, E))
    l[rows // 2] = -np.inf
    l[-1, 1:] = -np.inf
    t = dev(l, torch.float32)
    kw = dict(top_k=6, routing="sigmoid", norm=True, groups=G, topk_groups=keep)
    check_route(t, route_on_gpu(t, **kw), **kw)


def test_layer_forked_and_joined_in_a_graph():
    """Two layers on streams of their own between the same ends, captured and replayed: a call waits for all that its
    stream waits for, whatever kind of work that was."""
    a, b = Layer(130, 256, 128, 16, 4, seed=1), Layer(60, 256, 128, 16, 4, seed=2)
    both = torch.empty(190, 256, dtype=torch.bfloat16, device="cuda")
    gate = torch.ones(130, device="cuda")
    perm = torch.arange(130, dtype=torch.int32, device="cuda")
    last = torch.empty(130, 256, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()

    def run():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        a.forward(main)
        with torch.cuda.stream(side):
            b.forward(side)
            both[130:].copy_(b.out)
        both[:130].copy_(a.out)
        main.wait_stream(side)
        # reads what both streams wrote
        B.moe_combine_rows(130, 256, 1, BF16, both[:130], 256, 130, perm, None, both[60:], 256, gate, BF16, last, 256, main)
        a.x.copy_(last)                               # ... and the next pass reads this

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            run()
    want = None
    for replay in (False, True, True):
        a.set_inputs(5)
        b.set_inputs(6)
        torch.cuda.synchronize()
        if replay:
            graph.replay()
        else:
            for _ in range(3):
                run()
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        got = [t.clone() for t in (a.out, b.out, both, last)]
        want = want or got
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert bool(want[3].any()) and status(a.mws) == B.MOE_OK and status(b.mws) == B.MOE_OK


@pytest.mark.parametrize("lo,hi", [(-206, -176), (-190, -188), (-200, -199.5), (-172, -171.9)])
def test_route_scores_below_the_normal_numbers(lo, hi):
    """sqrt(softplus(l)) = e^(l/2) has a few bits left in 32 bits, or none."""
    t = dev(np.random.default_rng(3).uniform(lo, hi, (200, 64)), torch.float32)
    zero = torch.zeros(64, device="cuda")
    for kw in (dict(bias=zero), dict(bias=zero, groups=8, topk_groups=3, group_score="top2"),
               dict(groups=8, topk_groups=3, group_score="top2")):
        kw = dict(kw, top_k=8, routing="sqrtsoftplus", norm=True)
        check_route(t, route_on_gpu(t, **kw), **kw)
