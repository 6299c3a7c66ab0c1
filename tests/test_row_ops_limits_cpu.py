"""CPU tests of the row operators at their limits: refusals, and rules that the kernels' sources keep."""
import os
import re

import numpy as np
import pytest
import torch

from mixture_experts_decode_gemv_b200 import binding as B

pytestmark = pytest.mark.cpu

CSRC = os.path.join(os.path.dirname(os.path.abspath(B.__file__)), "csrc")


def source(name):
    return open(os.path.join(CSRC, name)).read()


def test_arrivals_that_hand_over_plain_shared_memory_release_at_cluster_scope():
    """The buffer of the blocks' sums is written and read by plain stores and loads: no fence stands before an arrival
    on its barriers, so the arrival itself orders them for the other blocks."""
    arrivals = re.findall(r"(bar_arrive\w*)\(of_rank\(smem_addr\(&sh\.(red_\w+)", source("matmul_int8.cu"))
    assert sorted(arrivals) == [("bar_arrive_release", "red_free"), ("bar_arrive_release", "red_full")]
    body = re.search(r"void bar_arrive_release\(.*?\n\}", source("tc05.cuh"), re.S).group(0)
    assert "mbarrier.arrive.release.cluster.shared::cluster" in body


def test_addresses_as_plain_integers_are_taken_at_once():
    """An integer is asked for no method: looking for one raises inside, 0.4 us for each argument of each call."""
    class Address(int):
        def __getattr__(self, name):
            raise RuntimeError(f"asked for {name}")

    assert B._ptr(Address(4096)) == 4096 and B._ptr(0) == 0 and B._ptr(None) is None
    t, a = torch.empty(3), np.empty(3)
    assert B._ptr(t) == t.data_ptr() and B._ptr(a) == a.ctypes.data
    with pytest.raises(TypeError):
        B._ptr("x")
    with pytest.raises(ValueError):
        B._ptr(np.empty((4, 4))[:, ::2])


def test_route_workspace_never_shrinks_where_the_launch_changes():
    for E in (1, 3, 130, 512):
        c = B.moe_route_cfg(num_experts=E, top_k=1, routing=0, norm_topk_prob=1, select_on_raw_logits=0, has_expert_bias=0,
                            routed_scaling_factor=1.0, num_groups=1, topk_groups=1, group_score=0, logits_dtype=B.MOE_FMT_F32)
        sizes = [B.moe_route_workspace_bytes(c, r) for r in (0, 1, 15, 16, 17, 24, 25, 1183, 1184, 1185, 1193, 2**31 - 1)]
        assert sizes == sorted(sizes) and all(s % 256 == 0 for s in sizes)
