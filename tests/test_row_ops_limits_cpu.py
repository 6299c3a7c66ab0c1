"""CPU tests of the row operators at their limits: refusals, and rules that the kernels' sources keep."""
import os
import re

import pytest

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
