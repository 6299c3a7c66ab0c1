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
