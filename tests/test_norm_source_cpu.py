"""The norms' kernels as written: shared memory that is accessed 8 bytes at a
time through its address is declared of a type that is aligned so."""

import os
import re

from tests.conftest import ROOT


def test_buffers_of_paired_sums_are_aligned():
    with open(os.path.join(ROOT, "ternary_weight_quantization_b200", "csrc", "k_norm.cu")) as f:
        kernels = f.read().split("__global__")[1:]
    users = [k for k in kernels if "group_sum2(" in k]
    assert len(users) == 2
    for k in users:
        kind, = re.findall(r"__shared__ (\w+) sums\[", k)
        assert kind in ("float2", "float4"), k[:80]
