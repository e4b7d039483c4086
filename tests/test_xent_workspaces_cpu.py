"""Workspace sizes of the head cross-entropy: buffers made for one call serve the
calls that a training loop makes with them. The size functions need no GPU."""

import random

import pytest
import torch

import ternary_weight_quantization_b200 as bl

BF, F32 = torch.bfloat16, torch.float32
size = bl.bl_linear_xent_backward_workspace_size


def shapes(n, seed):
    rng = random.Random(seed)

    def spread(lo, hi):
        return int(lo * (hi / lo) ** rng.random())
    return [(spread(1, 131072), spread(1, 1 << 20), 8 * spread(1, 1024)) for _ in range(n)]


@pytest.mark.parametrize("M,V,K", [(391, 1739, 3312), (512, 8192, 4096), (256, 151936, 2048), (30, 8192, 512), (2048, 50304, 768)])
def test_fp32_buffer_serves_a_call_for_dh_alone(M, V, K):
    assert size(M, V, K, F32) >= size(M, V, K, BF) > 0


def test_fp32_size_is_never_below_the_bf16_size():
    for M, V, K in shapes(20000, 1):
        assert size(M, V, K, F32) >= size(M, V, K, BF) > 0, (M, V, K)
