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


@pytest.mark.parametrize("M,short,V,K", [(2048, 1310, 50257, 768), (257, 256, 8192, 512), (17, 16, 8192, 512), (100, 9, 32000, 2048),
                                         (4096, 1, 32000, 2560), (777, 300, 50001, 1000)])
def test_a_short_batch_fits(M, short, V, K):
    assert bl.bl_linear_xent_forward_workspace_size(short, V, K) <= bl.bl_linear_xent_forward_workspace_size(M, V, K)
    for dt in (BF, F32):
        assert 0 < size(short, V, K, dt) <= size(M, V, K, dt)


def test_sizes_never_shrink_with_more_tokens():
    rng = random.Random(2)
    for M, V, K in shapes(4000, 3):
        # neighbours, the ends of the kernels' and the tiles' ranges, anything below
        for less in {max(1, M - 1), min(M, 16), min(M, 17), max(1, M // 256 * 256), rng.randint(1, M)}:
            assert bl.bl_linear_xent_forward_workspace_size(less, V, K) <= bl.bl_linear_xent_forward_workspace_size(M, V, K), (less, M, V, K)
            for dt in (BF, F32):
                assert size(less, V, K, dt) <= size(M, V, K, dt), (less, M, V, K, dt)


def planned(M, V, K, f32):
    """Bytes that the backward of more than 16 tokens lays out: dz of a piece
    (two terms for an fp32 dW), h, a factor, dH's partial sums."""
    def up(a, b):
        return -(-a // b)
    most = max((128 << 20) // (M * (4 if f32 else 2)) // 256 * 256, 256)
    pieces = up(up(V, 256) * 256, most)
    piece = up(up(V, pieces), 256) * 256
    pieces = up(V, piece)
    vcount = min(V, piece)
    tm, tk, tv, nkb = up(M, 256), up(K, 256), up(vcount, 256), up(vcount, 64)
    wkb = up(min(M, 1024) if f32 else M, 64) * (2 if f32 else 1) + 8
    share = (tm * tk * nkb + tv * tk * wkb) // 74 + 8
    slices = 1 if tm * tk >= 74 else max(1, min(up(3 * nkb, 2 * share), 32, nkb))
    sums = slices * tm * 256 * K * 4 if pieces > 1 or slices > 1 else 0
    return M * piece * (4 if f32 else 2) + up(M * K * 2, 256) * 256 + 256 + sums


def test_sizes_cover_what_the_backward_lays_out():
    for M, V, K in shapes(20000, 4) + [(17, 1 << 24, 8), (131072, 1, 65536), (131072, 1 << 24, 8), (300, 70, 4096)]:
        if M <= 16:
            continue
        assert planned(M, V, K, False) <= size(M, V, K, BF), (M, V, K)
        assert max(planned(M, V, K, True), planned(M, V, K, False)) <= size(M, V, K, F32), (M, V, K)
        # and not by more than the bound on dH's slices leaves
        assert size(M, V, K, BF) <= max(planned(M, V, K, False), 128 << 20) + (111 + 2 * 74) * 256 * 256 * 4 + 64 * V + (1 << 20), (M, V, K)
