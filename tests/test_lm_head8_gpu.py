"""The decoder LM's 8-bit head on the GPU: vocabularies that are no multiple of 8, and
targets outside the vocabulary."""

import dataclasses

import pytest
import torch

from ternary_weight_quantization_b200 import lm as plm
from workloads.lm import LM_TINY, lm_batches, lm_init

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [97, 103, 128, 1001])
@pytest.mark.parametrize("M", [1, 20, 50, 300])
def test_head8_gradients_of_any_vocabulary(M, V):
    """The rows that fill the codes up leave nothing in dX, and dW has the head's rows."""
    K, eps = 64, 1e-6
    g = torch.Generator().manual_seed(1000 * M + V)
    x, r = torch.randn(M, K, generator=g).to(torch.bfloat16).float().cuda(), torch.randn(M, K, generator=g).cuda()
    gain, head = (1 + 0.2 * torch.randn(K, generator=g)).cuda(), (0.1 * torch.randn(V, K, generator=g)).cuda()
    dy = torch.randn(M, V, generator=g).to(torch.bfloat16).float().cuda()
    wide = torch.zeros(-(-V // 8) * 8, K, device="cuda")
    wide[:V] = head
    out = []
    for h, d in ((head, dy), (wide, torch.nn.functional.pad(dy, (0, wide.shape[0] - V)))):
        leaves = [t.clone().requires_grad_(True) for t in (x, r, gain, h)]
        logits = plm.NormHead8Function.apply(*leaves[:3], eps, leaves[3])
        out.append((logits.detach(), *torch.autograd.grad(logits, leaves, d)))
    # a head with those rows written out: scales of 1e-5 / 127 for them, and the same sums
    assert torch.equal(out[0][0], out[1][0][:, :V])
    for a, w in zip(out[0][1:4], out[1][1:4]):
        assert torch.equal(a, w)
    assert torch.equal(out[0][4], out[1][4][:V])


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("target", [-1, 97, -100])
def test_a_target_outside_the_vocabulary(target, fused):
    cfg = dataclasses.replace(LM_TINY, vocab=97)
    init = lm_init(cfg, seed=2)
    init["head"] = torch.randn(init["head"].shape, generator=torch.Generator().manual_seed(3)) * 0.05
    ids = lm_batches(cfg, seed=3)[0]
    ids[0, -1] = target
    out = []
    for head8 in (True, False):
        params = {n: t.cuda().requires_grad_(True) for n, t in init.items()}
        loss = plm.lm_loss(params, ids.cuda(), cfg, library_ops=True, head8=head8, fused_norms=fused)
        grads = torch.autograd.grad(loss, list(params.values()))
        assert all(bool(t.isfinite().all()) for t in grads)
        out.append(float(loss.detach()))
    # either operand of a logit is off by half a step of 8 bits: with 64 normed values
    # (norm 8, amax up to 4) and head rows of norm 0.4 and amax up to 0.2
    assert abs(out[0] - out[1]) <= 2 * (8 * 8 * 0.2 + 8 * 4 * 0.4) / 254
