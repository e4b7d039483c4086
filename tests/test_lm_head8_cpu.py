"""The decoder LM with an 8-bit head, with the library's calls replaced by plain ones:
targets outside the vocabulary, and vocabularies of any size."""

import dataclasses
import math

import pytest
import torch

from tests import plain_calls
from ternary_weight_quantization_b200 import lm as plm
from workloads.lm import LM_TINY, lm_batches, lm_init


@pytest.fixture(autouse=True)
def _plain(monkeypatch):
    plain_calls.install(monkeypatch)


# The 8-bit operands are off by at most half a step, amax / 254 each: with 64 normed
# values (norm 8, amax up to 4) and head rows of norm 0.4 and amax up to 0.2 a logit by
# at most 8 * 8 * 0.2 / 254 + 8 * 4 / 254 * 0.4, a loss by twice that.
NEAR = 2 * (8 * 8 * 0.2 + 8 * 4 * 0.4) / 254


def model(cfg, ids, **how):
    init = lm_init(cfg, seed=2)
    init["head"] = torch.randn(init["head"].shape, generator=torch.Generator().manual_seed(3)) * 0.05
    params = {n: t.requires_grad_(True) for n, t in init.items()}
    loss = plm.lm_loss(params, ids, cfg, library_ops=True, **how)
    return loss, dict(zip(params, torch.autograd.grad(loss, list(params.values()))))


def last_target(value):
    """Two sequences, the last target (which no position reads) replaced."""
    ids = lm_batches(LM_TINY, seed=3)[0].clone()
    ids[0, -1] = value
    return ids


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("target", [-1, LM_TINY.vocab, -100, 10 ** 12])
def test_a_target_outside_the_vocabulary_leaves_its_token_out(target, fused):
    ids = last_target(target)
    loss, grads = model(LM_TINY, ids, head8=True, fused_norms=fused)
    other, _ = model(LM_TINY, ids)             # the library's own head follows the same rule
    assert abs(float(loss.detach()) - float(other.detach())) <= NEAR
    whole, _ = model(LM_TINY, last_target(5), head8=True, fused_norms=fused)
    assert abs(float(loss.detach()) - float(whole.detach())) > 1e-6
    assert all(bool(g.isfinite().all()) for g in grads.values())
    # its value does not matter
    again, same = model(LM_TINY, last_target(-7), head8=True, fused_norms=fused)
    assert torch.equal(loss, again) and all(torch.equal(grads[n], same[n]) for n in grads)


def test_no_target_at_all_gives_a_loss_of_0_and_no_gradients():
    cfg = dataclasses.replace(LM_TINY, seq=1)
    ids = torch.tensor([[3, -1], [4, cfg.vocab]])
    loss, grads = model(cfg, ids, head8=True)
    assert float(loss.detach()) == 0.0 and not any(bool(g.any()) for g in grads.values())


def test_mean_over_the_targets_inside():
    """The loss and its gradient, from the logits, against the formula in 64 bits."""
    g = torch.Generator().manual_seed(7)
    logits = torch.randn(40, 33, generator=g).requires_grad_(True)
    targets = torch.randint(-5, 38, (40,), generator=g)
    loss = plm._mean_loss(logits, targets)
    d, = torch.autograd.grad(loss, [logits])
    z = logits.detach().double()
    held = (targets >= 0) & (targets < 33)
    n = int(held.sum())
    assert 20 < n < 40
    p = torch.softmax(z, 1)
    want = -torch.log(p[held, targets[held]]).sum() / n
    one = torch.zeros_like(p)
    one[held, targets[held]] = 1.0
    grad = (p - one) * held[:, None] / n
    # fp32: a log-sum-exp of 33 terms and a sum of at most 40 losses; e^z's relative error is that of z
    assert abs(float(loss.detach()) - float(want)) <= (40 + 33 + 8) * 2.0 ** -24 * float(z.abs().amax() + math.log(33))
    assert bool(((d.double() - grad).abs() <= (33 + 16 * 4) * 2.0 ** -24 / n).all())


@pytest.mark.parametrize("vocab", [97, 103, 121, 128])
def test_a_vocabulary_of_any_size_has_gradients(vocab):
    cfg = dataclasses.replace(LM_TINY, vocab=vocab)
    ids = lm_batches(cfg, seed=3)[0]
    loss, grads = model(cfg, ids, head8=True)
    other, want = model(cfg, ids)
    assert abs(float(loss.detach()) - float(other.detach())) <= NEAR
    assert grads["head"].shape == (vocab, cfg.d)
    # dW = dz^T x_hat: x_hat is off by 4 / 254 of its norm at most, dz by exp(NEAR) - 1 of
    # each probability, so of a row's norm of about 1 by that times sqrt(1 / vocab), 0.02
    assert float((grads["head"] - want["head"]).norm()) <= 0.04 * float(want["head"].norm())


@pytest.mark.parametrize("V", [97, 100, 104])
def test_norm_head8_gradients_are_the_products(V):
    """NormHead8Function against the formula on the same codes."""
    M, K = 10, 64
    g = torch.Generator().manual_seed(V)
    x, r = torch.randn(M, K, generator=g).to(torch.bfloat16).float(), torch.randn(M, K, generator=g)
    gain, head = 1 + 0.2 * torch.randn(K, generator=g), 0.1 * torch.randn(V, K, generator=g)
    leaves = [t.requires_grad_(True) for t in (x, r, gain, head)]
    logits = plm.NormHead8Function.apply(*leaves[:3], 1e-6, head)
    assert logits.shape == (M, V)
    dy = torch.randn(M, V, generator=g).to(torch.bfloat16).float()
    got = torch.autograd.grad(logits, leaves, dy)
    total = (x + r).detach().double()
    rstd = torch.rsqrt(total.square().mean(1, keepdim=True) + 1e-6)
    y = total * rstd * gain.detach().double()
    a = y.abs().amax(1, keepdim=True)
    x_hat = torch.round(y * 127 / a) * (a / 127)
    assert got[3].shape == (V, K)
    # x_hat in bf16 once, and a code next to a tie that fp32 leaves elsewhere
    size = dy.double().abs().t() @ x_hat.abs()
    step = dy.double().abs().t() @ (a / 127).expand(M, K)
    assert bool(((got[3].double() - dy.double().t() @ x_hat).abs() <= 1.01 * 2.0 ** -8 * size + 0.02 * step).all())
    assert all(bool(t.isfinite().all()) and bool(t.any()) for t in got)
