"""Padded batches in the decoder LM, with the library's calls replaced by plain ones: ids
outside the vocabulary at a sequence's end are targets that are left out, and inputs of
positions that are left out too, so the loss and the gradients are the short batch's."""

import pytest
import torch

from tests import plain_calls, plain_lm
from workloads.lm import LM_TINY


@pytest.mark.parametrize("pad", [-100, -1, LM_TINY.vocab, 1 << 40])
@pytest.mark.parametrize("how", [dict(), dict(fused_norms=True), dict(head8=True), dict(fused_norms=True, head8=True)])
def test_a_padded_batch_is_the_short_batch(monkeypatch, how, pad):
    plain_calls.install(monkeypatch)
    init, ids = plain_lm.case(LM_TINY, 2)
    short = ids[:, :12]
    padded = torch.full_like(ids, pad)
    padded[:, :12] = short
    loss, got = plain_lm.of_library(init, padded, LM_TINY, "cpu", **how)
    want_loss, want = plain_lm.of_library(init, short, LM_TINY, "cpu", **how)
    # the same terms in sums of more zeros: fp32 sums over at most 128 logits and 34 tokens.
    # A logit or a gradient off by that may round to bf16 the other way, by 2^-7 of itself
    # (a whole step), in 9 products on the way and back
    assert abs(float(loss) - float(want_loss)) <= (128 + 34) * 2.0 ** -23 * float(want_loss)
    distance, name = plain_lm.far(got, {n: g.double() for n, g in want.items()})
    assert distance <= 18 * 2.0 ** -7, name
    assert all(bool(g.isfinite().all()) for g in got.values())


@pytest.mark.parametrize("pad", [-100, -1, LM_TINY.vocab])
def test_the_harness_leaves_padding_out_too(monkeypatch, pad):
    """The model in plain torch around the layers, in 64 bits."""
    from ternary_weight_quantization_b200 import lm
    monkeypatch.setattr(lm.BitLinearFunction, "apply", staticmethod(lambda x, w: x @ w.T))
    init, ids = plain_lm.case(LM_TINY, 2)
    params = {n: t.double().requires_grad_(True) for n, t in init.items()}
    padded = torch.full_like(ids, pad)
    padded[:, :12] = ids[:, :12]
    loss, want = lm.lm_loss(params, padded, LM_TINY), lm.lm_loss(params, ids[:, :12], LM_TINY)
    # the same terms, in sums of at most 128 and 34
    assert abs(float(loss.detach()) - float(want.detach())) <= (128 + 34) * 2.0 ** -52 * float(want.detach())
    assert all(bool(g.isfinite().all()) for g in torch.autograd.grad(loss, list(params.values())))


def test_ids_inside_embed_as_before():
    ids = torch.tensor([[0, 3, 127, 5]])
    embed = torch.randn(128, 64)
    one_hot = (ids.reshape(-1, 1) == torch.arange(128)).to(embed.dtype)
    assert torch.equal(one_hot, torch.nn.functional.one_hot(ids.reshape(-1), 128).to(embed.dtype))
