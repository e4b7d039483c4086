"""Padded batches in the decoder LM on the GPU: ids outside the vocabulary at a
sequence's end leave the loss and the gradients of the short batch."""

import pytest
import torch

from tests import plain_lm
from workloads.lm import LM_TINY

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how", [dict(), dict(saved8=True), dict(fused_norms=True), dict(head8=True),
                                 dict(fused_norms=True, head8=True)])
@pytest.mark.parametrize("pad", [-100, LM_TINY.vocab])
def test_a_padded_batch_is_the_short_batch(how, pad):
    init, ids = plain_lm.case(LM_TINY, 2)
    short = ids[:, :12]
    padded = torch.full_like(ids, pad)
    padded[:, :12] = short
    loss, got = plain_lm.of_library(init, padded, LM_TINY, "cuda", **how)
    want_loss, want = plain_lm.of_library(init, short, LM_TINY, "cuda", **how)
    # attention and its sums run over other lengths, in another order: a code next to a tie
    # may be another one, as against the model written out
    distance, name = plain_lm.far(got, {n: g.double().cpu() for n, g in want.items()})
    assert distance <= plain_lm.NEAR, name
    # a logit: head rows of norm 0.2 * 8 times the normed stream's 8, off by 9 operands' halves of a step
    assert abs(float(loss) - float(want_loss)) <= 9 * 3.5 / 254 * 0.2 * 8
    assert all(bool(g.isfinite().all()) for g in got.values())
