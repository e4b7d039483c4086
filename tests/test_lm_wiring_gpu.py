"""The decoder LM's gradients, with the residual's addition fused into the norms and with
an 8-bit head, against the model written out in 64 bits and against its separate calls."""

import pytest

from tests import plain_lm
from workloads.lm import LM_TINY

pytestmark = pytest.mark.gpu

HOW = [dict(), dict(fused_norms=True), dict(head8=True), dict(fused_norms=True, head8=True)]


@pytest.mark.parametrize("seed", [2, 3])
@pytest.mark.parametrize("how", HOW)
def test_gradients_are_those_of_the_model(how, seed):
    init, ids = plain_lm.case(LM_TINY, seed)
    _, got = plain_lm.of_library(init, ids, LM_TINY, "cuda", **how)
    _, want = plain_lm.gradients(init, ids, LM_TINY, head8=how.get("head8", False))
    distance, name = plain_lm.far(got, want)
    assert distance <= plain_lm.NEAR, name


@pytest.mark.parametrize("how", HOW[1:])
def test_gradients_are_those_of_the_separate_calls(how):
    init, ids = plain_lm.case(LM_TINY, 2)
    _, got = plain_lm.of_library(init, ids, LM_TINY, "cuda", **how)
    _, want = plain_lm.of_library(init, ids, LM_TINY, "cuda")
    distance, name = plain_lm.far(got, {n: t.double().cpu() for n, t in want.items()})
    assert distance <= plain_lm.NEAR, name
