"""How the decoder LM puts its calls together, with each call replaced by a plain one:
every parameter's gradient against the model written out, which a projection's output
that is lost, added twice or added behind the next norm moves far away."""

import pytest

from tests import plain_calls, plain_lm
from workloads.lm import LM_TINY

HOW = [dict(), dict(fused_norms=True), dict(head8=True), dict(fused_norms=True, head8=True)]


@pytest.mark.parametrize("seed", [2, 3])
@pytest.mark.parametrize("how", HOW)
def test_gradients_are_those_of_the_model(monkeypatch, how, seed):
    plain_calls.install(monkeypatch)
    init, ids = plain_lm.case(LM_TINY, seed)
    _, got = plain_lm.of_library(init, ids, LM_TINY, "cpu", **how)
    _, want = plain_lm.gradients(init, ids, LM_TINY, head8=how.get("head8", False))
    distance, name = plain_lm.far(got, want)
    assert distance <= plain_lm.NEAR, name
    for what in ("lost", "twice", "late"):
        for k in range(2 * LM_TINY.layers):
            _, other = plain_lm.gradients(init, ids, LM_TINY, head8=how.get("head8", False), mistake=(what, k))
            assert plain_lm.far(got, other)[0] > 1.5 * plain_lm.NEAR, (what, k)
