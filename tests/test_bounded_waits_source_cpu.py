"""The kernels' bounded waits as written. A wait that runs out returns to a warp whose
lanes look at the barrier one by one; what follows (tcgen05.ld, ldmatrix, mma.sync, a
vote) takes the whole warp, so the warp has to decide as one. One lane's own waits, in
a branch that only it takes, need no vote."""

import os
import re

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "ternary_weight_quantization_b200", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_the_warps_wait_votes():
    body = code("bl_mma.cuh").split("mbar_wait_warp(", 1)[1].split("}", 1)[0]
    assert "__all_sync(0xffffffffu, mbar_wait(" in body


@pytest.mark.parametrize("name", ["k_int8.cu", "k_xent.cu"])
def test_waits_are_the_warps(name):
    text = code(name)
    assert re.search(r"\bmbar_wait_warp\(", text)
    assert not re.findall(r"\bmbar_wait\([^\n]*", text), "a wait that each lane decides for itself"
