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


def test_the_layers_products_keep_their_warps_together():
    """k_gemm.cu: one lane multiplies, in a branch of its own; every other role's lanes
    decide together, on the wait or (loads, rebuilding) at the end of the tile."""
    text = code("k_gemm.cu")
    kernel = text[text.index("auto agreed = "):]
    kernel = kernel[:kernel.index("tmem_dealloc_pair(")]
    own = kernel.index("if (leader && lane == 0) {", kernel.index("warp == kWarpMma"))
    end = kernel.index("mma_commit_pair(done_bar", own)
    waits = list(re.finditer(r"(\S+ ?\S*?)\bwait\((&?\w+)", kernel))
    assert len(waits) == 6
    for m in waits:
        assert own < m.start() < end or m.group(1).endswith("agreed(") or kernel[:m.end()].rstrip().endswith(
            ("ok &= wait(&empty", "ok &= wait(&src_full")), m.group(0)
    # a loop whose lanes may differ ends by a vote, and has no other way out
    assert kernel.count("agreed(ok) && next_tile(") == kernel.count("ok &= wait(") == 2
    for part in kernel.split("agreed(ok) && next_tile(")[1:]:
        assert "break" not in part[:part.index("phase ^= 1;", part.index("ok &= wait("))]
    # who failed loads nothing and arrives nowhere
    assert len(re.findall(r"lane == 0 && ok\) (?:issued_parity|mbar_arrive_cluster)", kernel)) == 2
    stage = text[text.index("void load_stage("):]
    stage = stage[:stage.index("\ntemplate") if "\ntemplate" in stage else stage.index("\n}\n")]
    assert "if (lane == 0 && ok) {" in stage
    copies = stage[stage.index("if (ok) {"):]
    copies = copies[:copies.index("__syncwarp();")]
    assert stage.count("cp_async_8(") == copies.count("cp_async_8(") == copies.count("cp_async_mbar_arrive(") == 1
