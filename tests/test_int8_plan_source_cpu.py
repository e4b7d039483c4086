"""The INT8 product's host code as written: what host threads share."""

import os
import re

from tests.conftest import ROOT


def host_code():
    with open(os.path.join(ROOT, "ternary_weight_quantization_b200", "csrc", "k_int8.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return text[text.index("bool make_map("):]


def function(text, head):
    body = text[text.index(head):]
    return body[:body.index("\n}\n")]


def test_the_narrow_tiles_shared_memory_limit_has_one_value():
    """The question of how many clusters fit and a launch of the same kernel, from another
    thread, must not lower each other's limit."""
    text = host_code()
    for head in ("int clusters_at_once(", "cudaError_t launch_mid("):
        body = function(text, head)
        assert "cudaFuncSetAttribute" not in body and "allow_smem(" not in body and "allow_mid<" in body, head
    assert len(re.findall(r"allow_smem\(int8_mid_kernel", text)) == 1


def test_an_answer_that_failed_is_not_kept():
    body = function(host_code(), "int clusters_at_once(")
    kept = body.index("if (keep) known")
    assert "if (clusters <= 0) return" in body[:kept] and "std::atomic" in body
