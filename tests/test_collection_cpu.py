"""What the suite's collection leaves out, and the clipping's lists that are allowed,
shown by an error that comes behind the lists' checks and in front of the device."""

import pytest
import torch

from ternary_weight_quantization_b200 import bitlinear as b
from tests import conftest
from tests.test_quant_ops_cpu import _gc


class _Item:
    def __init__(self, nodeid, *keywords):
        self.nodeid, self.keywords, self.marks = nodeid, set(keywords), []

    def add_marker(self, mark):
        self.marks.append(mark.name)


UNSAFE = "tests/test_quant_ops_cpu.py::test_lists_that_are_allowed_reach_the_device[<lambda>0]"


@pytest.mark.parametrize("device,expect", [(True, ["skip", None, None]), (False, [None, "skip", None])])
def test_made_up_addresses_never_meet_a_device(monkeypatch, device, expect):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: device)
    items = [_Item(UNSAFE), _Item("tests/test_x_gpu.py::test_kernel", "gpu"), _Item("tests/test_x_cpu.py::test_host")]
    conftest.pytest_collection_modifyitems(None, items)
    assert [it.marks[0] if it.marks else None for it in items] == expect


@pytest.mark.parametrize("how", [
    dict(out=(0x30000, 0x20000)), dict(), dict(out=(0x30000, 0x30000 + 200)),
    dict(items=((0x10000, 100, 0), (0x10000 + 200, 4, 1), (None, 0, 0))),
])
def test_lists_that_are_allowed_get_as_far_as_the_workspace(how):
    lib = b.load_library()
    assert _gc(n=16, **how)(lib) == 8
    assert "workspace" in lib.bl_last_error_message().decode()
