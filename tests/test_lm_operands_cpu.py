"""What the LM hands to the training operators, without a GPU."""

import torch

from ternary_weight_quantization_b200 import lm as plm


def test_operands_are_dense_and_on_16_bytes():
    ids = torch.arange(9)[None]
    t = ids[:, 1:].reshape(-1)
    assert t.is_contiguous() and t.data_ptr() % 16 == 8      # a view into ids
    for x in (t, torch.arange(40.0)[3:33].view(5, 6), torch.arange(40.0).view(5, 8).t(), torch.arange(9, dtype=torch.bfloat16)[1:]):
        y = plm._operand(x)
        assert torch.equal(x, y) and y.dtype == x.dtype and y.is_contiguous() and y.data_ptr() % 16 == 0
    x = torch.arange(8.0)
    assert plm._operand(x) is x
