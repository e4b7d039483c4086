"""Which gradients clip_gradients copies and which it scales where they are, with the
library's call replaced by its formula."""

import pytest
import torch

from ternary_weight_quantization_b200 import lm as plm


@pytest.fixture(autouse=True)
def _plain_clip(monkeypatch):
    def clip(grads, most, norm, workspace):
        spans = sorted((g.data_ptr(), g.data_ptr() + g.numel() * g.element_size()) for g in grads if g.numel())
        assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:])), "the library refuses gradients that overlap"
        assert all(g.is_contiguous() for g in grads)
        norm.copy_(torch.sqrt(sum(g.double().square().sum() for g in grads)))
        for g in grads:
            g.mul_(min(1.0, most / float(norm)))
    monkeypatch.setattr(plm.b, "bl_clip_grads", clip)


def rnd(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def check(grads, in_place):
    """grads are clipped right, and those at `in_place` in their own memory."""
    keep = [g.clone() for g in grads]
    total = float(torch.sqrt(sum(k.double().square().sum() for k in keep)))
    got, norm = plm.clip_gradients(grads, 1.0)
    assert abs(float(norm) - total) <= 2.0 ** -23 * total
    for i, (g, k) in enumerate(zip(got, keep)):
        # the factor and the product are rounded to fp32 once each
        assert torch.allclose(g.double(), k.double() / total, rtol=3 * 2.0 ** -24, atol=0.0), i
    assert [g is h or (g.data_ptr() == h.data_ptr() and g.shape == h.shape) for g, h in zip(got, grads)] == in_place
    for i, stays in enumerate(in_place):
        if stays:
            assert torch.equal(grads[i], got[i])


def test_views_side_by_side_in_one_buffer_are_scaled_where_they_are():
    flat = rnd(1000)
    grads = [flat[:300].view(30, 10), flat[300:301], flat[301:301], flat[301:900].view(599), flat[900:]]
    whole = flat.double() / flat.double().norm()
    check(grads, [True] * 5)
    assert torch.allclose(flat.double(), whole, rtol=3 * 2.0 ** -24, atol=0.0)


def test_views_in_any_order():
    flat = rnd(640, seed=1)
    check([flat[64 * i:64 * (i + 1)] for i in (7, 0, 9, 3, 1, 8, 2, 6, 4, 5)], [True] * 10)


def test_overlapping_and_strided_gradients_are_copied():
    a, flat = rnd(40, 30), rnd(100, seed=2)
    check([a, a, rnd(30, 40, seed=1).t()], [True, False, False])
    check([flat[10:50], flat[49:60], flat[:11], flat[60:]], [True, False, False, True])
    check([flat[:10], flat[20:30], flat[5:25]], [True, True, False])
    check([rnd(3, 1, seed=4).expand(3, 5), torch.zeros(0), rnd(7, seed=5)], [False, True, True])
