"""GPU: the 8-bit form where its roundings show. A group's largest value runs
through every bf16 mantissa, and half of it is exactly between two codes."""

import numpy as np
import pytest
import torch

import ternary_weight_quantization_b200 as bl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
f = np.float32


def form(x):
    """Codes, scales and saved values as the header states them, in numpy's
    fp32: each operation rounded once."""
    M, K = x.shape
    G = -(-K // 128)
    v = np.zeros((M, G * 128), f)
    v[:, :K] = x.float().cpu().numpy()
    v = v.reshape(M, G, 128)
    a = np.maximum(np.abs(v).max(-1, keepdims=True), f(1e-30))
    inv = (f(1) / a) * f(127)
    codes = np.rint(v * inv)
    scale = a * (f(1) / f(127))
    values = codes * scale
    quotients = np.rint((v.astype(np.float64) * 127.0) / a.astype(np.float64))
    return tuple(torch.from_numpy(np.ascontiguousarray(t)).cuda() for t in (
        codes.reshape(M, -1)[:, :K].astype(np.int8), scale[:, :, 0], values.reshape(M, -1)[:, :K],
        quotients.reshape(M, -1)[:, :K].astype(np.int8)))


def groups(K, dtype):
    """Row r: the largest value of each group has mantissa 1 + r / 128."""
    r = torch.arange(128, dtype=F32)[:, None]
    c = torch.arange(K, dtype=F32)[None, :]
    a = (1 + r / 128) * 2.0 ** ((c // 128) * 5 - 3)
    part = torch.stack([torch.ones_like(c), torch.full_like(c, 0.5), torch.full_like(c, -0.5), torch.full_like(c, -1.0),
                        (c * 37 % 128) / 128, -(c * 29 % 64) / 128 - 2.0 ** -9])
    x = torch.empty(128, K)
    for i in range(K):
        x[:, i] = a[:, i] * part[i % 6, 0, i]
    return x.to(dtype).cuda()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [256, 264, 261])
def test_every_mantissa_and_ties(K, dtype):
    x = groups(K, dtype)
    M = x.shape[0]
    codes, scales, values, quotients = form(x)
    a, n, g, u = (bl.Act8.allocate(M, K) for _ in range(4))
    out, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(M, device="cuda")
    bl.bl_act8_encode(x, a)
    bl.bl_act8_decode(a, out)
    bl.bl_norm_forward(x, None, None, 1e-6, y, None, rstd, rms=True, saved8=n)
    bl.bl_swiglu_forward(x, x, y, g, u)
    torch.cuda.synchronize()
    assert bl.bl_get_last_error() == 0
    for s in (a, n, g, u):
        assert torch.equal(s.codes, codes) and torch.equal(s.scales, scales)
    assert torch.equal(out, values.to(dtype))
    # next to codes of the rounded quotient 127 x / a: another one only at a tie,
    # and as near. x inv is off by three roundings: 127 3 2^-24 < 2^-15
    assert int((codes.int() - quotients.int()).abs().max()) <= 1
    step = scales.repeat_interleave(128, 1)[:, :K].double()
    assert bool(((values.double() - x.double()).abs() <= (0.5 + 2.0 ** -14) * step).all())
    halves = torch.arange(K, device="cuda") % 6
    assert set(codes[:, halves == 1].unique().tolist()) <= {63, 64}
    assert set(codes[:, halves == 2].unique().tolist()) <= {-63, -64}
    assert bool((codes[:, halves == 0] == 127).all()) and bool((codes[:, halves == 3] == -127).all())


@pytest.mark.parametrize("K", [256, 261])
def test_constant_rows_exactly(K):
    x = torch.tensor([3.0, 1.0, -0.7, 1e-20, 3e38], device="cuda")[:, None].repeat(1, K)
    s, out = bl.Act8.allocate(*x.shape), torch.empty_like(x)
    bl.bl_act8_encode(x, s)
    bl.bl_act8_decode(s, out)
    torch.cuda.synchronize()
    want = [f(np.sign(v)) * f(127) * (f(abs(v)) * (f(1) / f(127))) for v in x[:, 0].cpu().numpy()]
    assert torch.equal(out, torch.tensor(np.array(want)).cuda()[:, None].expand_as(x))
    assert bool((s.codes.abs() == 127).all())
