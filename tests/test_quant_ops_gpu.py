"""GPU: the norm with an INT8 result, the product of INT8 operands and the
gradients' norm and clipping against 64-bit forms.

Tolerances count roundings. u = 2^-24 is half a step of fp32 relative to the
value, ``half(dtype)`` that of the output's type. An fp32 value made by n
rounded operations on terms of magnitude A is off by at most about n u A.
"""

import math

import pytest
import torch

import ternary_weight_quantization_b200 as bl

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TINY = 2.0 ** -120
BF, F32 = torch.bfloat16, torch.float32


def half(dtype):
    return torch.finfo(dtype).eps / 2


def rnd(*shape, seed=0, dtype=F32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def close(got, want, tol, what):
    """|got - want| <= tol + the rounding to got's type, elementwise."""
    want = want.double()
    bound = tol + half(got.dtype) * (want.abs() + tol) + TINY
    bad = ~((got.double() - want).abs() <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float((got.double() - want).abs().max()), float(bound.max()))


def ok():
    torch.cuda.synchronize()
    assert bl.bl_get_last_error() == 0


# ----------------------------------------------------------------- the norm with an INT8 result
EPS = 1e-6
# x, stream, gain
TYPES = [(BF, BF, BF), (BF, BF, F32), (BF, F32, F32), (F32, F32, F32), (F32, F32, BF), (BF, F32, BF)]
# one vector, less than a warp, a warp's row, odd rows, blocks of each size, the widest
SIZES = [(1, 8), (3, 64), (1, 2560), (5, 1000), (2, 1024), (777, 1000), (129, 264), (300, 512), (2048, 512), (40, 4104),
         (17, 8192), (500, 2560), (33, 6912), (1200, 72)]


def norm_inputs(M, K, xt, st, pt, seed=0):
    x, r = rnd(M, K, seed=seed, dtype=xt), rnd(M, K, seed=seed + 1, dtype=st, scale=2.0)
    r[:, K // 3] *= 20                           # a feature much larger than the others
    w = (1 + rnd(K, seed=seed + 2, scale=0.3)).to(pt)
    return x, r, w


def check_forward(total, w, b, eps=EPS):
    """The forward's outputs against 64 bits, from the stream as it was kept."""
    K = total.shape[1]
    r = total.double()
    rstd = 1 / torch.sqrt((r * r).mean(1) + eps)
    # a thread adds at most 32 squares in pairs (16 roundings and a square's), then
    # 5 steps of a warp and 16 warps; the mean, eps; half of it all after the root,
    # whose own two steps and the factor 1 / K round too
    close(b.rstd, rstd, 26 * U * rstd, "rstd")
    y = r * rstd[:, None] * (1.0 if w is None else w.double())
    a = y.abs().amax(1).clamp(min=1e-5)
    close(b.sx, a / 127, 30 * U * a / 127, "sx")
    # a code is rint(t f): t and f carry at most 30 roundings
    off = (b.xq.double() - y * (127 / a)[:, None]).abs()
    assert bool((off <= 0.5 + 127 * 40 * U).all()), float(off.max())
    assert int(b.xq.min()) >= -127 and int(b.xq.max()) <= 127
    full = a > 1.1e-5
    assert bool((b.xq.abs().amax(1)[full] == 127).all())


def gradients(dy, dsum, total, w, eps=EPS):
    """d and dweight in 64 bits, and what their errors are relative to."""
    r, dy = total.double(), dy.double()
    rstd = 1 / torch.sqrt((r * r).mean(1, keepdim=True) + eps)
    n, g = r * rstd, dy * (1.0 if w is None else w.double())
    d = rstd * (g - n * (g * n).mean(1, keepdim=True))
    size = rstd * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dsum is not None:
        d, size = d + dsum.double(), size + dsum.double().abs()
    return d, size, (dy * n).sum(0), (dy * n).abs().sum(0)


def check_backward(dy, dsum, total, w, got, names=("dresidual", "dx")):
    d, size, dw, dwsize = gradients(dy, dsum, total, w)
    for name in names:
        if getattr(got, name) is not None:
            # n has rstd's 26 roundings, the row's sum its 26 + 40, and a few follow
            close(getattr(got, name), d, 80 * U * size, name)
    # a thread's rows, the groups and the partial rows follow one another
    M = total.shape[0]
    close(got.dweight, dw, (30 + M / 148 + 16 + 148) * U * dwsize, "dweight")


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("M,K", SIZES)
def test_norm_quant(M, K, types):
    xt, st, pt = types
    x, r, w = norm_inputs(M, K, xt, st, pt, seed=M + K)
    b = bl.NormQuantBuffers.allocate(M, K, xt, st, pt)
    bl.bl_norm_quant_forward(x, r, w, EPS, b.sum, b.rstd, b.xq, b.sx)
    ok()
    assert torch.equal(b.sum, (x.float() + r.float()).to(st))
    check_forward(b.sum, w, b)
    for dt in (BF, F32):
        dy, dsum = rnd(M, K, seed=7, dtype=dt), rnd(M, K, seed=8, dtype=st, scale=0.3)
        bl.bl_norm_quant_backward(dy, dsum, b.sum, w, b.rstd, b.dx, b.dresidual, b.dweight, b.workspace)
        ok()
        check_backward(dy, dsum, b.sum, w, b)
        if b.dx is not None:
            # one value, rounded to either type
            close(b.dx, b.dresidual.double(), 0, "dx")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K", [(1, 16), (70, 2560), (301, 520)])
def test_norm_quant_without_residual_gain_and_stream_gradient(M, K, dtype):
    x, _, w = norm_inputs(M, K, dtype, dtype, dtype)
    for gain in (w, None):
        b = bl.NormQuantBuffers.allocate(M, K, dtype, dtype, dtype)
        bl.bl_norm_quant_forward(x, None, gain, EPS, None, b.rstd, b.xq, b.sx)
        dy = rnd(M, K, seed=3, dtype=BF)
        bl.bl_norm_quant_backward(dy, None, x, gain, b.rstd, None, b.dresidual, b.dweight, b.workspace)
        ok()
        check_forward(x, gain, b)
        check_backward(dy, None, x, gain, b)


def test_norm_quant_in_place_and_each_output_alone():
    M, K = 333, 1048
    for xt, st in ((BF, BF), (BF, F32), (F32, F32)):
        x, r, w = norm_inputs(M, K, xt, st, F32)
        b = bl.NormQuantBuffers.allocate(M, K, xt, st, F32)
        bl.bl_norm_quant_forward(x, r, w, EPS, b.sum, b.rstd, b.xq, b.sx)
        dy, dsum = rnd(M, K, seed=5, dtype=xt), rnd(M, K, seed=6, dtype=st)
        dx, dw = torch.empty(M, K, dtype=xt, device="cuda"), torch.empty(K, device="cuda")
        bl.bl_norm_quant_backward(dy, dsum, b.sum, w, b.rstd, dx, b.dresidual, b.dweight, b.workspace)
        ok()
        # the stream updated in place, into the residual or into x
        for into in ("r",) + (("x",) if xt == st else ()):
            c = bl.NormQuantBuffers.allocate(M, K, xt, st, F32, backward=False)
            x2, r2 = x.clone(), r.clone()
            bl.bl_norm_quant_forward(x2, r2, w, EPS, r2 if into == "r" else x2, c.rstd, c.xq, c.sx)
            ok()
            assert torch.equal(r2 if into == "r" else x2, b.sum) and torch.equal(c.xq, b.xq)
            assert torch.equal(c.sx, b.sx) and torch.equal(c.rstd, b.rstd)
        # each gradient alone, and the gradients in the place of what they come from
        one = torch.empty_like(b.dresidual)
        bl.bl_norm_quant_backward(dy, dsum, b.sum, w, b.rstd, None, one)
        ok()
        assert torch.equal(one, b.dresidual)
        one = torch.empty_like(dx)
        bl.bl_norm_quant_backward(dy, dsum, b.sum, w, b.rstd, one)
        ok()
        assert torch.equal(one, dx)
        bl.bl_norm_quant_backward(dy, dsum, b.sum, w, b.rstd, None, None, dw, b.workspace)
        ok()
        assert torch.equal(dw, b.dweight)
        dy2, ds2 = dy.clone(), dsum.clone()
        bl.bl_norm_quant_backward(dy2, ds2, b.sum, w, b.rstd, dy2, ds2, dw, b.workspace)
        ok()
        assert torch.equal(dy2, dx) and torch.equal(ds2, b.dresidual) and torch.equal(dw, b.dweight)


@pytest.mark.parametrize("pt", [BF, F32])
def test_norm_quant_accumulates_and_takes_no_tokens(pt):
    M, K = 50, 264
    x, r, w = norm_inputs(M, K, BF, F32, pt)
    b = bl.NormQuantBuffers.allocate(M, K, BF, F32, pt)
    bl.bl_norm_quant_forward(x, r, w, EPS, b.sum, b.rstd, b.xq, b.sx)
    dy = rnd(M, K, seed=5, dtype=BF)
    start = rnd(K, seed=9, dtype=pt)
    b.dweight.copy_(start)
    bl.bl_norm_quant_backward(dy, None, b.sum, w, b.rstd, None, None, b.dweight, b.workspace, accumulate=True)
    ok()
    _, _, dw, size = gradients(dy, None, b.sum, w)
    close(b.dweight, dw + start.double(), 200 * U * (size + start.double().abs()), "dweight")
    none = bl.NormQuantBuffers.allocate(0, K, BF, F32, pt)
    bl.bl_norm_quant_forward(x[:0], r[:0], w, EPS, none.sum, none.rstd, none.xq, none.sx)
    kept = b.dweight.clone()
    bl.bl_norm_quant_backward(dy[:0], None, none.sum, w, none.rstd, None, None, b.dweight, none.workspace, accumulate=True)
    ok()
    assert torch.equal(b.dweight, kept)
    bl.bl_norm_quant_backward(dy[:0], None, none.sum, w, none.rstd, None, none.dresidual, b.dweight, none.workspace)
    ok()
    assert not bool(b.dweight.any())


@pytest.mark.parametrize("K", [64, 1000, 2560])
@pytest.mark.parametrize("st", [BF, F32])
def test_norm_quant_rows_of_any_range(K, st):
    """Zero rows, rows below the floor, rows that leave fp32 and rows with an
    infinity or a NaN leave the others alone."""
    M = 12
    x, r, w = norm_inputs(M, K, BF, st, F32)
    x[0], r[0] = 0, 0
    x[1], r[1] = 1e-30, 1e-30                   # normed to values below the least absmax
    x[2], r[2] = 0, 1e20                        # its squares leave fp32
    x[3, K // 2] = float("inf")
    r[4, 1] = float("nan")
    x[5], r[5] = 0, 3e18                        # 64 of its squares and more do too: 64 * 9e36 = 5.8e38 > 3.4e38
    x[6, 0] = float("-inf")
    x[7], r[7] = 0, 1e17                        # 2560 of its squares do not: 2560 * 1e34 = 2.6e37
    b = bl.NormQuantBuffers.allocate(M, K, BF, st, F32)
    bl.bl_norm_quant_forward(x, r, w, EPS, b.sum, b.rstd, b.xq, b.sx)
    ok()
    bad = torch.tensor([2, 3, 4, 5, 6], device="cuda")
    fine = torch.tensor([0, 1, 7, 8, 9, 10, 11], device="cuda")
    assert bool(b.sx[bad].isnan().all()) and bool(b.rstd[bad].isnan().all())
    assert not bool(b.xq[:2].any())
    assert torch.equal(b.sx[:2], torch.full((2,), 1e-5, device="cuda") / 127)

    class Part:
        rstd, xq, sx = b.rstd[fine], b.xq[fine], b.sx[fine]
    check_forward(b.sum[fine], w, Part)
    zero = torch.zeros(K, device="cuda")
    bl.bl_norm_quant_forward(x, r, zero, EPS, b.sum, b.rstd, b.xq, b.sx)   # a gain of zeros
    ok()
    assert not bool(b.xq[fine].any()) and bool((b.sx[fine] == b.sx[0]).all())


def test_norm_quant_codes_feed_the_ternary_forward():
    """The codes as bl_forward's operand: the layer's product of the normed stream."""
    M, K, N = 130, 320, 256
    x, r, w = norm_inputs(M, K, BF, F32, F32)
    W = rnd(N, K, seed=4, scale=0.05)
    b = bl.NormQuantBuffers.allocate(M, K, BF, F32, F32, backward=False)
    s = bl.StepBuffers.allocate(M, N, K)
    bl.bl_norm_quant_forward(x, r, w, EPS, b.sum, b.rstd, b.xq, b.sx)
    bl.bl_quantize_weight(W, s.w_packed, s.gamma, s.workspace)
    bl.bl_forward(b.xq, b.sx, s.w_packed, s.gamma, s.y)
    ok()
    gamma = W.double().abs().mean()
    codes = torch.round(W.double() / gamma).clamp(-1, 1)
    want = (b.xq.double() * b.sx.double()[:, None]) @ codes.t() * gamma
    size = (b.xq.double().abs() * b.sx.double()[:, None]) @ codes.abs().t() * gamma
    close(s.y, want, 2.0 ** -20 * size, "y")


# ----------------------------------------------------------------- INT8 product
def codes(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-128, 128, shape, generator=g, device="cuda", dtype=torch.int8)


def scales(n, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(n, generator=g, device="cuda") * 0.02 + 1e-4


def product(xq, sx, wq, sw, dtype):
    """The product with its three roundings (integers are exact in fp64 here)."""
    acc = xq.double() @ wq.double().t()
    return (acc.float() * (sx[:, None] * sw[None, :])).to(dtype)


# the few tokens' kernels and the tiles, at and next to their sizes in each dimension
MNK = [(1, 1, 16), (1, 6912, 2560), (2, 17, 48), (7, 100, 64), (8, 256, 80), (9, 33, 144), (16, 5001, 1040), (17, 16, 16),
       (31, 130, 4096), (32, 1000, 528), (33, 8, 16), (33, 1000, 128), (64, 129, 144), (100, 5001, 1040), (128, 128, 256),
       (129, 512, 272), (255, 257, 400), (256, 256, 128), (257, 24, 2560), (300, 6912, 512), (513, 1001, 896), (1000, 3, 32),
       (2048, 1408, 512), (700, 9999, 240), (2100, 8004, 64)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", MNK)
def test_int8_linear(M, N, K, dtype):
    xq, wq, sx, sw = codes(M, K, seed=M), codes(N, K, seed=N), scales(M, 1), scales(N, 2)
    y = torch.empty(M, N, dtype=dtype, device="cuda")
    bl.bl_int8_linear_forward(xq, sx, wq, sw, y)
    ok()
    assert torch.equal(y, product(xq, sx, wq, sw, dtype))


# tens of tokens, K split over 2 to 8 CTAs: more and fewer tiles than clusters fit at
# once, N that ends anywhere in a tile and in a group of four channels
SPLIT = [(64, 6912, 2560), (33, 7001, 2576), (40, 3001, 1504), (64, 5600, 4096), (33, 2040, 4096), (200, 130, 6000),
         (63, 1000, 8208), (17, 1803, 2576), (32, 2560, 6912), (100, 129, 16384), (35, 1030, 256)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", SPLIT)
def test_int8_linear_split_over_a_cluster(M, N, K, dtype):
    xq, wq, sx, sw = codes(M, K, seed=M), codes(N, K, seed=N), scales(M, 1), scales(N, 2)
    hold = torch.full((M * N + 64,), 7.0, dtype=dtype, device="cuda")
    y = hold[32 : 32 + M * N].view(M, N)
    bl.bl_int8_linear_forward(xq, sx, wq, sw, y)
    ok()
    assert torch.equal(y, product(xq, sx, wq, sw, dtype))
    assert bool((hold[:32] == 7).all()) and bool((hold[32 + M * N :] == 7).all())


@pytest.mark.parametrize("M", [1, 20, 300])
def test_int8_linear_largest_sums(M):
    """K at its limit with the largest codes: 65536 * 128^2 = 2^30, and sums that
    fp32 has to round."""
    K, N = 65536, 40
    for value in (-128, 127):
        xq, wq = (torch.full((n, K), value, dtype=torch.int8, device="cuda") for n in (M, N))
        wq[1::2, ::7] = 1
        wq[2::3] = -wq[2::3].clamp(min=-127)
        y = torch.empty(M, N, device="cuda")
        sx, sw = scales(M), scales(N, 1)
        bl.bl_int8_linear_forward(xq, sx, wq, sw, y)
        ok()
        assert torch.equal(y, product(xq, sx, wq, sw, F32))


@pytest.mark.parametrize("M,N,K", [(1, 40, 32), (20, 1000, 64), (40, 1001, 64), (300, 600, 64), (300, 601, 64)])
def test_int8_linear_leaves_the_neighbours_alone(M, N, K):
    """Nothing is written before or behind y, nor read behind the operands."""
    for dtype in (BF, F32):
        hold = torch.full((M * N + 512,), 7.0, dtype=dtype, device="cuda")
        y = hold[256:256 + M * N].view(M, N)
        big_x, big_w = codes(M * K + 512), codes(N * K + 512)
        sx, sw = (torch.full((n + 64,), float("nan"), device="cuda") for n in (M, N))
        sx[:M], sw[:N] = scales(M), scales(N)
        xq, wq = big_x[:M * K].view(M, K), big_w[:N * K].view(N, K)
        bl.bl_int8_linear_forward(xq, sx[:M], wq, sw[:N], y)
        ok()
        assert torch.equal(y, product(xq, sx[:M], wq, sw[:N], dtype))
        assert bool((hold[:256] == 7).all()) and bool((hold[256 + M * N:] == 7).all())


def test_int8_linear_scales_that_are_not_finite_stay_with_their_token_and_channel():
    for M in (5, 100):
        xq, wq, sx, sw = codes(M, 64), codes(300, 64, seed=1), scales(M), scales(300)
        sx[3], sw[7] = float("nan"), float("nan")
        y = torch.empty(M, 300, dtype=BF, device="cuda")
        bl.bl_int8_linear_forward(xq, sx, wq, sw, y)
        ok()
        want = product(xq, sx, wq, sw, BF)
        assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.nan_to_num(), want.nan_to_num())
        assert int(y.isnan().sum()) == M + 300 - 1


GRADS = [(1, 8, 16), (3, 64, 48), (16, 256, 512), (33, 1000, 128), (100, 136, 272), (257, 5000, 144), (700, 1408, 512),
         (64, 32000, 80), (1030, 264, 400), (2048, 512, 1408),
         # dW's tokens in slices; more than 1024 tokens into an fp32 dW whose sums would be too many
         (4200, 136, 272), (2100, 72, 2096), (4099, 520, 1552), (2500, 4992, 528),
         # a few tokens: the codes' own kernel, one or more slices, ends inside its tiles
         (2, 8, 2576), (7, 24, 16), (17, 40, 32), (32, 1000, 144), (31, 2056, 1040), (5, 11976, 272), (20, 6912, 2560),
         (33, 24, 48), (64, 1000, 2560), (50, 2056, 80), (64, 2568, 1040)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", GRADS)
def test_int8_linear_gradients(M, N, K, dtype):
    xq, wq, sx, sw = codes(M, K, seed=M), codes(N, K, seed=N), scales(M, 1), scales(N, 2)
    dY = rnd(M, N, seed=3, dtype=BF)
    b = bl.Int8LinearBuffers.allocate(M, N, K, BF, dtype)
    b.workspace.fill_(255)
    bl.bl_int8_linear_backward(dY, xq, sx, wq, sw, b.dX, b.dW, workspace=b.workspace)
    ok()
    x, w, d = (xq.float() * sx[:, None]).to(BF).double(), (wq.float() * sw[:, None]).to(BF).double(), dY.double()
    # the tensor cores' sums may drop a step of fp32 per 16 terms; partial sums' joins
    tol = (N / 16 + 64) * 2 * U
    close(b.dX, d @ w, tol * (d.abs() @ w.abs()), "dX")
    tol = (M / 16 + 64) * 2 * U
    close(b.dW, d.t() @ x, tol * (d.abs().t() @ x.abs()), "dW")
    # each alone, and dW added to what it holds
    alone = bl.Int8LinearBuffers.allocate(M, N, K, BF, dtype)
    bl.bl_int8_linear_backward(dY, xq, sx, wq, sw, alone.dX, None, workspace=alone.workspace)
    bl.bl_int8_linear_backward(dY, xq, sx, wq, sw, None, alone.dW, workspace=alone.workspace)
    ok()
    assert torch.equal(alone.dX, b.dX) and torch.equal(alone.dW, b.dW)
    start = rnd(N, K, seed=4, dtype=dtype)
    alone.dW.copy_(start)
    bl.bl_int8_linear_backward(dY, xq, sx, wq, sw, None, alone.dW, accumulate_dW=True, workspace=alone.workspace)
    ok()
    close(alone.dW, d.t() @ x + start.double(), tol * (d.abs().t() @ x.abs() + start.double().abs()), "dW added")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", [(5, 264, 48), (20, 1032, 80), (70, 136, 48), (2100, 72, 272)])
def test_int8_linear_gradients_leave_the_neighbours_alone(M, N, K, dtype):
    xq, wq, sx, sw = codes(M, K, seed=M), codes(N, K, seed=N), scales(M, 1), scales(N, 2)
    dY = rnd(M, N, seed=3, dtype=BF)
    n = bl.bl_int8_linear_backward_workspace_size(M, N, K)
    hx = torch.full((M * K + 64,), 7.0, dtype=BF, device="cuda")
    hw = torch.full((N * K + 64,), 7.0, dtype=dtype, device="cuda")
    ws = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    dX, dW = hx[32 : 32 + M * K].view(M, K), hw[32 : 32 + N * K].view(N, K)
    bl.bl_int8_linear_backward(dY, xq, sx, wq, sw, dX, dW, workspace=ws[256 : 256 + n])
    ok()
    x, w, d = (xq.float() * sx[:, None]).to(BF).double(), (wq.float() * sw[:, None]).to(BF).double(), dY.double()
    close(dX, d @ w, (N / 16 + 64) * 2 * U * (d.abs() @ w.abs()), "dX")
    close(dW, d.t() @ x, (M / 16 + 64) * 2 * U * (d.abs().t() @ x.abs()), "dW")
    for hold, size in ((hx, M * K), (hw, N * K)):
        assert bool((hold[:32] == 7).all()) and bool((hold[32 + size :] == 7).all())
    assert bool((ws[:256] == 0xA5).all()) and bool((ws[256 + n :] == 0xA5).all())


def test_int8_linear_gradient_against_differences():
    """The gradients are those of the product of the operands' values."""
    M, N, K = 40, 64, 32
    xq, wq, sx, sw = codes(M, K), codes(N, K, seed=1), scales(M), scales(N)
    dY = rnd(M, N, dtype=BF)
    b = bl.Int8LinearBuffers.allocate(M, N, K, F32, F32)
    bl.bl_int8_linear_backward(dY, xq, sx, wq, sw, b.dX, b.dW, workspace=b.workspace)
    ok()
    x, w = (xq.float() * sx[:, None]).to(BF).double(), (wq.float() * sw[:, None]).to(BF).double()
    gen = torch.Generator(device="cuda").manual_seed(2)
    for _ in range(4):
        vx, vw = (torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64) for t in (x, w))
        h = 1e-4
        def f(s):
            return ((x + s * h * vx) @ (w + s * h * vw).t() * dY.double()).sum()
        slope = float((f(1) - f(-1)) / (2 * h))          # exact for a product of two: its third difference is zero
        got = float((b.dX.double() * vx).sum() + (b.dW.double() * vw).sum())
        # dX is rounded to bf16, dW to fp32 after sums of 40 terms
        bound = 2.0 ** -8 * float((b.dX.double() * vx).abs().sum()) + 2.0 ** -18 * float((b.dW.double() * vw).abs().sum())
        assert abs(got - slope) <= bound + 1e-8


def test_int8_linear_takes_no_tokens():
    y = torch.empty(0, 24, device="cuda")
    xq, wq, sx, sw = codes(0, 32), codes(24, 32), scales(0), scales(24)
    bl.bl_int8_linear_forward(xq, sx, wq, sw, y)
    dW = torch.full((24, 32), 3.0, device="cuda")
    dY = torch.empty(0, 24, dtype=BF, device="cuda")
    bl.bl_int8_linear_backward(dY, xq, sx, wq, sw, None, dW, accumulate_dW=True)
    ok()
    assert bool((dW == 3).all())
    bl.bl_int8_linear_backward(dY, xq, sx, wq, sw, torch.empty(0, 32, dtype=BF, device="cuda"), dW)
    ok()
    assert not bool(dW.any())


# ----------------------------------------------------------------- the gradients' norm and clipping
def tensors(sizes, types=(F32, BF), seed=0, scale=1e-2):
    return [rnd(n, seed=seed + i, dtype=types[i % len(types)], scale=scale * (1 + i % 5)) for i, n in enumerate(sizes)]


def workspace(count):
    return torch.full((max(bl.bl_grad_norm_workspace_size(count), 16),), 255, dtype=torch.uint8, device="cuda")


def norm64(grads):
    return math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))


def check_clip(grads, most, out=None, norm=None):
    """One call against 64 bits; returns what it wrote."""
    norm = torch.full((1,), -1.0, device="cuda") if norm is None else norm
    before = [g.clone() for g in grads]
    bl.bl_clip_grads(grads, most, norm, workspace(len(grads)), out=out)
    ok()
    want = norm64(before)
    # up to 32 squares in fp32 (their own roundings, 8 steps), the root halves it, one rounding at the end
    assert abs(float(norm) - want) <= 7 * U * want
    factor = most / want if want > most else 1.0
    got = grads if out is None else out
    for g, o in zip(before, got):
        if factor == 1.0:
            assert torch.equal(o, g)
        else:
            # the norm's roundings, the factor's and the product's
            close(o, g.double() * factor, 9 * U * (g.double() * factor).abs(), "clipped")
    if out is not None:
        assert all(torch.equal(a, b) for a, b in zip(before, grads))
    return got


LISTS = [[1], [7], [8, 0, 3], [4096], [1023, 1, 5, 4097, 0, 2], [100000, 333, 2048], [5] * 64, [17] * 65, [1000] * 300, [3] * 1025,
         [2560 * 6912, 2560, 6912 * 100], [0, 0], []]


@pytest.mark.parametrize("sizes", LISTS)
def test_clip(sizes):
    for types in ((F32,), (BF,), (F32, BF)):
        grads = tensors(sizes, types)
        total = norm64(grads)
        norm = torch.full((1,), -1.0, device="cuda")
        bl.bl_grad_norm(grads, norm, workspace(len(grads)))
        ok()
        assert abs(float(norm) - total) <= 7 * U * total
        out = [torch.full_like(g, 9.0) for g in grads]
        a = check_clip(grads, total / 3, out)
        b = check_clip([g.clone() for g in grads], total / 3)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        check_clip(grads, total * 3, out)
        check_clip([g.clone() for g in grads], total * 3)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_clip_of_views_that_start_anywhere(dtype, shift):
    """Tensors packed one behind the other, clipped in place and into others that
    start at another place of a line; what lies between stays."""
    sizes, gap = [1, 5, 4095, 10007, 2, 20000, 31], 3
    flat = rnd(sum(sizes) + gap * len(sizes) + 64, dtype=dtype)
    def views(t, first):
        at, out = first, []
        for n in sizes:
            out.append(t[at:at + n])
            at += n + gap
        return out
    grads = views(flat, 1)
    to = torch.full_like(flat, 5.0)
    check_clip(grads, 0.5, views(to, 1 + shift))
    mask = torch.ones_like(to, dtype=torch.bool)
    for v in views(mask, 1 + shift):
        v.fill_(False)
    assert bool((to[mask] == 5).all())
    keep = flat.clone()
    check_clip(grads, 0.5)
    mask = torch.ones_like(flat, dtype=torch.bool)
    for v in views(mask, 1):
        v.fill_(False)
    assert torch.equal(flat[mask], keep[mask])


@pytest.mark.parametrize("scale", [1e30, 1e19, 3e-19, 1e-20, 1e-30])
def test_clip_over_the_range_of_fp32(scale):
    """Values whose squares overflow or vanish in fp32, next to zeros."""
    for dtype in (F32, BF):
        grads = [rnd(5000, dtype=dtype, scale=scale), torch.zeros(9000, dtype=dtype, device="cuda"), rnd(3, seed=1, dtype=dtype, scale=scale)]
        total = norm64(grads)
        check_clip([g.clone() for g in grads], total / 7)
        check_clip([g.clone() for g in grads], total / 1e6, [torch.empty_like(g) for g in grads])


def test_clip_a_norm_beyond_fp32():
    grads = [torch.full((100000,), 3e38, device="cuda")]
    norm = torch.zeros(1, device="cuda")
    bl.bl_clip_grads(grads, 1.0, norm, workspace(1))
    ok()
    assert float(norm) == math.inf
    assert bool(((grads[0].double() - 1 / math.sqrt(100000)).abs() <= 9 * U).all())


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_clip_leaves_gradients_that_are_not_finite(bad):
    grads = tensors([1000, 333])
    grads[1][5] = bad
    keep, norm = [g.clone() for g in grads], torch.zeros(1, device="cuda")
    out = [torch.empty_like(g) for g in grads]
    for to in (None, out):
        bl.bl_clip_grads(grads, 0.1, norm, workspace(2), out=to)
        ok()
        assert not bool(norm.isfinite().any()) and bool(norm.isnan().all()) == math.isnan(bad)
        for a, b in zip(keep, grads if to is None else out):
            assert torch.equal(a.nan_to_num(3), b.nan_to_num(3)) and torch.equal(a.isnan(), b.isnan())


def test_clip_to_zero_and_to_infinity():
    grads = tensors([1000, 333])
    keep = [g.clone() for g in grads]
    norm = torch.zeros(1, device="cuda")
    bl.bl_clip_grads(grads, math.inf, norm, workspace(2))
    ok()
    assert all(torch.equal(a, b) for a, b in zip(keep, grads))
    bl.bl_clip_grads(grads, 0.0, norm, workspace(2))
    ok()
    assert not any(bool(g.any()) for g in grads)
    bl.bl_clip_grads(grads, 0.0, norm, workspace(2))   # a norm of zero is not above zero
    ok()
    assert float(norm) == 0 and not any(bool(g.any()) for g in grads)


def test_norm_of_a_tensor_listed_twice_counts_it_twice():
    g = rnd(1000)
    norm = torch.zeros(1, device="cuda")
    bl.bl_grad_norm([g, g], norm, workspace(2))
    ok()
    assert abs(float(norm) - norm64([g, g])) <= 7 * U * float(norm)
