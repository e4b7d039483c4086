"""GPU: 8-bit activations, the SwiGLU gate and the norms against 64-bit forms.

Tolerances count roundings. u = 2^-24 is half a step of fp32 relative to the
value, ``half(dtype)`` that of the output's type. An fp32 value made by n
rounded operations on terms of magnitude A is off by at most about n u A.
"""

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
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def close(got, want, tol, what):
    """|got - want| <= tol + the rounding to got's type, elementwise."""
    want = want.double()
    bound = tol + half(got.dtype) * (want.abs() + tol) + TINY
    bad = ~((got.double() - want).abs() <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float((got.double() - want).abs().max()), float(bound.max()))


def saved_values(x):
    """codes, scales and values of the 8-bit form, in 64 bits with its fp32
    roundings (a product of two fp32 numbers is exact in 64 bits, and a
    quotient rounded through 64 bits is rounded as if once: 53 >= 2 24 + 2)."""
    M, K = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -K % 128)).reshape(M, -1, 128)
    a = v.abs().amax(-1, keepdim=True).clamp(min=float(torch.tensor(1e-30)))
    inv = ((1.0 / a).float().double() * 127.0).float().double()
    scale = (a * (torch.ones(1, dtype=torch.float64) / 127.0).float().double().cuda()).float()
    codes = torch.round((v * inv).float().double())
    values = (codes * scale.double()).float()
    return codes.reshape(M, -1)[:, :K].to(torch.int8), scale[:, :, 0], values.reshape(M, -1)[:, :K]


def ok():
    torch.cuda.synchronize()
    assert bl.bl_get_last_error() == 0


# sizes around the vector layout (8), the group (128), the units per thread and odd rows
SIZES = [(1, 1), (1, 8), (2, 7), (3, 127), (2, 128), (5, 129), (3, 136), (17, 264), (33, 1001), (64, 1408), (9, 2565),
         (130, 6912), (4099, 24)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K", SIZES)
def test_act8_matches_its_definition(M, K, dtype):
    x = rnd(M, K, seed=M + K, dtype=dtype) * (10.0 ** torch.arange(-3, 3, device="cuda", dtype=F32).repeat(K)[:K]).to(dtype)
    x[0, 0] = 0
    s = bl.Act8.allocate(M, K)
    out = torch.empty_like(x)
    bl.bl_act8_encode(x, s)
    bl.bl_act8_decode(s, out)
    ok()
    codes, scales, values = saved_values(x)
    assert torch.equal(s.codes, codes) and torch.equal(s.scales, scales)
    assert torch.equal(out, values.to(dtype))
    assert s.codes.abs().max() <= 127
    # half a step of the group's largest value
    step = scales.repeat_interleave(128, 1)[:, :K]
    assert bool(((values.double() - x.double()).abs() <= (0.5 + 2.0 ** -14) * step.double()).all())


@pytest.mark.parametrize("K", [256, 261])
def test_act8_zero_tiny_and_non_finite_groups(K):
    x = torch.zeros(6, K, device="cuda")
    x[1, :128] = 1e-35            # below the floor: codes 0
    x[2, 3] = float("inf")
    x[3, 200] = float("nan")
    x[4, 5] = float("-inf")
    x[5] = 3.0
    s = bl.Act8.allocate(6, K)
    out = torch.empty_like(x)
    bl.bl_act8_encode(x, s)
    bl.bl_act8_decode(s, out)
    ok()
    assert bool((out[:2] == 0).all()) and torch.equal(out.nan_to_num(9), saved_values(x.nan_to_num(0, 0, 0))[2].where(out.isfinite(), out).nan_to_num(9))
    assert bool(((out[5] - 3.0).abs() <= 4 * U * 3.0).all())
    assert bool(out[2, :128].isnan().all()) and bool((out[2, 128:] == 0).all())
    assert bool(out[3, 128:256].isnan().all()) and bool((out[3, :128] == 0).all())
    assert bool(out[4, :128].isnan().all()) and bool((out[4, 128:] == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K", SIZES)
def test_swiglu_forward_and_backward(M, K, dtype):
    gate, up, dy = (rnd(M, K, seed=i + K, dtype=dtype, scale=3.0) for i in range(3))
    gate[0, 0] = 90.0
    gate[-1, -1] = -100.0
    b = bl.SwigluBuffers.allocate(M, K, dtype)
    bl.bl_swiglu_forward(gate, up, b.y, b.gate8, b.up8)
    plain = torch.empty_like(b.y)
    bl.bl_swiglu_forward(gate, up, plain)
    bl.bl_swiglu_backward(dy, b.gate8, b.up8, b.dgate, b.dup)
    ok()
    assert torch.equal(plain, b.y)
    for t, x in ((b.gate8, gate), (b.up8, up)):
        codes, scales, _ = saved_values(x)
        assert torch.equal(t.codes, codes) and torch.equal(t.scales, scales)
    # 1 / (1 + exp(-g)): exp to 2 units and g log2(e) rounded (a relative error
    # of |g| log2(e) u in exp), the sum, the quotient and the products
    def units(g):
        return (16 + 4 * g.abs()) * 2 * U
    g, u = gate.double(), up.double()
    y = g * torch.sigmoid(g) * u
    close(b.y, y, units(g) * y.abs(), "y")
    g, u, d = saved_values(gate)[2].double(), saved_values(up)[2].double(), dy.double()
    s = torch.sigmoid(g)
    dup = d * g * s
    close(b.dup, dup, units(g) * dup.abs(), "dup")
    # 1 - s and 1 + g (1 - s) cancel: counted on the terms
    close(b.dgate, d * u * s * (1 + g * (1 - s)), units(g) * (d * u * s).abs() * (1 + g.abs()), "dgate")


def test_swiglu_backward_in_place_and_by_differences():
    M, K = 7, 264
    gate, up, dy = (rnd(M, K, seed=i) for i in range(3))
    b = bl.SwigluBuffers.allocate(M, K, F32)
    bl.bl_swiglu_forward(gate, up, b.y, b.gate8, b.up8)
    bl.bl_swiglu_backward(dy, b.gate8, b.up8, b.dgate, b.dup)
    d2, other = dy.clone(), torch.empty_like(dy)
    bl.bl_swiglu_backward(d2, b.gate8, b.up8, d2, other)
    d3 = dy.clone()
    bl.bl_swiglu_backward(d3, b.gate8, b.up8, other, d3)
    ok()
    assert torch.equal(d2, b.dgate) and torch.equal(d3, b.dup)
    # central differences of sum(dy * silu(g) u) at the saved values: the step
    # 1e-4 leaves an error of 1e-8 |f'''| / 6, and |f'''| < 1 for silu
    g, u = saved_values(gate)[2].double(), saved_values(up)[2].double()
    f = lambda g, u: dy.double() * g * torch.sigmoid(g) * u   # noqa: E731
    e = 1e-4
    scale = (dy * up).abs().double() + dy.abs().double() * (1 + g.abs())
    assert bool((((f(g + e, u) - f(g - e, u)) / (2 * e) - b.dgate.double()).abs() <= 1e-5 * scale + 1e-6).all())
    assert bool((((f(g, u + e) - f(g, u - e)) / (2 * e) - b.dup.double()).abs() <= 1e-5 * scale + 1e-6).all())


# ----------------------------------------------------------------- norms
NORM_SIZES = [(1, 1), (3, 2), (2, 8), (5, 31), (4, 32), (3, 33), (37, 64), (5, 100), (6, 128), (300, 136), (18, 264),
              (64, 512), (333, 1001), (9, 1024), (7, 1032), (34, 2560), (149, 2565), (17, 6912), (5, 8192), (4, 8200),
              (3, 10001), (2, 32768), (3, 32776), (2, 40001)]


def norm_case(M, K, dtype, pdtype, rms, bias, seed=0):
    x = rnd(M, K, seed=seed, dtype=F32) * (1 + 15 * (torch.arange(K, device="cuda") % 97 == 0)) + 0.5
    return (x.to(dtype), rnd(K, seed=seed + 1).mul(0.2).add(1).to(pdtype),
            rnd(K, seed=seed + 2, dtype=pdtype, scale=0.2) if bias else None, rnd(M, K, seed=seed + 3, dtype=dtype))


def run_norm(x, w, bias, dy, rms, saved8, eps=1e-6, **kw):
    M, K = x.shape
    b = bl.NormBuffers.allocate(M, K, x.dtype, w.dtype, rms=rms, bias=True, saved8=saved8)
    bl.bl_norm_forward(x, w, bias, eps, b.y, b.mean, b.rstd, rms=rms, saved8=b.saved8)
    bl.bl_norm_backward(dy, b.saved8 if saved8 else x, w, b.mean, b.rstd, b.dx, b.dweight, b.dbias, b.workspace,
                        rms=rms, **kw)
    ok()
    return b


def check_norm(b, x, w, bias, dy, rms, saved8, eps=1e-6):
    M, K = x.shape
    X, W, D = x.double(), w.double(), dy.double()
    mu = torch.zeros(M, 1, device="cuda", dtype=torch.float64) if rms else X.mean(1, keepdim=True)
    r = 1 / torch.sqrt(((X - mu) ** 2).mean(1, keepdim=True) + eps)
    # additions that one value goes through in a row's sum: at most 32 in a
    # thread (K / 1024 in the wide kernels), 5 in the warp, 32 over the warps
    n = 72 + K / 1024
    A = X.abs().mean(1, keepdim=True)
    if not rms:
        close(b.mean, mu[:, 0], n * U * A[:, 0], "mean")
    # (x - mean)^2 carries twice the error of x - mean: the sum's and one
    # rounding; rstd has half the relative error of the variance
    dm = (0 if rms else 1) * n * U * A
    rel = n * U + 2 * dm * r + (dm * r) ** 2
    close(b.rstd, r[:, 0], (rel * r)[:, 0], "rstd")
    xh = (X - mu) * r
    B = 0.0 if bias is None else bias.double()
    close(b.y, xh * W + B, (xh.abs() * (rel + 4 * U) + dm * r) * W.abs() + U * (torch.as_tensor(B).abs() if bias is not None else 0.0), "y")
    # backward, at the mean and rstd that it is given
    mu = mu if rms else b.mean.double()[:, None]
    r = b.rstd.double()[:, None]
    S = saved_values(x)[2].double() if saved8 else X
    xh, g = (S - mu) * r, D * W
    c1 = torch.zeros_like(r) if rms else g.mean(1, keepdim=True)
    c2 = (g * xh).mean(1, keepdim=True)
    terms = g.abs() + (0 if rms else 1) * g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True)
    close(b.dx, r * (g - c1 - xh * c2), (n + 8) * U * r * terms, "dx")
    # rows that one sum goes through: M / 148 blocks and what joins them (32
    # groups, 148 partial rows), and the three roundings of a term
    m = M / 100 + 200
    close(b.dweight, (D * xh).sum(0), (m + 4) * U * (D * xh).abs().sum(0), "dweight")
    if b.dbias is not None:
        close(b.dbias, D.sum(0), m * U * D.abs().sum(0), "dbias")


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("M,K", NORM_SIZES)
def test_norm_sizes(M, K, rms):
    for i, (dtype, pdtype, saved8, bias) in enumerate([(BF, BF, False, True), (F32, F32, False, False),
                                                       (BF, F32, True, False), (F32, BF, True, True)]):
        x, w, bias, dy = norm_case(M, K, dtype, pdtype, rms, bias, seed=10 * i + K)
        b = run_norm(x, w, bias, dy, rms, saved8)
        if saved8:
            codes, scales, _ = saved_values(x)
            assert torch.equal(b.saved8.codes, codes) and torch.equal(b.saved8.scales, scales)
        check_norm(b, x, w, bias, dy, rms, saved8)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K", [(4096, 2560), (2000, 1416), (5000, 72)])
def test_norm_many_rows(M, K, dtype):
    x, w, bias, dy = norm_case(M, K, dtype, F32, False, True)
    check_norm(run_norm(x, w, bias, dy, False, True), x, w, bias, dy, False, True)
    assert bl.bl_get_last_error() == 0


def test_norm_constant_zero_and_offset_rows():
    K = 512
    x = torch.zeros(4, K, device="cuda")
    x[1] = 5.0                       # variance 0: y = bias exactly
    x[2] = 1e4 + rnd(K, seed=1)      # mean far above the spread
    x[3] = rnd(K, seed=2, scale=1e-8)
    w, bias, dy = torch.ones(K, device="cuda"), rnd(K, seed=3), rnd(4, K, seed=4)
    b = run_norm(x, w, bias, dy, False, False)
    assert torch.equal(b.y[:2], bias.expand(2, K))
    check_norm(b, x, w, bias, dy, False, False)


def test_norm_without_parameters_and_skipped_outputs():
    M, K = 19, 264
    x, w, _, dy = norm_case(M, K, F32, F32, False, False)
    full = run_norm(x, torch.ones(K, device="cuda"), None, dy, False, False)
    y, mean, rstd = torch.empty_like(x), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    bl.bl_norm_forward(x, None, None, 1e-6, y, mean, rstd)
    dx, dw, db = torch.empty_like(x), torch.full((K,), 9.0, device="cuda"), torch.full((K,), 9.0, device="cuda")
    ws = full.workspace
    bl.bl_norm_backward(dy, x, None, mean, rstd, dx, None, None, ws)
    assert torch.equal(y, full.y) and torch.equal(dx, full.dx)
    bl.bl_norm_backward(dy, x, None, mean, rstd, None, dw, None, ws)
    assert torch.equal(dw, full.dweight) and bool((db == 9).all())
    bl.bl_norm_backward(dy, x, None, mean, rstd, None, None, db, ws)
    assert torch.equal(db, full.dbias)
    d2 = dy.clone()
    bl.bl_norm_backward(d2, x, None, mean, rstd, d2, None, None, ws)
    ok()
    assert torch.equal(d2, full.dx)


@pytest.mark.parametrize("K", [96, 8200])
@pytest.mark.parametrize("pdtype", [BF, F32])
def test_norm_accumulates_and_empty_batches(pdtype, K):
    M = 21
    x, w, bias, dy = norm_case(M, K, BF, pdtype, False, True)
    b = run_norm(x, w, bias, dy, False, False)
    f = bl.NormBuffers.allocate(M, K, BF, F32, bias=True)
    bl.bl_norm_backward(dy, x, w.float(), b.mean, b.rstd, None, f.dweight, f.dbias, f.workspace)
    dw, db = b.dweight.clone(), b.dbias.clone()
    bl.bl_norm_backward(dy, x, w, b.mean, b.rstd, None, dw, db, b.workspace, accumulate=True)
    ok()
    assert torch.equal(dw, (f.dweight + b.dweight.float()).to(pdtype))
    assert torch.equal(db, (f.dbias + b.dbias.float()).to(pdtype))
    e = bl.NormBuffers.allocate(0, K, BF, pdtype, bias=True)
    keep = dw.clone()
    bl.bl_norm_backward(dy[:0], x[:0], w, b.mean[:0], b.rstd[:0], None, dw, db, e.workspace, accumulate=True)
    assert torch.equal(dw, keep)
    bl.bl_norm_backward(dy[:0], x[:0], w, b.mean[:0], b.rstd[:0], None, dw, db, e.workspace)
    ok()
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_norm_one_bad_row_stays_alone():
    M, K = 40, 512
    x, w, bias, dy = norm_case(M, K, BF, F32, False, True)
    good = run_norm(x, w, bias, dy, False, True)
    x2 = x.clone()
    x2[7, 3], x2[20, 100] = float("inf"), float("nan")
    b = run_norm(x2, w, bias, dy, False, True)
    rest = [i for i in range(M) if i not in (7, 20)]
    assert torch.equal(b.y[rest], good.y[rest]) and torch.equal(b.dx[rest], good.dx[rest])
    assert bool(b.y[20].isnan().all()) and bool(b.dx[20].isnan().any()) and bool(b.dx[7].isnan().any())


def test_norm_gradients_by_differences():
    M, K = 5, 72
    x, w, bias, dy = norm_case(M, K, F32, F32, False, True)
    b = run_norm(x, w, bias, dy, False, False)
    g = torch.Generator(device="cuda").manual_seed(5)

    def loss(x, w, bias):
        mu, var = x.mean(1, keepdim=True), x.var(1, keepdim=True, correction=0)
        return (((x - mu) / torch.sqrt(var + 1e-6) * w + bias) * dy.double()).sum()
    X, W, B = x.double(), w.double(), bias.double()
    for name, grad, at in (("x", b.dx, 0), ("w", b.dweight, 1), ("bias", b.dbias, 2)):
        v = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        e = 1e-5
        args = [[X, W, B], [X, W, B]]
        args[0][at], args[1][at] = args[0][at] + e * v, args[1][at] - e * v
        num = (loss(*args[0]) - loss(*args[1])) / (2 * e)
        # truncation of order e^2; the gradient's own error is below 1e-5 of its terms
        assert abs(float(num - (grad.double() * v).sum())) <= 1e-5 * float((grad.double() * v).abs().sum()) + 1e-6, name


def test_rows_leave_neighbours_alone_and_repeat():
    M, K = 13, 2565
    x, w, bias, dy = norm_case(M, K, BF, F32, False, True)
    big = [torch.full((M + 2, K), 7.0, dtype=BF, device="cuda") for _ in range(2)]
    # the buffers start at row 0 of larger ones: what follows them stays
    y, dx = big[0][:M], big[1][:M]
    b = run_norm(x, w, bias, dy, False, True)
    bl.bl_norm_forward(x, w, bias, 1e-6, y, b.mean, b.rstd, saved8=b.saved8)
    bl.bl_norm_backward(dy, b.saved8, w, b.mean, b.rstd, dx, b.dweight, b.dbias, b.workspace)
    ok()
    assert torch.equal(y, b.y) and torch.equal(dx, b.dx)
    assert all(bool((t[M:] == 7).all()) for t in big)
    again = run_norm(x, w, bias, dy, False, True)
    for a, c in ((again.dweight, b.dweight), (again.dbias, b.dbias), (again.dx, b.dx)):
        assert torch.equal(a, c)


@pytest.mark.parametrize("K", [32768, 32765])
def test_offsets_past_32_bits(K):
    """More than 2^31 values: rows near the end against the same rows alone."""
    M, tail = 2 ** 31 // K + 40, 16
    x = torch.zeros(M, K, dtype=BF, device="cuda")
    x[-tail:] = rnd(tail, K, seed=1, dtype=BF)
    dy = torch.zeros(M, K, dtype=BF, device="cuda")
    dy[-tail:] = rnd(tail, K, seed=2, dtype=BF)
    w = rnd(K, seed=3)

    def run(x, dy):
        m = x.shape[0]
        s, out, s2 = bl.Act8.allocate(m, K), torch.empty_like(x), bl.Act8.allocate(m, K)
        bl.bl_act8_encode(x, s)
        bl.bl_act8_decode(s, out)
        got = [s.codes[-tail:].clone(), s.scales[-tail:].clone(), out[-tail:].clone()]
        y, rstd = out, torch.empty(m, device="cuda")
        bl.bl_swiglu_forward(x, dy, y, s, s2)
        got.append(y[-tail:].clone())
        bl.bl_norm_forward(x, w, None, 1e-6, y, None, rstd, rms=True, saved8=s)
        got += [y[-tail:].clone(), rstd[-tail:].clone(), s.codes[-tail:].clone()]
        dw, dx = torch.empty(K, device="cuda"), y
        ws = torch.empty(bl.bl_norm_backward_workspace_size(m, K), dtype=torch.uint8, device="cuda")
        bl.bl_norm_backward(dy, s, w, None, rstd, dx, dw, None, ws, rms=True)
        got += [dx[-tail:].clone()]
        ok()
        return got, dw
    (a, dwa), (b, dwb) = run(x, dy), run(x[-tail:].clone(), dy[-tail:].clone())
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    # the other rows' dy is 0: the same terms, added in another order (two sums
    # of `tail` terms and zeros)
    xh = saved_values(x[-tail:])[2].double() * b[5].double()[:, None]
    assert bool(((dwa - dwb).double().abs() <= 2 * (tail + 4) * U * (dy[-tail:].double() * xh).abs().sum(0)).all())


def test_calls_on_other_streams_and_side_by_side():
    """Every call on a stream given to it, and two chains on two streams at once
    (their own buffers), against the same calls on the current stream."""
    M, K = 260, 520
    args = [norm_case(M, K, BF, F32, False, True, seed=s) for s in (1, 2)]

    def chain(x, w, bias, dy, stream=None):
        n, s = bl.NormBuffers.allocate(M, K, BF, F32, bias=True, saved8=True), bl.SwigluBuffers.allocate(M, K, BF)
        out = torch.empty_like(x)
        bl.bl_norm_forward(x, w, bias, 1e-6, n.y, n.mean, n.rstd, saved8=n.saved8, stream=stream)
        bl.bl_swiglu_forward(n.y, x, s.y, s.gate8, s.up8, stream=stream)
        bl.bl_swiglu_backward(dy, s.gate8, s.up8, s.dgate, s.dup, stream=stream)
        bl.bl_norm_backward(s.dgate, n.saved8, w, n.mean, n.rstd, n.dx, n.dweight, n.dbias, n.workspace, stream=stream)
        bl.bl_act8_encode(n.dx, n.saved8, stream=stream)
        bl.bl_act8_decode(n.saved8, out, stream=stream)
        return [n.y, s.y, s.dgate, s.dup, n.dx, n.dweight, n.dbias, out]
    want = [chain(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[chain(*a, stream=s) for a, s in zip(args, streams)] for _ in range(5)]
    ok()
    for run in got:
        for a, b in zip(run, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_refused_on_the_gpu():
    """The quick binding refuses what the checks in Python refuse, before
    anything is launched."""
    M, K = 4, 64
    x, w, y = rnd(M, K, dtype=BF), rnd(K), rnd(M, K, dtype=BF)
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    s8 = bl.Act8.allocate(M, K)
    for bad in (dict(x=x.half()), dict(x=x.t()), dict(x=x[:2]), dict(x=x.cpu()), dict(weight=w[:-1]), dict(weight=w.half()),
                dict(bias=w.to(BF)), dict(mean=mean.double()), dict(rstd=rstd.cpu()), dict(y=y.float()),
                dict(saved8=bl.Act8.allocate(M, K + 128))):
        a = dict(x=x, weight=w, bias=w, eps=1e-6, y=y, mean=mean, rstd=rstd, saved8=s8) | bad
        with pytest.raises(ValueError):
            bl.bl_norm_forward(**a)
    with pytest.raises(bl.BitLinearError, match="eps"):
        bl.bl_norm_forward(x, w, None, float("nan"), y, mean, rstd)
    with pytest.raises(bl.BitLinearError, match="null"):
        bl.bl_norm_forward(x, w, None, 1e-6, y, None, rstd)
    with pytest.raises(bl.BitLinearError, match="workspace"):
        bl.bl_norm_backward(y, x, w, mean, rstd, y, w, None, torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(bl.BitLinearError, match="workspace"):
        bl.bl_norm_backward(y, x, w, mean, rstd, y, w, None, None)
    odd = torch.empty(M * K + 8, dtype=BF, device="cuda")[1:M * K + 1].view(M, K)
    with pytest.raises(bl.BitLinearError, match="aligned"):
        bl.bl_act8_encode(odd, s8)
    with pytest.raises(bl.BitLinearError, match="same memory"):
        bl.bl_swiglu_backward(x, s8, s8, y, y)
    with pytest.raises(ValueError):
        bl.bl_swiglu_forward(x, y, x.float())
    ok()
