"""GPU: the head cross-entropy and its gradients against 64-bit forms.

Tolerances count roundings. The products of bf16 numbers are exact in fp32;
an fp32 sum on the tensor cores takes 16 products per step and may drop up to
one step of fp32 (2^-23) of the running sum each time, so a logit is off by at
most (K / 16 + 4) 2^-23 sum |h W|. ``loss`` and ``lse`` add the roundings of
exp, log and the final subtraction. dz is rounded to bf16 (2^-8 relative; with
an fp32 dW to two bf16 terms, 2^-16), the gradients' sums again drop a step
per 16 terms, and a bf16 result is rounded once more. These are worst cases
for every element; errors in the norm are smaller and are held to twice the
rounding of the result's type."""

import pytest
import torch

import ternary_weight_quantization_b200 as bl

pytestmark = pytest.mark.gpu
S = 2.0 ** -23
BF, F32 = torch.bfloat16, torch.float32


def case(M, V, K, seed=0, scale=1.0, left_out=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.randn(M, K, generator=g, device="cuda").to(BF)
    W = (torch.randn(V, K, generator=g, device="cuda") * (scale / K ** 0.5)).to(BF)
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    t[torch.rand(M, generator=g, device="cuda") < left_out] = -100
    dl = torch.rand(M, generator=g, device="cuda") * 0.1 - 0.02
    return h, W, t, dl


def run(h, W, t, dl, dw_dtype=BF, dW=None, accumulate=False, stream=None):
    (M, K), V = h.shape, W.shape[0]
    b = bl.XentBuffers.allocate(M, V, K, dw_dtype)
    if dW is not None:
        b.dW = dW
    bl.bl_linear_xent_forward(h, W, t, b.loss, b.lse, b.workspace, stream=stream)
    bl.bl_linear_xent_backward(h, W, t, b.lse, dl, b.dH, b.dW, b.workspace, accumulate_dW=accumulate, stream=stream)
    torch.cuda.synchronize()
    assert bl.bl_get_last_error() == 0
    return b


def check(b, h, W, t, dl, dw_dtype=BF, dW0=None):
    (M, K), V = h.shape, W.shape[0]
    hd, Wd = h.double(), W.double()
    live = (t >= 0) & (t < V)
    z = hd @ Wd.t()
    ez = (K / 16 + 4) * S * (hd.abs() @ Wd.abs().t()).amax(1)         # per token
    lse = torch.logsumexp(z, 1)
    e_lse = ez + 8 * S * (1 + lse.abs())
    assert bool(((b.lse.double() - lse).abs() <= e_lse).all()), "lse"
    zt = z.gather(1, t.clamp(0, V - 1)[:, None])[:, 0]
    loss = torch.where(live, lse - zt, 0.0)
    assert bool(((b.loss.double() - loss).abs() <= ez + e_lse + 2 * S * (lse.abs() + zt.abs())).all()), "loss"
    p = torch.exp(z - lse[:, None])
    dz = p.clone()
    dz[torch.arange(M, device="cuda")[live], t[live]] -= 1
    # p: the errors of z and lse in its exponent, and ex2 itself; all relative
    # to p, also where dz = p - 1
    ep = torch.expm1(ez + e_lse + 8 * S * (1 + lse.abs()))[:, None] * p + 4 * S
    w = torch.where(live, dl.double(), 0.0)[:, None]
    dz, ep = dz * w, ep * w.abs()
    q = 2.0 ** -16 if dw_dtype == F32 else 2.0 ** -8
    for name, got, a, c, n, rz, old in (("dH", b.dH, dz, Wd, V, 2.0 ** -8, None),
                                        ("dW", b.dW, dz.t(), hd, M, q, dW0)):
        if got is None:
            continue
        e = ep if name == "dH" else ep.t()
        want = a @ c
        mag = a.abs() @ c.abs()
        if old is not None:
            want = want + old.double()
        half = torch.finfo(got.dtype).eps / 2
        # fp32 dW: sums of 1024 tokens and their joining, both terms of dz
        steps = min(n, 1024) / 8 + n / 1024 + 8 if got.dtype == F32 else n / 16 + 8 + 64
        tol = rz * mag + e @ c.abs() + steps * S * (mag + (0 if old is None else old.double().abs()))
        bound = tol + half * (want.abs() + tol) + 1e-36
        err = (got.double() - want).abs()
        assert bool((err <= bound).all()), (name, float(err.max()), float(bound.max()))
        norm = float(want.norm())
        if norm and n > 1 and old is None:
            # rounding errors of independent signs: dz's and the result's add in
            # squares. The logits' and ex2's errors are common to a row of dz
            rel = float(err.norm()) / norm
            row = float((e @ c.abs()).norm()) / norm
            assert rel <= 2 * max(half, rz if got.dtype == BF else half) + row + 64 * S, (name, rel)
        assert bool(got.isfinite().all())
    if not bool(live.all()):
        assert bool((b.loss[~live] == 0).all()) and (b.dH is None or bool((b.dH[~live] == 0).all()))


# sizes around the pair tile (256), its halves (128), the box (64), the
# output box (32), the reduction block (64) and K's multiple of 8
SIZES = [(1, 1, 8), (1, 2, 8), (2, 31, 16), (3, 33, 64), (1, 1000, 64), (31, 255, 72), (33, 256, 128), (127, 257, 136),
         (128, 64, 264), (129, 511, 40), (255, 513, 512), (256, 1024, 256), (257, 300, 520), (300, 5003, 200),
         (513, 769, 1000), (64, 8192, 512), (200, 9472, 64), (200, 9473, 64), (257, 4736, 72), (65, 129, 24), (192, 128, 8)]


@pytest.mark.parametrize("dw_dtype", [BF, F32])
@pytest.mark.parametrize("M,V,K", SIZES)
def test_sizes(M, V, K, dw_dtype):
    args = case(M, V, K, seed=M + V + K, left_out=0.2 if M > 3 else 0.0)
    check(run(*args, dw_dtype), *args, dw_dtype)


@pytest.mark.parametrize("M,V,K,dw_dtype", [(8192, 8200, 64, BF), (8192, 20001, 64, BF), (2100, 20001, 72, F32), (4096, 17000, 136, BF),
                                            (1025, 40000, 64, F32)])
def test_pieces_of_the_vocabulary_and_partial_sums(M, V, K, dw_dtype):
    args = case(M, V, K, seed=7, left_out=0.1)
    check(run(*args, dw_dtype), *args, dw_dtype)


def test_layer_widths():
    """The repository's LM (2048 tokens, width 512, vocabulary 8192)."""
    args = case(2048, 8192, 512, seed=3)
    check(run(*args), *args)


@pytest.mark.parametrize("scale", [0.0, 30.0, 200.0])
def test_flat_and_peaked_distributions(scale):
    args = case(130, 700, 128, seed=11, scale=scale)
    b = run(*args)
    if scale == 0.0:
        import math
        assert bool(((b.loss - math.log(700)).abs() <= 8 * S * (1 + math.log(700))).all())
    check(b, *args)


@pytest.mark.parametrize("dw_dtype", [BF, F32])
def test_left_out_tokens_reach_nothing(dw_dtype):
    """Tokens without a target may hold anything: infinities, NaN, huge dloss."""
    M, V, K = 300, 600, 72
    h, W, t, dl = case(M, V, K, seed=5)
    t[::3] = torch.tensor([-100, -1, V, 2 ** 40, -2 ** 62], device="cuda").repeat(20)
    dirty, dl2 = h.clone(), dl.clone()
    dirty[0::9], dirty[3::9], dirty[6::9] = float("nan"), float("inf"), float("-inf")
    dl2[::3] = float("nan")
    clean = torch.where(((t >= 0) & (t < V))[:, None], h, torch.zeros_like(h))
    a, b = run(clean, W, t, dl, dw_dtype), run(dirty, W, t, dl2, dw_dtype)
    assert torch.equal(a.dW, b.dW) and torch.equal(a.dH, b.dH) and torch.equal(a.loss, b.loss)
    check(a, clean, W, t, dl, dw_dtype)


def test_every_token_left_out():
    h, W, t, dl = case(70, 300, 64)
    t.fill_(-100)
    b = run(h, W, t, dl)
    assert not b.loss.any() and not b.dH.any() and not b.dW.any()


def test_non_finite_rows_stay_alone():
    M, V, K = 40, 300, 64
    h, W, t, dl = case(M, V, K, seed=2)
    good = run(h, W, t, dl)
    h2 = h.clone()
    h2[5] = float("nan")
    b = run(h2, W, t, dl)
    rest = [i for i in range(M) if i != 5]
    assert torch.equal(b.loss[rest], good.loss[rest]) and torch.equal(b.dH[rest], good.dH[rest])
    assert bool(b.loss[5].isnan()) and bool(b.dH[5].isnan().all()) and bool(b.dW.isnan().any())


@pytest.mark.parametrize("M", [1, 70, 1100])
@pytest.mark.parametrize("dw_dtype", [BF, F32])
def test_accumulation(M, dw_dtype):
    args = case(M, 520, 72, seed=M)
    dW0 = torch.randn(520, 72, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(dw_dtype)
    b = run(*args, dw_dtype, dW=dW0.clone(), accumulate=True)
    check(b, *args, dw_dtype, dW0=dW0)


def test_one_gradient_alone_and_none():
    h, W, t, dl = case(140, 700, 136, left_out=0.1)
    for dt in (BF, F32):
        b = run(h, W, t, dl, dt)
        for dH, dW in ((True, False), (False, True)):
            x = torch.full_like(b.dH, 9.0) if dH else None
            y = torch.full_like(b.dW, 9.0) if dW else None
            bl.bl_linear_xent_backward(h, W, t, b.lse, dl, x, y, b.workspace)
            assert x is None or torch.equal(x, b.dH)
            assert y is None or torch.equal(y, b.dW)
        bl.bl_linear_xent_backward(h, W, t, b.lse, dl, None, None, b.workspace)
    torch.cuda.synchronize()
    assert bl.bl_get_last_error() == 0


@pytest.mark.parametrize("dw_dtype", [BF, F32])
def test_empty_batch(dw_dtype):
    h, W, t, dl = case(4, 300, 64)
    b = bl.XentBuffers.allocate(0, 300, 64, dw_dtype)
    bl.bl_linear_xent_forward(h[:0], W, t[:0], b.loss, b.lse, b.workspace)
    b.dW.fill_(3.0)
    bl.bl_linear_xent_backward(h[:0], W, t[:0], b.lse, dl[:0], b.dH, b.dW, b.workspace, accumulate_dW=True)
    assert bool((b.dW == 3).all())
    bl.bl_linear_xent_backward(h[:0], W, t[:0], b.lse, dl[:0], b.dH, b.dW, b.workspace)
    torch.cuda.synchronize()
    assert bool((b.dW == 0).all())


@pytest.mark.parametrize("M", [333, 7])
def test_runs_repeat_and_neighbours_stay(M):
    V, K = 1111, 264
    h, W, t, dl = case(M, V, K, seed=9)
    a = run(h, W, t, dl)
    big = {"loss": torch.full((M + 8,), 7.0, device="cuda"), "dH": torch.full((M + 3, K), 7.0, dtype=BF, device="cuda"),
           "dW": torch.full((V + 3, K), 7.0, dtype=BF, device="cuda"),
           "lse": torch.full((M + 8,), 7.0, device="cuda"),
           "ws": torch.full((a.workspace.numel() + 4096,), 0xA5, dtype=torch.uint8, device="cuda")}
    n = a.workspace.numel()
    lse = big["lse"][:M]
    bl.bl_linear_xent_forward(h, W, t, big["loss"][:M], lse, big["ws"][:n])
    bl.bl_linear_xent_backward(h, W, t, lse, dl, big["dH"][:M], big["dW"][:V], big["ws"][:n])
    torch.cuda.synchronize()
    assert torch.equal(big["loss"][:M], a.loss) and torch.equal(big["dH"][:M], a.dH) and torch.equal(big["dW"][:V], a.dW)
    assert bool((big["loss"][M:] == 7).all()) and bool((big["lse"][M:] == 7).all()) and bool((big["dH"][M:] == 7).all()) and bool((big["dW"][V:] == 7).all())
    assert bool((big["ws"][n:] == 0xA5).all())


@pytest.mark.parametrize("M", [20, 6])
def test_gradients_by_differences(M):
    """Directional differences of the 64-bit loss at the bf16 inputs."""
    V, K = 300, 64
    h, W, t, dl = case(M, V, K, seed=4, left_out=0.2)
    b = run(h, W, t, dl, F32)
    live = t >= 0

    def loss(h, W):
        z = h @ W.t()
        each = torch.logsumexp(z, 1) - z.gather(1, t.clamp(min=0)[:, None])[:, 0]
        return (torch.where(live, each, 0.0) * dl.double()).sum()
    g = torch.Generator(device="cuda").manual_seed(6)
    e = 1e-5
    for grad, at, rel in ((b.dH, 0, 2.0 ** -7), (b.dW, 1, 2.0 ** -14)):
        v = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        hi, lo = [h.double(), W.double()], [h.double(), W.double()]
        hi[at], lo[at] = hi[at] + e * v, lo[at] - e * v
        num = float((loss(*hi) - loss(*lo)) / (2 * e))
        # dz's and the result's roundings, at most, of every term
        assert abs(num - float((grad.double() * v).sum())) <= rel * float((grad.double() * v).abs().sum()) + 1e-7


@pytest.mark.parametrize("M", [200, 5])
def test_other_stream_and_graphs_sharing_a_workspace(M):
    V, K = 900, 128
    cases = [case(M, V, K, seed=i) for i in (21, 22)]
    want = [run(*c) for c in cases]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = run(*cases[0], stream=side)
    assert torch.equal(b.dW, want[0].dW) and torch.equal(b.loss, want[0].loss)
    # two graphs over one workspace, replayed in turn on one stream
    ws = torch.empty(b.workspace.numel(), dtype=torch.uint8, device="cuda")
    graphs, outs, ins = [], [], []
    for c in cases:
        o = bl.XentBuffers.allocate(M, V, K)
        i = [x.clone() for x in cases[0]]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="thread_local"):
            bl.bl_linear_xent_forward(*i[:3], o.loss, o.lse, ws)
            bl.bl_linear_xent_backward(*i[:3], o.lse, i[3], o.dH, o.dW, ws)
        graphs.append(g), outs.append(o), ins.append(i)
    for _ in range(2):
        for k in (0, 1):
            for dst, src in zip(ins[k], cases[k]):
                dst.copy_(src)
            graphs[k].replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o.loss, w.loss) and torch.equal(o.dH, w.dH) and torch.equal(o.dW, w.dW)
    assert bl.bl_get_last_error() == 0


@pytest.mark.parametrize("M", [3, 9, 18])
def test_weight_offsets_past_32_bits(M):
    """A head of more than 2^31 weights: loss, lse and the gradients' last rows
    against 64-bit sums over blocks of the vocabulary."""
    K = 1024
    V = 2 ** 31 // K + 3000
    g = torch.Generator(device="cuda").manual_seed(1)
    W = torch.empty(V, K, dtype=BF, device="cuda")
    for i in range(0, V, 65536):
        W[i:i + 65536] = (torch.randn(min(65536, V - i), K, generator=g, device="cuda") * 0.03).to(BF)
    h = torch.randn(M, K, generator=g, device="cuda").to(BF)
    t = torch.tensor([V - 1, 5, V - 2000] * (M // 3), device="cuda")
    dl = torch.tensor([0.5, 0.25, 1.0] * (M // 3), device="cuda")
    b = run(h, W, t, dl)
    hd = h.double()
    z = torch.cat([hd @ W[i:i + 65536].double().t() for i in range(0, V, 65536)], 1)
    ez = (K / 16 + 4) * S * 3 * K ** 0.5     # sum |h W| is below 3 sqrt(K) here (K products of mean 0.02)
    lse = torch.logsumexp(z, 1)
    assert bool(((b.lse.double() - lse).abs() <= ez + 8 * S * lse).all())
    assert bool(((b.loss.double() - (lse - z[torch.arange(M), t])).abs() <= 2 * ez + 16 * S * lse).all())
    dz = torch.exp(z - lse[:, None])
    dz[torch.arange(M), t] -= 1
    dz *= dl.double()[:, None]
    want = dz[:, -3000:].t() @ hd
    tol = (2.0 ** -8 + 2 * ez + 1e-5) * (dz[:, -3000:].abs().t() @ hd.abs())
    assert bool(((b.dW[-3000:].double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol) + 1e-36).all())
    dH = sum(dz[:, i:i + 65536] @ W[i:i + 65536].double() for i in range(0, V, 65536))
    mag = sum(dz[:, i:i + 65536].abs() @ W[i:i + 65536].double().abs() for i in range(0, V, 65536))
    tol = (2.0 ** -8 + 2 * ez + 1e-5 + V / 16 * S / 8) * mag
    assert bool(((b.dH.double() - dH).abs() <= tol + 2.0 ** -8 * (dH.abs() + tol)).all())


@pytest.mark.parametrize("M", [300, 4])
def test_two_calls_side_by_side(M):
    """Two steps on two streams at once, each with its own buffers."""
    args = [case(M, 5000, 256, seed=s) for s in (31, 32)]
    want = [run(*a) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    bufs = [[bl.XentBuffers.allocate(M, 5000, 256) for _ in args] for _ in range(6)]
    torch.cuda.synchronize()
    for row in bufs:
        for (h, W, t, dl), b, s in zip(args, row, streams):
            bl.bl_linear_xent_forward(h, W, t, b.loss, b.lse, b.workspace, stream=s)
            bl.bl_linear_xent_backward(h, W, t, b.lse, dl, b.dH, b.dW, b.workspace, stream=s)
    torch.cuda.synchronize()
    for row in bufs:
        for b, w in zip(row, want):
            assert torch.equal(b.loss, w.loss) and torch.equal(b.dH, w.dH) and torch.equal(b.dW, w.dW)
    assert bl.bl_get_last_error() == 0


@pytest.mark.parametrize("M", [200, 8])
def test_uniform_and_wide_ranges_of_dloss(M):
    """A mean (equal dloss), signs, zeros and magnitudes far apart."""
    h, W, t, _ = case(M, 600, 128, seed=8)
    for dl in (torch.full((M,), 1 / 777.0), torch.linspace(-1, 1, M), torch.zeros(M),
               torch.logspace(-30, 3, M), torch.full((M,), -1e-20)):
        dl = dl.to(torch.float32).cuda()
        b = run(h, W, t, dl)
        check(b, h, W, t, dl)
    # equal dloss: dz's target term is exact before the products, so the whole
    # gradient is off by the other terms' roundings and the result's own only
    dl = torch.full((M,), 1 / 777.0, device="cuda")
    b = run(h, W, t, dl)
    p = torch.softmax(h.double() @ W.double().t(), 1)
    p[torch.arange(M), t] -= 1
    want = (p / 777.0) @ W.double()
    assert float((b.dH.double() - want).norm()) <= 1.5 * 2.0 ** -9 * float(want.norm())


def test_refused_on_the_gpu():
    h, W, t, dl = case(4, 100, 64)
    b = bl.XentBuffers.allocate(4, 100, 64)
    for bad in (dict(h=h.float()), dict(W=W[:, :32]), dict(targets=t.int()), dict(loss=b.loss.double()), dict(lse=b.lse[:2]),
                dict(h=h.cpu()), dict(workspace=b.workspace.cpu()), dict(W=W.t().contiguous().t())):
        a = dict(h=h, W=W, targets=t, loss=b.loss, lse=b.lse, workspace=b.workspace) | bad
        with pytest.raises(ValueError):
            bl.bl_linear_xent_forward(**a)
    with pytest.raises(bl.BitLinearError, match="workspace"):
        bl.bl_linear_xent_forward(h, W, t, b.loss, b.lse, b.workspace[:16])
    with pytest.raises(bl.BitLinearError, match="multiple of 8"):
        bl.bl_linear_xent_forward(h[:, :60].contiguous(), W[:, :60].contiguous(), t, b.loss, b.lse, b.workspace)
    with pytest.raises(ValueError):
        bl.bl_linear_xent_backward(h, W, t, b.lse, dl, b.dH, b.dW.half(), b.workspace)
    assert bl.bl_get_last_error() == 0


# a few tokens: their own kernels, by one or two groups of 8 tokens, units of 16 rows of W,
# steps of 32 columns (128 at once) and tiles of 64; a vocabulary of less than
# one unit, and one whose units are dealt out unevenly
FEW = [(1, 5, 8), (1, 33, 2048), (2, 31, 2056), (3, 129, 4088), (4, 4737, 4096), (4, 20001, 512), (5, 4, 2048), (5, 1, 8), (6, 9473, 520),
       (7, 40000, 16), (8, 3, 2040), (8, 1000, 2048), (8, 66000, 72), (5, 700, 2056), (8, 300, 4096), (9, 700, 512), (4, 300, 4104),
       (16, 1009, 136), (17, 1009, 136), (25, 15, 264), (32, 17, 8192), (32, 40001, 160), (11, 1, 65536), (7, 1, 65536), (8, 40, 65536), (2, 600, 32768), (1, 37889, 24), (33, 500, 264), (9, 31, 8), (15, 4000, 8184), (16, 66001, 88), (12, 17, 65536), (10, 9473, 520)]


@pytest.mark.parametrize("dw_dtype", [BF, F32])
@pytest.mark.parametrize("M,V,K", FEW)
def test_few_tokens(M, V, K, dw_dtype):
    args = case(M, V, K, seed=M * V + K, left_out=0.3 if M > 3 else 0.0)
    check(run(*args, dw_dtype), *args, dw_dtype)


@pytest.mark.parametrize("M,V,K", [(3, 2500, 4096), (8, 2500, 512), (13, 3000, 200), (32, 900, 1000)])
@pytest.mark.parametrize("dw_dtype", [BF, F32])
def test_few_tokens_left_out_accumulated_and_parts(M, V, K, dw_dtype):
    h, W, t, dl = case(M, V, K, seed=2)
    t[1], dl[1] = -1, float("nan")
    clean = h.clone()
    h[1], clean[1] = float("nan"), 0.0
    dW0 = torch.randn(V, K, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(dw_dtype)
    b = run(h, W, t, dl, dw_dtype, dW=dW0.clone(), accumulate=True)
    b.lse[1] = torch.logsumexp(clean[1].double() @ W.double().t(), 0)  # of the token itself: not a number
    check(b, clean, W, t, dl, dw_dtype, dW0=dW0)
    again = run(h, W, t, dl, dw_dtype, dW=dW0.clone(), accumulate=True)
    assert torch.equal(b.dW, again.dW) and torch.equal(b.dH, again.dH) and torch.equal(b.loss, again.loss)
    # one gradient without the other
    dH, dW = torch.empty_like(b.dH), torch.empty_like(b.dW)
    bl.bl_linear_xent_backward(h, W, t, again.lse, dl, dH, None, b.workspace)
    bl.bl_linear_xent_backward(h, W, t, again.lse, dl, None, dW, b.workspace)
    whole = run(h, W, t, dl, dw_dtype)
    assert torch.equal(dH, whole.dH) and torch.equal(dW, whole.dW)
    assert bl.bl_get_last_error() == 0


@pytest.mark.parametrize("M,K", [(2, 2560), (8, 512), (20, 128)])
def test_few_tokens_with_infinite_and_no_number_logits(M, K):
    h, W, t, dl = case(M, 700, K, seed=4)
    W[11, 3], h[:, 3] = float("-inf"), 1.0  # a logit of -inf: probability zero
    t[:] = 5
    b = run(h, W, t, dl)
    z = h.float() @ W.float().t()
    assert torch.isfinite(b.loss).all() and torch.allclose(b.lse, torch.logsumexp(z, 1), rtol=1e-4, atol=1e-4)
    assert bool((b.dW[11] == 0).all())
    W[11, 3] = float("nan")
    b = run(h, W, t, dl)
    assert bool(b.loss.isnan().all()) and bool(b.lse.isnan().all())
