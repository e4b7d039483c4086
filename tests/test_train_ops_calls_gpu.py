"""GPU: calls of the training operators that their documentation allows, in the
shapes, buffers and views that a training loop brings them."""

import pytest
import torch

import ternary_weight_quantization_b200 as bl
from ternary_weight_quantization_b200 import lm as plm

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def rnd(*shape, seed=0, dtype=F32, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def targets(M, V, seed=0):
    return torch.randint(-1, V, (M,), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def ok():
    torch.cuda.synchronize()
    assert bl.bl_get_last_error() == 0


# ----------------------------------------------------------------- head cross-entropy: workspaces
@pytest.mark.parametrize("M,V,K", [(391, 1739, 3312), (30, 8192, 512), (140, 700, 136), (9, 700, 136)])
def test_dh_alone_with_the_buffers_of_an_fp32_dw(M, V, K):
    h, W, t, dl = rnd(M, K, dtype=BF), rnd(V, K, seed=1, dtype=BF, scale=0.02), targets(M, V), torch.full((M,), 0.01, device="cuda")
    b = bl.XentBuffers.allocate(M, V, K, F32)
    bl.bl_linear_xent_forward(h, W, t, b.loss, b.lse, b.workspace)
    bl.bl_linear_xent_backward(h, W, t, b.lse, dl, b.dH, None, b.workspace)
    ok()
    z = h.double() @ W.double().t()
    dz = torch.softmax(z, 1)
    dz[torch.arange(M, device="cuda"), t.clamp(min=0)] -= 1
    dz = torch.where((t >= 0)[:, None], dz * dl.double()[:, None], 0.0)
    want, mag = dz @ W.double(), dz.abs() @ W.double().abs()
    # dz and dH rounded to bf16 (2^-8 each, at most); a tensor-core sum drops up
    # to a step of fp32 per 16 terms: of the logits (an error of p's exponent)
    # and of dH
    e = (K / 16 + 16) * 2.0 ** -23 * float((h.double().abs() @ W.double().abs().t()).amax())
    tol = (2.0 ** -8 + 2 * e + (V / 16 + 64) * 2.0 ** -23) * mag
    assert bool(((b.dH.double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol) + 1e-36).all())


def test_frozen_head():
    """The loss's gradient for h alone, as when the head is not trained."""
    M, V, K = 391, 1739, 3312
    h, W, t = rnd(M, K).requires_grad_(True), rnd(V, K, seed=1, scale=0.02), targets(M, V)
    dh, = torch.autograd.grad(plm.HeadLossFunction.apply(h, W, t), [h])
    both = torch.autograd.grad(plm.HeadLossFunction.apply(h, W.requires_grad_(True), t), [h, W])
    ok()
    # dz goes to dH in bf16 either way; the order of dH's partial sums differs
    assert float((dh - both[0]).norm()) <= 2.0 ** -8 * float(both[0].norm())
    assert bool(both[1].any())


@pytest.mark.parametrize("M,short,V,K,dt", [(2048, 1310, 50257, 768, BF), (257, 256, 8192, 512, F32), (40, 9, 5000, 264, BF)])
def test_short_batch_in_the_buffers_of_a_whole_one(M, short, V, K, dt):
    h, W, t, dl = rnd(M, K, dtype=BF), rnd(V, K, seed=1, dtype=BF, scale=0.02), targets(M, V), torch.full((M,), 0.01, device="cuda")
    b, own = bl.XentBuffers.allocate(M, V, K, dt), bl.XentBuffers.allocate(short, V, K, dt)
    n = short
    for x in (b, own):
        bl.bl_linear_xent_forward(h[:n], W, t[:n], x.loss[:n], x.lse[:n], x.workspace)
        bl.bl_linear_xent_backward(h[:n], W, t[:n], x.lse[:n], dl[:n], x.dH[:n], x.dW, x.workspace)
    ok()
    assert torch.equal(b.loss[:n], own.loss) and torch.equal(b.lse[:n], own.lse)
    assert torch.equal(b.dH[:n], own.dH) and torch.equal(b.dW, own.dW) and bool(own.dW.isfinite().all())


# ----------------------------------------------------------------- the LM's functions
def off(t, n=1):
    """The same values n elements into a larger storage."""
    x = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)[n:].view(t.shape)
    return x.copy_(t)


def test_views_that_start_off_a_16_byte_boundary():
    """Inputs and gradients that are views into other tensors give what their
    copies give."""
    M, K, V = 6, 40, 100
    x, w, up, gy = rnd(M, K), rnd(K, seed=1), rnd(M, K, seed=2), rnd(M, K, seed=3)
    head, t = rnd(V, K, seed=4, scale=0.1), targets(M, V)
    calls = {
        "norm": (lambda a, b: plm.RMSNormFunction.apply(a, b, 1e-6, False), (x, w), gy),
        "norm saved8": (lambda a, b: plm.RMSNormFunction.apply(a, b, 1e-6, True), (x, w), gy),
        "gate": (plm.SwigluFunction.apply, (x, up), gy),
        "gate bf16": (plm.SwigluFunction.apply, (x.to(BF), up.to(BF)), gy.to(BF)),
    }
    for name, (call, args, g) in calls.items():
        want, got = ([a.clone().requires_grad_(True) for a in args] for _ in range(2))
        got = [off(a.detach()).requires_grad_(True) for a in got]
        yw, yg = call(*want), call(*got)
        assert off(g).data_ptr() % 16 and got[0].data_ptr() % 16
        pairs = zip([yw, *torch.autograd.grad(yw, want, g)], [yg, *torch.autograd.grad(yg, got, off(g))])
        assert all(torch.equal(a, b) for a, b in pairs), name
    for dt in (F32, BF):
        h1, w1 = x.to(dt).requires_grad_(True), head.to(dt).requires_grad_(True)
        h2, w2 = off(x.to(dt)).requires_grad_(True), off(head.to(dt)).requires_grad_(True)
        a, b = plm.HeadLossFunction.apply(h1, w1, t), plm.HeadLossFunction.apply(h2, w2, off(t))
        pairs = zip([a, *torch.autograd.grad(a, [h1, w1])], [b, *torch.autograd.grad(b, [h2, w2])])
        assert all(torch.equal(p, q) for p, q in pairs), dt
    ok()


def test_batch_of_one_sequence():
    """One sequence: its targets are a view that starts 8 bytes into the ids."""
    from workloads.lm import LM_TINY, lm_batches, lm_init
    params = {n: p.cuda().requires_grad_(True) for n, p in lm_init(LM_TINY, seed=1).items()}
    ids = lm_batches(LM_TINY, seed=1)[0].cuda()
    one = plm.lm_loss(params, ids[:1], LM_TINY, library_ops=True)
    assert all(bool(g.isfinite().all()) for g in torch.autograd.grad(one, list(params.values())))
    # a zero head: every probability is 1 / V, exactly in fp32 up to the log
    import math
    assert abs(float(one.detach()) - math.log(LM_TINY.vocab)) <= 16 * 2.0 ** -23 * math.log(LM_TINY.vocab)
    ok()


# ----------------------------------------------------------------- SwiGLU
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [136, 131])
def test_gates_far_below_zero_next_to_large_values(K, dtype):
    """1 / (1 + exp(-g)) down to where exp(-g) leaves fp32 (g = -88.7): below
    2^-126 from g = -87.4 on, which large values of up and dy make visible."""
    gates = torch.tensor([-80.0, -86.0, -87.0, -87.5, -88.0, -88.5, -20.0, 80.0], device="cuda")
    M = gates.numel()
    gate = gates[:, None].expand(M, K).to(dtype).contiguous()
    up, dy = torch.full_like(gate, 2.0 ** 90), torch.full_like(gate, 2.0 ** 25)
    b = bl.SwigluBuffers.allocate(M, K, dtype)
    bl.bl_swiglu_forward(gate, up, b.y, b.gate8, b.up8)
    bl.bl_swiglu_backward(dy, b.gate8, b.up8, b.dgate, b.dup)
    ok()
    half = torch.finfo(dtype).eps / 2

    def close(got, want, g, what):
        # g log2(e) rounded in exp's argument, exp, sum, quotient and products,
        # the quotient on the grid of 2^-149 (2.4e-7 of 2.9e-39), the result
        rel = (20 + 4 * g.abs()) * 2.0 ** -23 + 2.0 ** -21 + 2 * half
        assert bool(((got.double() - want).abs() <= rel * want.abs()).all()), (what, got[:, 0], want[:, 0])
    g = gate.double()
    close(b.y, g * torch.sigmoid(g) * up.double(), g, "y")
    # the saved value of a constant group: the constant to three roundings
    g, u = ((t.codes.double() * t.scales.double().repeat_interleave(128, 1)[:, :K]).float().double() for t in (b.gate8, b.up8))
    d = dy.double()
    s = torch.sigmoid(g)
    close(b.dup, d * g * s, g, "dup")
    close(b.dgate, d * u * s * (1 + g * (1 - s)), g, "dgate")


# ----------------------------------------------------------------- norms
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [64, 100, 1032, 8200, 10001])
def test_mean_of_rows_with_infinities(K, dtype):
    """The mean is the sum over K also where that is infinite; y and rstd of such
    a row are not numbers, as the formula says, and other rows are untouched."""
    inf = float("inf")
    x = rnd(6, K, dtype=dtype)
    x[1, 3], x[2, K - 1], x[3, 0], x[3, 1], x[4, 5] = inf, -inf, inf, -inf, float("nan")
    clean = rnd(6, K, dtype=dtype)
    y, mean, rstd = torch.empty_like(x), torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    y2, mean2, rstd2 = torch.empty_like(x), torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    bl.bl_norm_forward(x, None, None, 1e-6, y, mean, rstd)
    bl.bl_norm_forward(clean, None, None, 1e-6, y2, mean2, rstd2)
    ok()
    assert float(mean[1]) == inf and float(mean[2]) == -inf
    assert bool(mean[3:5].isnan().all()) and bool(rstd[1:5].isnan().all()) and bool(y[1:5].isnan().all())
    for a, b in ((y, y2), (mean, mean2), (rstd, rstd2)):
        assert torch.equal(a[[0, 5]], b[[0, 5]])


@pytest.mark.parametrize("M,K", [(3, 512), (16, 64), (20, 128), (300, 72)])
def test_infinite_logits(M, K):
    """+infinity makes its token's loss and lse NaN, other tokens keep theirs."""
    V = 700
    h, W, t = rnd(M, K, dtype=BF), rnd(V, K, seed=1, dtype=BF, scale=0.05), targets(M, V).clamp(min=0)
    h[:, 3] = 0
    b = bl.XentBuffers.allocate(M, V, K)
    bl.bl_linear_xent_forward(h, W, t, b.loss, b.lse, b.workspace)
    loss, lse = b.loss.clone(), b.lse.clone()
    h2 = h.clone()
    h2[1, 3] = 1e30
    big = W.clone()
    big[:, 3] = 0
    big[11, 3] = 3e38          # token 1's logit of row 11 overflows; the others have 0 there
    W0 = W.clone()
    W0[:, 3] = 0
    bl.bl_linear_xent_forward(h, W0, t, b.loss, b.lse, b.workspace)
    torch.cuda.synchronize()
    assert torch.equal(b.loss, loss) and torch.equal(b.lse, lse)     # h is 0 there
    bl.bl_linear_xent_forward(h2, big, t, b.loss, b.lse, b.workspace)
    ok()
    rest = [i for i in range(M) if i != 1]
    assert bool(b.loss[1].isnan()) and bool(b.lse[1].isnan())
    assert torch.equal(b.loss[rest], loss[rest]) and torch.equal(b.lse[rest], lse[rest])


# ----------------------------------------------------------------- head cross-entropy: ragged tiles
@pytest.mark.parametrize("M,V,K", [(359, 8263, 3888), (359, 8263, 8000), (130, 300, 32768), (300, 5120 + 64, 4096), (20, 130, 65536),
                                   (257, 1025, 8192), (1025, 257, 8192)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_tiles_of_which_one_cta_holds_no_rows(M, V, K, dt):
    """Token and vocabulary tiles that end in their first half, over many stages:
    the second CTA of the last pair has nothing to load, and no wait may run out."""
    h, W, t, dl = rnd(M, K, dtype=BF), rnd(V, K, seed=1, dtype=BF, scale=0.02), targets(M, V), torch.full((M,), 1 / M, device="cuda")
    b = bl.XentBuffers.allocate(M, V, K, dt)
    for _ in range(3):
        bl.bl_linear_xent_forward(h, W, t, b.loss, b.lse, b.workspace)
        bl.bl_linear_xent_backward(h, W, t, b.lse, dl, b.dH, b.dW, b.workspace)
        ok()
    z = h.double() @ W.double().t()
    lse = torch.logsumexp(z, 1)
    e = (K / 16 + 16) * 2.0 ** -23 * float((h.double().abs() @ W.double().abs().t()).amax())
    assert bool(((b.lse.double() - lse).abs() <= e + 2.0 ** -19 * (1 + lse.abs())).all())
    dz = torch.exp(z - lse[:, None])
    dz[torch.arange(M, device="cuda"), t.clamp(min=0)] -= 1
    dz = torch.where((t >= 0)[:, None], dz * dl.double()[:, None], 0.0)
    for got, a, c, n in ((b.dH, dz, W.double(), V), (b.dW, dz.t(), h.double(), M)):
        want, mag = a @ c, a.abs() @ c.abs()
        # dz's and the result's roundings, p's exponent, a step per 16 terms
        tol = (2.0 ** -8 + 2 * e + (n / 16 + 64) * 2.0 ** -23) * mag
        assert bool(((got.double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol) + 1e-36).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [144, 1312, 8176, 14768, 141])
def test_norm_backward_uses_the_rounded_saved_values(K, dtype):
    """One row, whose dweight is dy xhat: also where a saved value lies next to
    the mean, x - mean is that of the fp32 saved value, in every kernel."""
    from tests.test_rows_gpu import saved_values
    M = 1
    for seed in range(8):
        x, w, dy = (rnd(M, K, seed=seed) + 0.5).to(dtype), torch.ones(K, device="cuda"), rnd(M, K, seed=seed + 100, dtype=dtype)
        b = bl.NormBuffers.allocate(M, K, dtype, F32, saved8=True)
        bl.bl_norm_forward(x, w, None, 1e-6, b.y, b.mean, b.rstd, saved8=b.saved8)
        bl.bl_norm_backward(dy, b.saved8, w, b.mean, b.rstd, b.dx, b.dweight, None, b.workspace)
        ok()
        want = dy.double() * (saved_values(x)[2].double() - b.mean.double()[:, None]) * b.rstd.double()[:, None]
        # three roundings of half a step
        assert bool(((b.dweight.double() - want[0]).abs() <= 3.001 * 2.0 ** -24 * want[0].abs()).all())


@pytest.mark.parametrize("M,V", [(16, 151936), (5, 1 << 20), (48, 151936), (300, 32000), (20, 1 << 20)])
def test_lse_keeps_its_bits_over_many_joins(M, V):
    """Logits that are exact in fp32 and all alike, or all alike but a few: lse
    is the logit plus log V, whatever the number of partial sums."""
    K = 8
    h, W = torch.zeros(M, K, dtype=BF, device="cuda"), torch.zeros(V, K, dtype=BF, device="cuda")
    h[:, 0] = torch.linspace(-90, 90, M, device="cuda").to(BF)
    W[:, 0] = 1.0
    W[::1000, 0] = 0.5
    t = torch.arange(M, device="cuda") * 3 + 1
    b = bl.XentBuffers.allocate(M, V, K, backward=False)
    bl.bl_linear_xent_forward(h, W, t, b.loss, b.lse, b.workspace)
    ok()
    z = h[:, 0].double()[:, None] * torch.tensor([1.0, 0.5], device="cuda", dtype=torch.float64)
    n = -(-V // 1000)
    lse = torch.logsumexp(z + torch.log(torch.tensor([V - n, n], device="cuda", dtype=torch.float64)), 1)
    # the sum: additions that a term goes through (16 in a chunk, 4 chunks, a
    # thread's parts and 12 joins; few tokens: a lane's logits), ex2's and log's
    # two units each; z log2 e and the result: half a step of lse each, log2 e
    # and ln 2 another
    adds = 40 + max(V / 128 / 64, V / (16 * 8 * 296) * 2)
    tol = (adds / 2 + 8) * 2.0 ** -23 + 3 * 2.0 ** -24 * 2 * lse.abs()
    assert bool(((b.lse.double() - lse).abs() <= tol).all()), ((b.lse.double() - lse).abs() / tol).max()
    live = lse - z[:, 0]
    assert bool(((b.loss.double() - live).abs() <= 2 * tol).all())


def test_calls_from_two_host_threads():
    """Two threads, each with its own stream and buffers, at once: the same bits
    as the calls alone, by the current stream and by one that is given."""
    import threading
    M, K, V = 300, 264, 5000
    sets = [(rnd(M, K, seed=s, dtype=BF), rnd(V, K, seed=s + 1, dtype=BF, scale=0.05), targets(M, V, s), rnd(K, seed=s + 2))
            for s in (1, 11)]
    dl = torch.full((M,), 1 / M, device="cuda")

    def chain(h, W, t, w, stream=None):
        x, n, g = bl.XentBuffers.allocate(M, V, K), bl.NormBuffers.allocate(M, K, saved8=True), bl.SwigluBuffers.allocate(M, K)
        bl.bl_norm_forward(h, w, None, 1e-6, n.y, n.mean, n.rstd, saved8=n.saved8, stream=stream)
        bl.bl_swiglu_forward(n.y, h, g.y, g.gate8, g.up8, stream=stream)
        bl.bl_linear_xent_forward(g.y, W, t, x.loss, x.lse, x.workspace, stream=stream)
        bl.bl_linear_xent_backward(g.y, W, t, x.lse, dl, x.dH, x.dW, x.workspace, stream=stream)
        bl.bl_swiglu_backward(x.dH, g.gate8, g.up8, g.dgate, g.dup, stream=stream)
        bl.bl_norm_backward(g.dgate, n.saved8, w, n.mean, n.rstd, n.dx, n.dweight, None, n.workspace, stream=stream)
        return [x.loss, x.lse, x.dH, x.dW, g.dgate, g.dup, n.dx, n.dweight]
    want = [chain(*s) for s in sets]
    ok()
    got = [[], []]

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for k in range(10):
                got[i].append(chain(*sets[i], stream=stream if k % 2 else None))
        stream.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    ok()
    for runs, w in zip(got, want):
        assert len(runs) == 10
        assert all(torch.equal(a, b) for run in runs for a, b in zip(run, w))
