"""GPU: calls of the norm with an INT8 result, of the product of INT8 operands
and of the gradients' clipping that their documentation allows: on streams, in
graphs, side by side, in the buffers of a larger batch, past 32-bit offsets; and
the LM's functions over them."""

import math
import threading

import pytest
import torch

import ternary_weight_quantization_b200 as bl
from tests.test_quant_ops_gpu import (BF, EPS, F32, U, check_backward, check_clip, check_forward, close, codes, gradients,
                                      norm64, norm_inputs, ok, product, rnd, scales, tensors, workspace)
from ternary_weight_quantization_b200 import lm as plm
from workloads.lm import LM_TINY, lm_batches, lm_init

pytestmark = pytest.mark.gpu


class Step:
    """An 8-bit layer's step: norm, product, gradients, clipping; every buffer its own."""

    def __init__(self, M, K, N, seed=0, st=F32):
        self.M, self.K, self.N = M, K, N
        self.x, self.r, self.w = norm_inputs(M, K, BF, st, F32, seed=seed)
        self.wq, self.sw = codes(N, K, seed=seed + 3), scales(N, seed + 4)
        self.dY, self.dsum = rnd(M, N, seed=seed + 5, dtype=BF, scale=0.1), rnd(M, K, seed=seed + 6, dtype=st)
        self.n = bl.NormQuantBuffers.allocate(M, K, BF, st, F32)
        self.l = bl.Int8LinearBuffers.allocate(M, N, K, F32, F32)
        self.norm, self.ws = torch.zeros(1, device="cuda"), workspace(3)
        self.clipped = [torch.empty_like(t) for t in (self.l.dW, self.n.dweight, self.n.dresidual)]

    def run(self, stream=None):
        n, l = self.n, self.l
        bl.bl_norm_quant_forward(self.x, self.r, self.w, EPS, n.sum, n.rstd, n.xq, n.sx, stream=stream)
        bl.bl_int8_linear_forward(n.xq, n.sx, self.wq, self.sw, l.y, stream=stream)
        bl.bl_int8_linear_backward(self.dY, n.xq, n.sx, self.wq, self.sw, l.dX, l.dW, stream=stream, workspace=l.workspace)
        bl.bl_norm_quant_backward(l.dX, self.dsum, n.sum, self.w, n.rstd, n.dx, n.dresidual, n.dweight, n.workspace, stream=stream)
        bl.bl_clip_grads([l.dW, n.dweight, n.dresidual], 1.0, self.norm, self.ws, out=self.clipped, stream=stream)

    def outputs(self):
        n, l = self.n, self.l
        return [n.sum, n.rstd, n.xq, n.sx, l.y, l.dX, l.dW, n.dx, n.dresidual, n.dweight, self.norm, *self.clipped]

    def wipe(self):
        for t in self.outputs():
            t.fill_(7)


# one shape per kernel of the product: a few tokens, tens, tiles
SHAPES = [(5, 256, 520), (40, 512, 1000), (300, 1408, 512)]


def same(a, b):
    assert all(torch.equal(x, y) for x, y in zip(a, b, strict=True))


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_a_step_against_64_bits(M, K, N):
    """The calls as they follow one another in a training step."""
    s = Step(M, K, N)
    s.run()
    ok()
    check_forward(s.n.sum, s.w, s.n)
    assert torch.equal(s.l.y, product(s.n.xq, s.n.sx, s.wq, s.sw, F32))
    x = (s.n.xq.float() * s.n.sx[:, None]).to(BF).double()
    w = (s.wq.float() * s.sw[:, None]).to(BF).double()
    d = s.dY.double()
    close(s.l.dX, d @ w, (N / 16 + 64) * 2 * U * (d.abs() @ w.abs()), "dX")
    close(s.l.dW, d.t() @ x, (M / 16 + 64) * 2 * U * (d.abs().t() @ x.abs()), "dW")
    check_backward(s.l.dX, s.dsum, s.n.sum, s.w, s.n)
    total = norm64([s.l.dW, s.n.dweight, s.n.dresidual])
    assert abs(float(s.norm) - total) <= 7 * U * total
    factor = min(1.0, 1.0 / total)
    for g, c in zip((s.l.dW, s.n.dweight, s.n.dresidual), s.clipped):
        close(c, g.double() * factor, 9 * U * g.double().abs() * factor, "clipped")


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_equal_inputs_give_equal_bits_on_any_stream(M, K, N):
    s = Step(M, K, N)
    s.run()
    ok()
    want = [t.clone() for t in s.outputs()]
    for w in (s.l.workspace, s.n.workspace, s.ws):
        w.fill_(255)
    s.wipe()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s.run(stream=side)
    ok()
    same(s.outputs(), want)
    s.wipe()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    ok()
    same(s.outputs(), want)


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_captured_steps_replay_on_new_inputs_and_side_by_side(M, K, N):
    a, b = Step(M, K, N), Step(M, K, N, seed=50)
    stream = torch.cuda.Stream()
    graphs = []
    for s in (a, b):
        s.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            s.run()
        graphs.append(g)
    want = []
    for s, seed in ((a, 100), (b, 200)):
        fresh = Step(M, K, N, seed=seed)
        fresh.run()
        ok()
        want.append([t.clone() for t in fresh.outputs()])
        for name in ("x", "r", "w", "wq", "sw", "dY", "dsum"):
            getattr(s, name).copy_(getattr(fresh, name))
        s.wipe()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    ok()
    same(a.outputs(), want[0])
    same(b.outputs(), want[1])


def test_calls_from_two_host_threads():
    steps = [Step(33, 512, 264, seed=1), Step(300, 256, 1000, seed=9)]
    want = []
    for s in steps:
        s.run()
        ok()
        want.append([t.clone() for t in s.outputs()])
        s.wipe()
    torch.cuda.synchronize()
    failed = []

    def work(s):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    s.run()
        except Exception as e:  # noqa: BLE001 (told to the test's own thread)
            failed.append(e)
    threads = [threading.Thread(target=work, args=(s,)) for s in steps]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    ok()
    assert not failed
    for s, w in zip(steps, want):
        same(s.outputs(), w)


@pytest.mark.parametrize("short", [1, 16, 17, 64, 65, 250])
def test_short_batch_in_the_buffers_of_a_whole_one(short):
    """Rows behind the last token stay as they were."""
    M, K, N = 300, 528, 264
    whole, own = Step(M, K, N), Step(M, K, N)
    n, l = whole.n, whole.l
    whole.wipe()
    k = short
    bl.bl_norm_quant_forward(whole.x[:k], whole.r[:k], whole.w, EPS, n.sum[:k], n.rstd[:k], n.xq[:k], n.sx[:k])
    bl.bl_int8_linear_forward(n.xq[:k], n.sx[:k], whole.wq, whole.sw, l.y[:k])
    bl.bl_int8_linear_backward(whole.dY[:k], n.xq[:k], n.sx[:k], whole.wq, whole.sw, l.dX[:k], l.dW, workspace=l.workspace)
    bl.bl_norm_quant_backward(l.dX[:k], whole.dsum[:k], n.sum[:k], whole.w, n.rstd[:k], n.dx[:k], n.dresidual[:k], n.dweight,
                              n.workspace)
    ok()
    for t in (n.sum, n.rstd, n.xq, n.sx, l.y, l.dX, n.dx, n.dresidual):
        assert bool((t[k:] == 7).all())
    own.run()
    ok()
    # a token's forward does not depend on the others
    same([n.sum[:k], n.rstd[:k], n.xq[:k], n.sx[:k], l.y[:k]], [own.n.sum[:k], own.n.rstd[:k], own.n.xq[:k], own.n.sx[:k], own.l.y[:k]])
    x = (n.xq[:k].float() * n.sx[:k, None]).to(BF).double()
    d = whole.dY[:k].double()
    close(l.dW, d.t() @ x, (k / 16 + 64) * 2 * U * (d.abs().t() @ x.abs()), "dW")

    class Part:
        dresidual, dx, dweight = n.dresidual[:k], n.dx[:k], n.dweight
    check_backward(l.dX[:k], whole.dsum[:k], n.sum[:k], whole.w, Part)


# ----------------------------------------------------------------- offsets past 32 bits
def test_norm_quant_past_32_bit_offsets():
    M, K = 264000, 8192          # 2.16e9 values
    x = torch.full((M, K), 0.5, dtype=BF, device="cuda")
    tail = rnd(3, K, dtype=BF)
    x[-3:] = tail
    w = 1 + rnd(K, seed=1, scale=0.3)
    rstd, sx = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    xq = torch.empty(M, K, dtype=torch.int8, device="cuda")
    bl.bl_norm_quant_forward(x, None, w, EPS, None, rstd, xq, sx)
    ok()

    class Part:
        pass
    Part.rstd, Part.xq, Part.sx = rstd[-3:], xq[-3:], sx[-3:]
    check_forward(tail, w, Part)
    assert torch.equal(xq[0], xq[M // 2]) and torch.equal(xq[0], xq[-4])
    dweight, ws = torch.empty(K, device="cuda"), torch.empty(bl.bl_norm_quant_backward_workspace_size(M, K), dtype=torch.uint8, device="cuda")
    dy = torch.zeros(M, K, dtype=BF, device="cuda")
    dy[-3:] = rnd(3, K, seed=2, dtype=BF)
    dres = torch.empty_like(x)
    bl.bl_norm_quant_backward(dy, None, x, w, rstd, None, dres, dweight, ws)
    ok()
    assert not bool(dres[:3].any()) and not bool(dres[M // 2].any())
    Part.dresidual, Part.dx, Part.dweight = dres[-3:], None, dweight
    check_backward(dy[-3:], None, tail, w, Part)


@pytest.mark.parametrize("M,N,K", [(3, 1 << 20, 2064), (40, 1 << 20, 2064), (3000, 720000, 32), (131072, 16400, 16)])
def test_int8_linear_past_32_bit_offsets(M, N, K):
    """Weights, or outputs, of more than 2^31 elements: the last ones."""
    xq, sx, sw = codes(M, K), scales(M), scales(N, 1)
    wq = torch.zeros(N, K, dtype=torch.int8, device="cuda")
    wq[-300:] = codes(300, K, seed=2)
    y = torch.empty(M, N, dtype=BF, device="cuda")
    bl.bl_int8_linear_forward(xq, sx, wq, sw, y)
    ok()
    assert torch.equal(y[:, -300:], product(xq, sx, wq[-300:], sw[-300:], BF))
    assert not bool(y[0, :-300].any()) and not bool(y[-1, :-300].any())


def test_int8_linear_gradient_over_many_channels():
    """Above 131072 channels dX is a sum of fp32 partial sums even where it has
    tiles enough without: sampled rows."""
    M, N, K = 1200, 140000, 4096
    wq, sw, dY = codes(N, K), scales(N, 1), rnd(M, N, seed=2, dtype=BF)
    xq, sx = codes(M, K, seed=3), scales(M)
    b = bl.Int8LinearBuffers.allocate(M, N, K)
    b.workspace.fill_(255)
    bl.bl_int8_linear_backward(dY, xq, sx, wq, sw, b.dX, None, workspace=b.workspace)
    ok()
    rows = torch.tensor([0, 255, 256, 700, M - 1], device="cuda")
    w, d = (wq.float() * sw[:, None]).to(BF).double(), dY[rows].double()
    close(b.dX[rows], d @ w, (131072 / 16 + 64) * 2 * U * (d.abs() @ w.abs()), "dX")
    # the sums lose nothing to one side: the errors' mean is far below that bound
    err = (b.dX[rows].double() - d @ w) / (d.abs() @ w.abs())
    assert abs(float(err.mean())) <= 2.0 ** -12


def test_clip_past_32_bit_offsets():
    n = (1 << 31) + 12345
    g = torch.zeros(n, dtype=BF, device="cuda")
    g[-3:] = torch.tensor([3.0, 4.0, 12.0])
    g[5] = 84.0
    norm = torch.zeros(1, device="cuda")
    bl.bl_clip_grads([g], 17.0, norm, workspace(1))
    ok()
    assert float(norm) == 85.0
    assert g[-3:].tolist() == [torch.tensor(v * 0.2).to(BF).item() for v in (3.0, 4.0, 12.0)]
    assert int((g != 0).sum()) == 4


# ----------------------------------------------------------------- refusals on the device
def test_what_does_not_fit_is_refused_and_nothing_is_written():
    s = Step(9, 64, 40)
    s.wipe()
    off = torch.empty(9 * 64 + 1, dtype=BF, device="cuda")[1:].view(9, 64)
    with pytest.raises(bl.BitLinearError, match="aligned"):
        bl.bl_norm_quant_forward(off, s.r, s.w, EPS, s.n.sum, s.n.rstd, s.n.xq, s.n.sx)
    with pytest.raises(bl.BitLinearError, match="go together"):
        bl.bl_norm_quant_forward(s.x, s.r, s.w, EPS, None, s.n.rstd, s.n.xq, s.n.sx)
    with pytest.raises(bl.BitLinearError, match="fp32 x with a bf16"):
        bl.bl_norm_quant_forward(s.x.float(), s.x, s.w, EPS, s.x.clone(), s.n.rstd, s.n.xq, s.n.sx)
    with pytest.raises(ValueError, match="contiguous"):
        bl.bl_norm_quant_forward(s.x.t().contiguous().t(), s.r, s.w, EPS, s.n.sum, s.n.rstd, s.n.xq, s.n.sx)
    with pytest.raises(bl.BitLinearError, match="multiple of 8"):
        z = torch.zeros(9, 60, dtype=BF, device="cuda")
        bl.bl_norm_quant_forward(z, None, None, EPS, None, s.n.rstd, z.to(torch.int8), s.n.sx)
    with pytest.raises(ValueError, match="wq must"):
        bl.bl_int8_linear_forward(s.n.xq, s.n.sx, s.wq.float(), s.sw, s.l.y)
    with pytest.raises(bl.BitLinearError, match="multiple of 16"):
        bl.bl_int8_linear_forward(s.n.xq[:, :40].contiguous(), s.n.sx, s.wq[:, :40].contiguous(), s.sw, s.l.y)
    with pytest.raises(bl.BitLinearError, match="workspace"):
        bl.bl_int8_linear_backward(s.dY, s.n.xq, s.n.sx, s.wq, s.sw, s.l.dX, s.l.dW)
    with pytest.raises(bl.BitLinearError, match="same memory"):
        bl.bl_clip_grads([s.l.dW, s.l.dW], 1.0, s.norm, s.ws)
    with pytest.raises(ValueError, match="shape"):
        bl.bl_clip_grads([s.l.dW], 1.0, s.norm, s.ws, out=[s.l.dW.view(-1)])
    with pytest.raises(ValueError, match="bf16 or f32"):
        bl.bl_grad_norm([s.n.xq], s.norm, s.ws)
    with pytest.raises(ValueError, match="contiguous"):
        bl.bl_grad_norm([s.l.dW.t()], s.norm, s.ws)
    ok()
    assert all(bool((t == 7).all()) for t in s.outputs())


def test_lists_of_any_kind_and_a_given_stream():
    grads = tensors([1000, 7, 0, 333])
    want = check_clip([g.clone() for g in grads], 0.1)
    norm, side = torch.zeros(1, device="cuda"), torch.cuda.Stream()
    for kind in (tuple, list, iter):
        got = [g.clone() for g in grads]
        torch.cuda.synchronize()
        bl.bl_clip_grads(kind(got), 0.1, norm, workspace(4), stream=side)
        ok()
        same(got, want)
        out = [torch.empty_like(g) for g in grads]
        torch.cuda.synchronize()
        bl.bl_clip_grads(kind(grads), 0.1, norm, workspace(4), out=kind(out), stream=side)
        ok()
        same(out, want)


# ----------------------------------------------------------------- the LM's functions
@pytest.mark.parametrize("first", [False, True])
def test_norm_projections_function(first):
    """Its outputs are those of the calls it is made of; its gradients the
    formulas' in 64 bits, on the codes that the forward left."""
    M, K, Ns = 60, 96, (64, 96, 160)
    x = None if first else rnd(M, K, seed=1, dtype=BF).float().requires_grad_(True)
    r = rnd(M, K, seed=2, scale=2.0).requires_grad_(True)
    gain = (1 + rnd(K, seed=3, scale=0.2)).requires_grad_(True)
    ws = [rnd(n, K, seed=4 + n, scale=0.1).requires_grad_(True) for n in Ns]
    stream, *ys = plm.NormProjectionsFunction.apply(x, r, gain, EPS, *ws)
    b = bl.NormQuantBuffers.allocate(M, K, BF, F32, F32, backward=False)
    total = r.detach() if first else x.detach() + r.detach()
    bl.bl_norm_quant_forward(total, None, gain.detach(), EPS, None, b.rstd, b.xq, b.sx)
    ok()
    assert torch.equal(stream.detach(), total)
    dsum = rnd(M, K, seed=20)
    dys = [rnd(M, n, seed=21 + n, dtype=BF).float() for n in Ns]
    dy, dysize = torch.zeros(M, K, dtype=torch.float64, device="cuda"), 0.0
    wants = []
    for w, y, g in zip(ws, ys, dys):
        N = w.shape[0]
        s = bl.StepBuffers.allocate(M, N, K, F32)
        bl.bl_quantize_weight(w.detach(), s.w_packed, s.gamma, s.workspace)
        bl.bl_forward(b.xq, b.sx, s.w_packed, s.gamma, s.y)
        bl.bl_backward(g.to(BF), b.xq, b.sx, s.w_packed, s.gamma, s.dX, s.dW)
        ok()
        assert torch.equal(y.detach(), s.y.float())
        wants.append(s.dW)
        dy += s.dX.double()
        dysize = dysize + s.dX.double().abs()
    leaves = [*([] if first else [x]), r, gain, *ws]
    grads = torch.autograd.grad([stream, *ys], leaves, [dsum, *dys])
    ok()
    same(grads[-len(ws):], wants)
    d, size, dg, dgsize = gradients(dy, dsum, total, gain.detach())
    # dy is a sum of three bf16 numbers in fp32: two roundings on top
    extra = 4 * U * dysize.amax() * float(size.amax() / dy.abs().amax().clamp(min=1e-9) + 10)
    at = 0 if first else 1
    close(grads[at], d, 90 * U * size + extra, "residual")
    close(grads[at + 1], dg, (30 + 16 + 148) * U * dgsize + 4 * U * (dysize * (total.double().abs() * b.rstd.double()[:, None])).sum(0), "gain")
    if not first:
        # rounded to bf16, as the projection behind it takes its gradient
        close(grads[0].to(BF), d, 90 * U * size + extra, "x")
        assert torch.equal(grads[0], grads[0].to(BF).float())


def test_norm_head8_function():
    M, K, V = 50, 64, 104
    x, r = rnd(M, K, seed=1, dtype=BF).float().requires_grad_(True), rnd(M, K, seed=2).requires_grad_(True)
    gain, head = (1 + rnd(K, seed=3, scale=0.2)).requires_grad_(True), rnd(V, K, seed=4, scale=0.1).requires_grad_(True)
    logits = plm.NormHead8Function.apply(x, r, gain, EPS, head)
    total = (x + r).detach()
    wide = [t.detach().double().requires_grad_(True) for t in (x, r, gain, head)]
    s = wide[0] + wide[1]
    y = s / torch.sqrt((s * s).mean(-1, keepdim=True) + EPS) * wide[2]
    want = y @ wide[3].t()
    # either operand is off by half a step of 8 bits, absmax / 254, in each of K
    # products; the head's rows by a rounding to bf16 too
    ya, ha = y.detach().abs(), head.detach().double().abs()
    tol = (ya.amax(1, keepdim=True) / 254) @ ha.sum(1)[None, :] + ya.sum(1)[:, None] @ (ha.amax(1)[None, :] / 254) + K * (
        ya.amax(1, keepdim=True) @ ha.amax(1)[None, :]) / 254 ** 2 + 2.0 ** -8 * (ya @ ha.t())
    assert bool(((logits.detach().double() - want.detach()).abs() <= 1.05 * tol).all())
    g = rnd(M, V, seed=6, dtype=BF).float()
    got = torch.autograd.grad(logits, [x, r, gain, head], g)
    ok()
    # straight through: the gradients of the product of the values, then the norm's
    hb = head.detach().to(BF)
    a = hb.float().abs().amax(1, keepdim=True).clamp(min=1e-5)
    w_hat = (torch.round(hb.float() * (127 / a)) * (a / 127)).to(BF).double()
    dy = g.double() @ w_hat
    dysize = g.double().abs() @ w_hat.abs()
    d, size, dg, dgsize = gradients(dy, None, total, gain.detach())
    step = 2.0 ** -8 * dysize.amax() * 1.5     # dX in bf16, and a code of w_hat next to a tie is in dysize
    assert bool(((got[1].double() - d).abs() <= 0.01 * size + step * 1e-1 + 1e-6).all())
    assert float((got[1].double() - d).norm()) <= 2.0 ** -7 * float(d.norm())
    assert float((got[2].double() - dg).norm()) <= 2.0 ** -7 * float(dg.norm())
    assert torch.equal(got[0], got[1].to(BF).float())
    # dW from x_hat: within half a step of 8 bits of y, and bf16 roundings
    dw = g.double().t() @ y.detach()
    bound = g.double().abs().t() @ (ya.amax(1, keepdim=True) / 254 + 2.0 ** -8 * ya)
    assert bool(((got[3].double() - dw).abs() <= 1.05 * bound).all())


@pytest.mark.parametrize("how", [dict(fused_norms=True), dict(head8=True), dict(fused_norms=True, head8=True)])
def test_model_runs_and_its_gradients_come_through(how):
    """The tiny model with a random head: loss and gradients near those of the
    library's separate calls. A value quantised from fp32 instead of bf16 moves by
    at most one step of 8 bits (1 / 127 of the largest) beyond the rounding; 8-bit
    heads by half a step in each operand: a few percent of a tensor's norm."""
    init = lm_init(LM_TINY, seed=2)
    init["head"] = torch.randn(init["head"].shape, generator=torch.Generator().manual_seed(3)) * 0.05
    ids = lm_batches(LM_TINY, seed=3)[0].cuda()
    out = []
    for kw in ({}, how):
        params = {n: t.cuda().requires_grad_(True) for n, t in init.items()}
        loss = plm.lm_loss(params, ids, LM_TINY, library_ops=True, **kw)
        out.append((loss.detach(), torch.autograd.grad(loss, list(params.values()))))
    ok()
    assert all(bool(g.isfinite().all()) and bool(g.any()) for g in out[1][1])
    assert abs(float(out[0][0]) - float(out[1][0])) <= 0.05 * float(out[0][0])


def test_training_with_everything_runs_and_repeats():
    init, ids = lm_init(LM_TINY, seed=0), lm_batches(LM_TINY, seed=0)
    runs = [plm.train_lm(init, ids, LM_TINY, torch.device("cuda"), steps=3, dtype=F32, library_ops=True, fused_norms=True,
                         head8=True, max_norm=0.5) for _ in range(2)]
    assert runs[0] == runs[1] and all(math.isfinite(x) for x in runs[0])
    # a zero head: every probability is 1 / V
    assert abs(runs[0][0] - math.log(LM_TINY.vocab)) <= 16 * 2.0 ** -23 * math.log(LM_TINY.vocab)


def test_clip_of_many_tensors_in_a_graph():
    """A list of more tensors than one launch takes, captured and replayed."""
    grads = tensors([37] * 1500)
    norm, ws = torch.zeros(1, device="cuda"), workspace(len(grads))
    out = [torch.empty_like(g) for g in grads]
    bl.bl_clip_grads(grads, 0.5, norm, ws, out=out)
    ok()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bl.bl_clip_grads(grads, 0.5, norm, ws, out=out)
    for t in grads:
        t.mul_(3)
    g.replay()
    ok()
    want = norm64(grads)
    assert abs(float(norm) - want) <= 7 * U * want
    for t, o in zip(grads, out):
        close(o, t.double() * 0.5 / want, 9 * U * t.double().abs() * 0.5 / want, "clipped")


def test_clip_gradients_copies_what_is_not_dense_or_shared():
    a = rnd(40, 30)
    shared, strided = a, rnd(30, 40, seed=1).t()
    keep = a.clone()
    got, norm = plm.clip_gradients([a, shared, strided], 1.0)
    ok()
    total = norm64([keep, keep, strided])
    assert abs(float(norm) - total) <= 7 * U * total
    for g, src in zip(got, (keep, keep, strided)):
        close(g, src.double() / total, 9 * U * src.double().abs() / total, "clipped")


def test_model_arguments_are_refused():
    params = {n: t.cuda() for n, t in lm_init(LM_TINY, seed=2).items()}
    ids = lm_batches(LM_TINY, seed=3)[0].cuda()
    for kw in (dict(fused_norms=True), dict(head8=True), dict(library_ops=True, saved8=True, fused_norms=True)):
        with pytest.raises(ValueError, match="fused_norms and head8"):
            plm.lm_loss(params, ids, LM_TINY, **kw)
    with pytest.raises(ValueError, match="max_norm"):
        plm.train_lm(lm_init(LM_TINY, seed=0), ids[None], LM_TINY, torch.device("cuda"), steps=1, max_norm=1.0)
