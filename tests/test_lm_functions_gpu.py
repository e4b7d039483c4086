"""GPU: the LM's autograd functions over the training operators, one by one and
together, against 64-bit forms that round where the operators round.

U = 2^-24 is half a step of fp32 relative to the value, HB = 2^-8 the most by
which one rounding to bf16 is off."""

import json
import math
import os

import pytest
import torch

import ternary_weight_quantization_b200 as bl
from tests.conftest import GOLDEN
from tests.test_rows_gpu import saved_values
from ternary_weight_quantization_b200 import lm as plm
from workloads.lm import LM_CONFIG, LM_TINY, lm_batches, lm_init

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HB = 2.0 ** -8
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-6


def rnd(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda") * scale


def bf(x):
    """x (fp64 or fp32) rounded once to bf16, in fp64."""
    return plm.to_bf16_rn(x).double()


def saved(x):
    return saved_values(x)[2].double()


def ok():
    torch.cuda.synchronize()
    assert bl.bl_get_last_error() == 0


# ----------------------------------------------------------------- the functions in 64 bits
class Norm64(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, eps, saved8):
        r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        ctx.save_for_backward(saved(x.float()) if saved8 else x, r, w)
        return x * r * w

    @staticmethod
    def backward(ctx, dy):
        x, r, w = ctx.saved_tensors
        xh, g = x * r, dy * w
        return r * (g - xh * (g * xh).mean(-1, keepdim=True)), (dy * xh).sum(0), None, None


class Gate64(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, up):
        g, u = plm.to_bf16_rn(gate), plm.to_bf16_rn(up)
        ctx.save_for_backward(saved(g), saved(u))
        g, u = g.double(), u.double()
        return bf(g * torch.sigmoid(g) * u)

    @staticmethod
    def backward(ctx, dy):
        g, u = ctx.saved_tensors
        dy, s = bf(dy), torch.sigmoid(g)
        return bf(dy * u * s * (1 + g * (1 - s))), bf(dy * g * s)


class Head64(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, w, t):
        h, w = bf(h), bf(w)
        z = h @ w.t()
        live = (t >= 0) & (t < w.shape[0])
        lse = torch.logsumexp(z, 1)
        at = torch.where(live, t, 0)[:, None]
        dz = torch.exp(z - lse[:, None]).scatter_add(1, at, torch.full_like(lse, -1.0)[:, None])
        n = max(int(live.sum()), 1)
        ctx.save_for_backward(h, w, torch.where(live[:, None], dz, 0.0))
        ctx.n = n
        return torch.where(live, lse - z.gather(1, at)[:, 0], 0.0).sum() / n

    @staticmethod
    def backward(ctx, g):
        h, w, dz = ctx.saved_tensors
        f = g / ctx.n
        # dz goes to dH in bf16 relative to the largest dloss, to an fp32 dW in
        # two bf16 terms (2^-17)
        return bf(f * (bf(dz) @ w)), f * (dz.t() @ h), None


# ----------------------------------------------------------------- one by one
@pytest.mark.parametrize("saved8", [False, True])
@pytest.mark.parametrize("M,K", [(1, 8), (7, 40), (33, 512), (5, 1001), (130, 264)])
def test_rms_norm_function(M, K, saved8):
    x, w, dy = rnd(M, K, seed=1, scale=2.0), 1 + 0.2 * rnd(K, seed=2), rnd(M, K, seed=3)
    a, b = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    p, q = x.double().requires_grad_(True), w.double().requires_grad_(True)
    y, want = plm.RMSNormFunction.apply(a, b, EPS, saved8), Norm64.apply(p, q, EPS, saved8)
    dx, dw = torch.autograd.grad(y, [a, b], dy)
    dx64, dw64 = torch.autograd.grad(want, [p, q], dy.double())
    ok()
    # additions a value goes through in a row's sum (32 in a thread, 5 in the
    # warp, 32 over warps) and the products around it: of rstd's variance, of
    # c2's terms; for dweight the rows of a block and their joining
    n = 100
    assert bool(((y.double() - want).abs() <= n * U * want.abs()).all())
    xs = saved(x) if saved8 else x.double()
    r = 1 / torch.sqrt((x.double() ** 2).mean(1, keepdim=True) + EPS)
    g, xh = dy.double() * w.double(), xs * r
    terms = r * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    assert bool(((dx.double() - dx64).abs() <= 3 * n * U * terms).all())
    assert bool(((dw.double() - dw64).abs() <= (3 * n + M) * U * (dy.double() * xh).abs().sum(0)).all())


@pytest.mark.parametrize("M,K", [(1, 8), (7, 40), (33, 1408), (5, 1001)])
def test_swiglu_function(M, K):
    gate, up, dy = rnd(M, K, seed=1, scale=3.0), rnd(M, K, seed=2), rnd(M, K, seed=3)
    a, b = gate.clone().requires_grad_(True), up.clone().requires_grad_(True)
    p, q = gate.double().requires_grad_(True), up.double().requires_grad_(True)
    y, want = plm.SwigluFunction.apply(a, b), Gate64.apply(p, q)
    assert y.dtype == F32
    dg, du = torch.autograd.grad(y, [a, b], dy)
    dg64, du64 = torch.autograd.grad(want, [p, q], dy.double())
    ok()
    # both sides are rounded to bf16: at most one step (2^-7) apart where the
    # fp32 value lies across a tie, and equal nearly everywhere else. dgate's
    # 1 + g (1 - s) cancels: its fp32 error counts on the terms
    for got, ref, terms in ((y, want, 0), (du, du64, 0),
                            (dg, dg64, (dy.double() * saved(up.to(BF))).abs() * (1 + saved(gate.to(BF)).abs()))):
        err = (got.double() - ref).abs()
        assert bool((err <= 2.0 ** -7 * ref.abs() + 128 * U * terms).all())
        assert int((err > 0).sum()) <= 0.02 * err.numel() + 2


@pytest.mark.parametrize("M,V,K", [(1, 100, 8), (5, 700, 64), (40, 300, 136), (300, 1000, 512)])
def test_head_loss_function(M, V, K):
    h, w = rnd(M, K, seed=1), rnd(V, K, seed=2, scale=K ** -0.5)
    t = torch.randint(0, V, (M,), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    t[1::3] = -100
    a, b = h.clone().requires_grad_(True), w.clone().requires_grad_(True)
    p, q = h.double().requires_grad_(True), w.double().requires_grad_(True)
    got, want = plm.HeadLossFunction.apply(a, b, t), Head64.apply(p, q, t)
    dh, dw = torch.autograd.grad(3.0 * got, [a, b])
    dh64, dw64 = torch.autograd.grad(3.0 * want, [p, q])
    ok()
    hd, wd = bf(h), bf(w)
    # a tensor-core sum drops up to a step of fp32 (2 U) per 16 terms
    ez = (K / 16 + 4) * 2 * U * float((hd.abs() @ wd.abs().t()).amax())
    assert abs(float(got.detach()) - float(want.detach())) <= 2 * ez + 64 * U * (1 + math.log(V))
    dz = torch.softmax(hd @ wd.t(), 1)
    dz[torch.arange(M, device="cuda"), t.clamp(min=0)] -= 1
    live = (t >= 0)[:, None]
    dz = torch.where(live, dz.abs() * 3.0 / int(live.sum()), 0.0)
    # p's relative error; dz in two bf16 terms; the sums; dH: dz and dH are
    # rounded to bf16 on both sides, each at most a step apart
    e = 2 * (2 * ez + 64 * U * (1 + math.log(V)))
    assert bool(((dw.double() - dw64).abs() <= (2.0 ** -16 + e + (M / 8 + 64) * 2 * U) * (dz.t() @ hd.abs()) + 1e-30).all())
    mag = dz @ wd.abs()
    assert bool(((dh.double() - dh64).abs() <= (2.0 ** -7 + e + (V / 16 + 64) * 2 * U) * mag + 2.0 ** -7 * dh64.abs() + 1e-30).all())
    assert float((dh.double() - dh64).norm()) <= (HB + e) * float(dh64.norm()) + 1e-30
    assert not dh[1::3].any()


# ----------------------------------------------------------------- together
def model64(params, ids, cfg, saved8):
    """The LM with plain products for its BitLinear layers, in fp64, with the
    operators' roundings."""
    B, S, d, H = ids.shape[0], ids.shape[1] - 1, cfg.d, cfg.heads
    h = params["embed"][ids[:, :S]]
    causal = torch.ones(S, S, dtype=torch.bool, device=ids.device).tril()
    for i in range(cfg.layers):
        p = lambda n: params[f"layer{i}.{n}"]   # noqa: E731
        a = Norm64.apply(h.reshape(B * S, d), p("attn_norm"), cfg.norm_eps, saved8)
        q, k, v = ((a @ p(n).T).reshape(B, S, H, d // H).transpose(1, 2) for n in ("q", "k", "v"))
        scores = (q @ k.transpose(-1, -2) / math.sqrt(d // H)).masked_fill(~causal, float("-inf"))
        o = (torch.softmax(scores, -1) @ v).transpose(1, 2).reshape(B * S, d)
        h = h + (o @ p("o").T).reshape(B, S, d)
        m = Norm64.apply(h.reshape(B * S, d), p("mlp_norm"), cfg.norm_eps, saved8)
        h = h + (Gate64.apply(m @ p("gate").T, m @ p("up").T) @ p("down").T).reshape(B, S, d)
    return Head64.apply(Norm64.apply(h.reshape(B * S, d), params["final_norm"], cfg.norm_eps, saved8), params["head"],
                        ids[:, 1:].reshape(-1))


@pytest.mark.parametrize("saved8", [False, True])
def test_model_gradients_against_the_same_roundings_in_fp64(monkeypatch, saved8):
    """Loss and gradients of the whole model. Both sides round at the same
    places, so they part only where an fp32 error (about 1e-6 of the value)
    carries a value across a tie: about 1 in 2000 values of a bf16 tensor, by a
    step of 2^-8 to 2^-7 (in the norm 2e-4), and 1 in 5000 of an 8-bit one by a
    step of 1/127 of the group's largest value, about 3 % of its spread (4e-4).
    A gradient's way has about 25 such tensors: 2e-3 in squares. The bound is four
    times that."""
    monkeypatch.setattr(plm.BitLinearFunction, "apply", staticmethod(lambda x, w: x @ w.T))
    cfg = LM_TINY
    init = lm_init(cfg, seed=2)
    init["head"] = torch.randn(init["head"].shape, generator=torch.Generator().manual_seed(3)) * 0.05
    ids = lm_batches(cfg, seed=3)[0].cuda()
    p32, p64 = ({n: t.to(device="cuda", dtype=dt).requires_grad_(True) for n, t in init.items()} for dt in (F32, F64))
    got, want = plm.lm_loss(p32, ids, cfg, library_ops=True, saved8=saved8), model64(p64, ids, cfg, saved8)
    assert abs(float(got.detach()) - float(want.detach())) <= 2.0 ** -12 * float(want.detach())
    for name, a, b in zip(p64, torch.autograd.grad(got, list(p32.values())), torch.autograd.grad(want, list(p64.values()))):
        assert float(b.norm()) > 0 and float((a.double() - b).norm()) <= 2.0 ** -7 * float(b.norm()), name
    ok()


@pytest.mark.parametrize("saved8", [False, True])
def test_lm_with_library_operators_tracks_the_stored_oracle_curve(saved8):
    """The bar of the LM trained through the library (0.01 over 50 steps) for its
    configuration with the library's operators. The run repeats bit for bit, and
    the gap (0.0096 with saved8, 0.0093 without) is that of an fp32 run: a
    last-bit difference turns a quantiser's code. The same model in fp32 with
    none of the operators parts by 0.0117."""
    with open(os.path.join(GOLDEN, "lm_oracle_losses.json")) as f:
        gold = json.load(f)["losses"]
    cfg = LM_CONFIG
    losses = plm.train_lm(lm_init(cfg, seed=0), lm_batches(cfg, seed=0), cfg, torch.device("cuda"), dtype=F32,
                          library_ops=True, saved8=saved8)
    diffs = [abs(a - b) for a, b in zip(losses, gold)]
    assert len(diffs) == cfg.steps and max(diffs) <= 0.01, (max(diffs), diffs.index(max(diffs)))
    ok()
