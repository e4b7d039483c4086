"""GPU: the training operators used together -- the decoder LM with its norms,
gating and head loss by the library, and one block's calls captured in a CUDA
graph -- against the same model in fp64."""

import math

import pytest
import torch

import ternary_weight_quantization_b200 as bl
from ternary_weight_quantization_b200 import lm as plm
from workloads.lm import LM_CONFIG, LM_TINY, lm_batches, lm_init

pytestmark = pytest.mark.gpu


def _params(cfg, seed, dtype):
    init = lm_init(cfg, seed=seed)
    init["head"] = torch.randn(init["head"].shape, generator=torch.Generator().manual_seed(seed + 1)) * 0.05
    return {n: t.to(device="cuda", dtype=dtype).requires_grad_(True) for n, t in init.items()}


@pytest.mark.parametrize("saved8", [False, True])
def test_model_gradients_against_fp64(monkeypatch, saved8):
    """With plain products in the place of the BitLinear layers (whose
    quantisers would turn a last-bit difference into another code), loss and
    gradients of the model with the library's operators against fp64 autograd.

    Relative to a tensor's norm, a bf16 rounding is off by at most 2^-8 and a
    value kept in 8 bits by half a step, absmax / 254 of its group of 128: at
    absmax = 4 standard deviations 1.6 % of the group's norm at most. A block
    has 3 bf16 roundings and 2 to 4 such tensors (gate, up, with saved8 the
    norms' inputs) on a gradient's way, the head 3 roundings; 2 blocks."""
    monkeypatch.setattr(plm.BitLinearFunction, "apply", staticmethod(lambda x, w: x @ w.T))
    cfg = LM_TINY
    ids = lm_batches(cfg, seed=3)[0].cuda()
    p64, p32 = _params(cfg, 2, torch.float64), _params(cfg, 2, torch.float32)
    want = plm.lm_loss(p64, ids, cfg)
    got = plm.lm_loss(p32, ids, cfg, library_ops=True, saved8=saved8)
    # the forward keeps fp32 or rounds to bf16: 3 roundings a block and 2 at the head
    assert abs(float(got.detach()) - float(want.detach())) <= (2 * 3 + 2) * 2.0 ** -8 * float(want.detach())
    bound = 2 * (3 * 2.0 ** -8 + (4 if saved8 else 2) * 0.016) + 3 * 2.0 ** -8
    for name, a, b in zip(p64, torch.autograd.grad(want, list(p64.values())), torch.autograd.grad(got, list(p32.values()))):
        assert float((a - b.double()).norm()) <= bound * float(a.norm()), name
    assert bl.bl_get_last_error() == 0


def test_left_out_targets_and_a_head_without_tokens():
    h = torch.randn(20, 64, device="cuda", requires_grad=True)
    w = torch.randn(100, 64, device="cuda", requires_grad=True)
    t = torch.randint(0, 100, (20,), device="cuda")
    t[::2] = -100
    loss = plm.HeadLossFunction.apply(h, w, t)
    want = torch.nn.functional.cross_entropy(h.bfloat16().double() @ w.bfloat16().double().T, t)
    # fp32 sums of 64 exact products, of 100 exponentials and of 10 losses
    assert abs(float(loss.detach()) - float(want.detach())) <= 64 * 2.0 ** -23 * (float(want.detach()) + float((h.abs() @ w.abs().T).max().detach()))
    dh, dw = torch.autograd.grad(loss, [h, w])
    assert not dh[::2].any() and bool(dh[1::2].any()) and bool(dw.isfinite().all())
    none = plm.HeadLossFunction.apply(h, w, torch.full_like(t, -1))
    assert float(none.detach()) == 0.0
    assert all(not g.any() for g in torch.autograd.grad(none, [h, w]))


@pytest.mark.parametrize("saved8", [False, True])
def test_training_runs_and_repeats(saved8):
    cfg = LM_CONFIG
    init, ids = lm_init(cfg, seed=0), lm_batches(cfg, seed=0)
    runs = [plm.train_lm(init, ids, cfg, torch.device("cuda"), steps=3, dtype=torch.float32, library_ops=True,
                         saved8=saved8) for _ in range(2)]
    assert runs[0] == runs[1] and all(math.isfinite(x) for x in runs[0])
    # a zero head: every probability is 1 / V
    assert abs(runs[0][0] - math.log(cfg.vocab)) <= 16 * 2.0 ** -23 * math.log(cfg.vocab)


def test_fp64_parameters_are_refused():
    p = _params(LM_TINY, 2, torch.float64)
    with pytest.raises(ValueError, match="fp32"):
        plm.lm_loss(p, lm_batches(LM_TINY, seed=3)[0].cuda(), LM_TINY, library_ops=True)


def test_one_block_captured_and_replayed():
    """Norm, gate and head loss, forward and backward, in one CUDA graph: a
    replay on new inputs gives what the calls give."""
    M, K, V = 300, 512, 1000
    bf = torch.bfloat16

    def make(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
        return dict(x=r(M, K).to(bf), up=r(M, K).to(bf), w=r(K), bias=r(K), W=(r(V, K) * 0.05).to(bf),
                    t=torch.randint(-1, V, (M,), generator=g, device="cuda"), dl=torch.rand(M, generator=g, device="cuda"))
    n = bl.NormBuffers.allocate(M, K, bf, torch.float32, bias=True, saved8=True)
    s = bl.SwigluBuffers.allocate(M, K, bf)
    e = bl.XentBuffers.allocate(M, V, K)

    def block(i):
        bl.bl_norm_forward(i["x"], i["w"], i["bias"], 1e-6, n.y, n.mean, n.rstd, saved8=n.saved8)
        bl.bl_swiglu_forward(n.y, i["up"], s.y, s.gate8, s.up8)
        bl.bl_linear_xent_forward(s.y, i["W"], i["t"], e.loss, e.lse, e.workspace)
        bl.bl_linear_xent_backward(s.y, i["W"], i["t"], e.lse, i["dl"], e.dH, e.dW, e.workspace)
        bl.bl_swiglu_backward(e.dH, s.gate8, s.up8, s.dgate, s.dup)
        bl.bl_norm_backward(s.dgate, n.saved8, i["w"], n.mean, n.rstd, n.dx, n.dweight, n.dbias, n.workspace)

    def outputs():
        torch.cuda.synchronize()
        return [t.clone() for t in (n.y, s.y, e.loss, e.lse, e.dH, e.dW, s.dgate, s.dup, n.dx, n.dweight, n.dbias)]
    inputs = make(1)
    block(inputs)
    first = outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        block(inputs)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(outputs(), first))
    other = make(2)
    for k, v in other.items():
        inputs[k].copy_(v)
    graph.replay()
    replayed = outputs()
    block(other)
    assert all(torch.equal(a, b) for a, b in zip(outputs(), replayed))
    assert not torch.equal(replayed[4], first[4]) and bl.bl_get_last_error() == 0
