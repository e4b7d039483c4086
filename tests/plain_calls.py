"""Plain stand-ins, on the CPU, for the library's calls that the decoder LM makes:
each from its formula, in 64 bits, rounded once to the type that the call writes.
For tests of the code around the calls."""

import torch

from ternary_weight_quantization_b200 import bitlinear as b

_PLACES = torch.tensor([0, 2, 4, 6])


def _out(to, value):
    to.copy_(value.to(to.dtype))


def _quantised(y):
    a = y.abs().amax(1, keepdim=True).clamp(min=1e-5)
    return torch.round(y * (127.0 / a)), (a / 127.0)[:, 0]


def _value(code, scale):
    return (code.float() * scale.float()[:, None]).to(torch.bfloat16).double()


def quantize_weight(w, packed, gamma, workspace):
    g = w.double().abs().mean()
    code = torch.round(w.double() / g.clamp(min=1e-5)).clamp(-1, 1).long() + 1
    packed.copy_((code.view(w.shape[0], -1, 4) << _PLACES).sum(-1))
    gamma.fill_(float(g))


def _ternary(packed, gamma):
    return (((packed.long()[..., None] >> _PLACES) & 3) - 1).reshape(packed.shape[0], -1).double() * float(gamma)


def quantize_act(x, xq, sx):
    q, s = _quantised(x.double())
    _out(xq, q)
    _out(sx, s)


def quantize(w, x, packed, gamma, xq, sx, workspace):
    quantize_weight(w, packed, gamma, workspace)
    quantize_act(x, xq, sx)


def forward(xq, sx, packed, gamma, y):
    _out(y, (xq.double() * sx.double()[:, None]) @ _ternary(packed, gamma).t())


def backward(dY, xq, sx, packed, gamma, dX, dW, workspace=None):
    _out(dX, dY.double() @ _ternary(packed, gamma))
    _out(dW, dY.double().t() @ _value(xq, sx))


def _norm_back(dy, x, weight, rstd):
    n = x.double() * rstd.double()[:, None]
    g = dy.double() * weight.double()
    return rstd.double()[:, None] * (g - n * (g * n).mean(1, keepdim=True)), (dy.double() * n).sum(0)


def norm_forward(x, weight, bias, eps, y, mean, rstd, rms, saved8=None):
    assert rms and bias is None and saved8 is None
    _out(rstd, torch.rsqrt(x.double().square().mean(1) + eps))
    _out(y, x.double() * rstd.double()[:, None] * weight.double())


def norm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, workspace, rms):
    d, dw = _norm_back(dy, x, weight, rstd)
    _out(dx, d)
    _out(dweight, dw)


def norm_quant_forward(x, residual, weight, eps, sum, rstd, xq, sx):
    assert (residual is None) == (sum is None)
    total = x
    if residual is not None:
        _out(sum, x.double() + residual.double())
        total = sum
    _out(rstd, torch.rsqrt(total.double().square().mean(1) + eps))
    quantize_act(total.double() * rstd.double()[:, None] * weight.double(), xq, sx)


def norm_quant_backward(dy, dsum, sum, weight, rstd, dx, dresidual, dweight, workspace):
    d, dw = _norm_back(dy, sum, weight, rstd)
    d = d if dsum is None else d + dsum.double()
    for to, v in ((dx, d), (dresidual, d), (dweight, dw)):
        if to is not None:
            _out(to, v)


def int8_linear_forward(xq, sx, wq, sw, y):
    _out(y, (xq.double() @ wq.double().t()) * (sx.double()[:, None] * sw.double()))


def int8_linear_backward(dY, xq, sx, wq, sw, dX, dW, workspace):
    assert dY.shape == (xq.shape[0], wq.shape[0]) and dY.shape[1] % 8 == 0 and dY.dtype == torch.bfloat16
    _out(dX, dY.double() @ _value(wq, sw))
    _out(dW, dY.double().t() @ _value(xq, sx))


def linear_xent_forward(h, W, targets, loss, lse, workspace):
    z = h.double() @ W.double().t()
    _out(lse, torch.logsumexp(z, 1))
    held = (targets >= 0) & (targets < W.shape[0])
    at = z.gather(1, targets.where(held, torch.zeros_like(targets))[:, None])[:, 0]
    _out(loss, (torch.logsumexp(z, 1) - at) * held)


def linear_xent_backward(h, W, targets, lse, dloss, dH, dW, workspace):
    z = h.double() @ W.double().t()
    held = (targets >= 0) & (targets < W.shape[0])
    dz = torch.exp(z - lse.double()[:, None])
    dz[held.nonzero()[:, 0], targets[held]] -= 1.0
    dz = dz * (dloss.double() * held)[:, None]
    for to, v in ((dH, dz @ W.double()), (dW, dz.t() @ h.double())):
        if to is not None:
            _out(to, v)


def install(monkeypatch):
    """Puts the stand-ins in the calls' places, and the gating in plain autograd."""
    from ternary_weight_quantization_b200 import lm
    for name in ("quantize_weight", "quantize_act", "quantize", "forward", "backward", "norm_forward", "norm_backward",
                 "norm_quant_forward", "norm_quant_backward", "int8_linear_forward", "int8_linear_backward",
                 "linear_xent_forward", "linear_xent_backward"):
        monkeypatch.setattr(b, "bl_" + name, globals()[name])
    monkeypatch.setattr(lm.SwigluFunction, "apply", staticmethod(lambda g, u: torch.nn.functional.silu(g) * u))
