"""A small decoder LM whose projections are BitLinear layers run by the library.

"bitnet-qat-train" (Measured behavior, Training) trains a 4-layer transformer
LM with the layer. Here the attention q, k, v, o and the SwiGLU gate, up,
down projections of every block go through the C ABI: the forward quantises
the fp32 master and the bf16 activations (``bl_quantize``) and runs the INT8
GEMM (``bl_forward``), keeping only the 2-bit codes, gamma, the INT8
activations and their scales; the backward rebuilds the operands from that
state (``bl_backward``: dX in bf16, dW in fp32). The pages give no other part
of the model; embedding, RMSNorm, attention, the SwiGLU gating, the LM head,
the cross-entropy and AdamW are plain PyTorch on the GPU, outside the
library, in the precision ``dtype`` (fp64 by default, the precision the LM
oracle keeps them in, so that a comparison of the two isolates the library's
calls; fp32 for a faster run):

  pre-norm blocks  h += o(attn(norm(h))); h += down(silu(gate(m)) * up(m)),
                   m = norm(h); RMSNorm x / sqrt(mean(x^2) + eps) * g
  attention        causal softmax, `heads` heads, no positional encoding
  loss             mean next-token cross-entropy
  AdamW            decoupled decay on the 2-D weights, not on the norm gains

Around each BitLinear call the model rounds as the calls require: its input
and its output gradient to bf16 (one rounding, straight from ``dtype``), the
master to fp32; y and dX come back in bf16 and dW in fp32. The embedding is a
one-hot product, so its gradient is a plain matrix product (the same sums on
every run) rather than an atomic scatter.

With ``library_ops`` (dtype fp32) the library also runs what lies between the
projections: the norms (``bl_norm_forward`` / ``bl_norm_backward``, whose
inputs are kept in 8 bits with ``saved8``), the SwiGLU gating
(``bl_swiglu_forward`` / ``bl_swiglu_backward``: gate and up are kept in 8 bits
for the backward, not in fp32) and the LM head with the cross-entropy
(``bl_linear_xent_forward`` / ``bl_linear_xent_backward``: no logits). The head
then takes the last norm's output and its weights in bf16, and a target outside
the vocabulary leaves its token out of the mean. (In the middle of a sequence it is
also the next token's id, which then embeds as zeros.)

With ``fused_norms`` too, what lies between two blocks' projections is one pass
(``bl_norm_quant_forward`` / ``bl_norm_quant_backward``): the last projection's
output is added to the residual stream, the sum normed, and the norm's result
quantised once for all projections that read it (q, k and v; gate and up). The
norm's result is then not rounded to bf16 in front of the quantiser. ``head8``
runs the head on 8-bit codes of the last norm's output and of the head's rows
(``bl_int8_linear_forward`` / ``bl_int8_linear_backward``, straight-through
gradients); its logits go through torch's cross-entropy, under the same rule for
targets outside the vocabulary. ``train_lm`` scales the gradients down to
``max_norm`` over all parameters (``bl_clip_grads``).
"""

from __future__ import annotations

import bisect
import math

import torch
from torch.autograd.function import once_differentiable

from . import bitlinear as b

__all__ = ["BitLinearFunction", "RMSNormFunction", "SwigluFunction", "HeadLossFunction", "NormProjectionsFunction",
           "NormHead8Function", "to_bf16_rn", "lm_loss", "clip_gradients", "adamw_step", "train_lm"]

_BF16_MIN_NORMAL = 2.0 ** -126


def to_bf16_rn(x: torch.Tensor) -> torch.Tensor:
    """Round a float64 (or float32) tensor to bf16 once, to nearest with ties to
    even. (A float64 -> bf16 cast through float32 rounds twice, which differs
    when the float32 value lands on a bf16 tie.) Finite inputs.

    Normal range: the float64 bit pattern is rounded at the 8th significant
    bit with an integer add of half a unit (less one, plus the kept lowest
    bit: ties go to even) and a mask; the result is exactly a bf16 value, so
    the cast that follows is exact. Below 2^-126 the bf16 quantum is 2^-133:
    the value is rounded on that grid with round-half-even.
    """
    if x.dtype == torch.float32:
        return x.to(torch.bfloat16)  # float32 -> bf16 is one rounding already
    x = x.to(torch.float64).contiguous()
    bits = x.view(torch.int64)
    keep = (bits >> 45) & 1
    rounded = ((bits + ((1 << 44) - 1) + keep) & ~((1 << 45) - 1)).view(torch.float64)
    tiny = torch.round(x * 2.0 ** 133) * 2.0 ** -133
    y = torch.where(x.abs() < _BF16_MIN_NORMAL, tiny, rounded)
    return y.to(torch.bfloat16)


class BitLinearFunction(torch.autograd.Function):
    """y [M, N] = BitLinear(x [M, K], W [N, K] master), in the dtype of x."""

    @staticmethod
    def forward(ctx, x2d, w):
        M, K = x2d.shape
        N = w.shape[0]
        dev = x2d.device
        xb = to_bf16_rn(x2d).contiguous()
        w32 = w.detach().to(torch.float32).contiguous()
        packed = torch.empty((N, K // 4), dtype=torch.uint8, device=dev)
        gamma = torch.empty(1, dtype=torch.float32, device=dev)
        ws = torch.empty(max(b.bl_quantize_weight_workspace_size(N, K), 16), dtype=torch.uint8, device=dev)
        xq = torch.empty((M, K), dtype=torch.int8, device=dev)
        sx = torch.empty(M, dtype=torch.float32, device=dev)
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        b.bl_quantize(w32, xb, packed, gamma, xq, sx, ws)
        b.bl_forward(xq, sx, packed, gamma, y)
        ctx.save_for_backward(xq, sx, packed, gamma)
        ctx.out_dtype = x2d.dtype
        ctx.w_dtype = w.dtype
        return y.to(x2d.dtype)

    @staticmethod
    def backward(ctx, gy):
        xq, sx, packed, gamma = ctx.saved_tensors
        M, K = xq.shape
        N = packed.shape[0]
        dy = to_bf16_rn(gy).contiguous()
        dX = torch.empty((M, K), dtype=torch.bfloat16, device=dy.device)
        dW = torch.empty((N, K), dtype=torch.float32, device=dy.device)
        b.bl_backward(dy, xq, sx, packed, gamma, dX, dW)
        return dX.to(ctx.out_dtype), dW.to(ctx.w_dtype)


def _operand(t: torch.Tensor) -> torch.Tensor:
    """t as the training operators take it: contiguous and on a 16-byte
    boundary. A view may start anywhere in its storage (the targets of a batch
    of one sequence are its ids from the second on)."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class RMSNormFunction(torch.autograd.Function):
    """y [M, K] = RMS norm of x [M, K] with gain weight [K]; x is kept for the
    backward as it is, or (saved8) in 8 bits."""

    @staticmethod
    def forward(ctx, x, weight, eps, saved8):
        M, K = x.shape
        x, weight = _operand(x), _operand(weight)
        y = torch.empty_like(x)
        rstd = torch.empty(M, dtype=torch.float32, device=x.device)
        keep = b.Act8.allocate(M, K, x.device) if saved8 else None
        b.bl_norm_forward(x, weight, None, eps, y, None, rstd, rms=True, saved8=keep)
        ctx.saved8 = saved8
        ctx.save_for_backward(weight, rstd, *((keep.codes, keep.scales) if saved8 else (x,)))
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        weight, rstd, *kept = ctx.saved_tensors
        x = b.Act8(*kept) if ctx.saved8 else kept[0]
        gy = _operand(gy)
        dx, dweight = torch.empty_like(gy), torch.empty_like(weight)
        ws = torch.empty(max(b.bl_norm_backward_workspace_size(*gy.shape), 16), dtype=torch.uint8, device=gy.device)
        b.bl_norm_backward(gy, x, weight, None, rstd, dx, dweight, None, ws, rms=True)
        return dx, dweight, None, None


class SwigluFunction(torch.autograd.Function):
    """y [M, K] = silu(gate) * up in bf16 (the type the BitLinear calls around
    it give and take), returned in the dtype of gate; gate and up are kept for
    the backward in 8 bits."""

    @staticmethod
    def forward(ctx, gate, up):
        g, u = _operand(gate.to(torch.bfloat16)), _operand(up.to(torch.bfloat16))
        y = torch.empty_like(g)
        g8, u8 = b.Act8.allocate(*g.shape, g.device), b.Act8.allocate(*g.shape, g.device)
        b.bl_swiglu_forward(g, u, y, g8, u8)
        ctx.save_for_backward(g8.codes, g8.scales, u8.codes, u8.scales)
        return y.to(gate.dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        gc, gs, uc, us = ctx.saved_tensors
        dy = _operand(gy.to(torch.bfloat16))
        dgate, dup = torch.empty_like(dy), torch.empty_like(dy)
        b.bl_swiglu_backward(dy, b.Act8(gc, gs), b.Act8(uc, us), dgate, dup)
        return dgate.to(gy.dtype), dup.to(gy.dtype)


class HeadLossFunction(torch.autograd.Function):
    """Mean cross-entropy of h [M, K] . head [V, K]^T at targets [M] over the
    tokens whose target lies in the vocabulary (0 if there is none)."""

    @staticmethod
    def forward(ctx, h, head, targets):
        (M, K), V = h.shape, head.shape[0]
        hb, wb = _operand(h.to(torch.bfloat16)), _operand(head.to(torch.bfloat16))
        targets = _operand(targets)
        buf = b.XentBuffers.allocate(M, V, K, backward=False, device=h.device)
        b.bl_linear_xent_forward(hb, wb, targets, buf.loss, buf.lse, buf.workspace)
        share = ((targets >= 0) & (targets < V)).sum().clamp(min=1).to(torch.float32).reciprocal()
        ctx.save_for_backward(hb, wb, targets, buf.lse, share)
        ctx.dtypes = h.dtype, head.dtype
        return (buf.loss.sum() * share).to(h.dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        h, head, targets, lse, share = ctx.saved_tensors
        (M, K), V = h.shape, head.shape[0]
        dloss = (g.to(torch.float32) * share).expand(M).contiguous()
        dH = torch.empty_like(h) if ctx.needs_input_grad[0] else None
        dW = torch.empty((V, K), dtype=torch.float32, device=h.device) if ctx.needs_input_grad[1] else None
        ws = torch.empty(max(b.bl_linear_xent_backward_workspace_size(M, V, K, torch.float32), 16), dtype=torch.uint8,
                         device=h.device)
        b.bl_linear_xent_backward(h, head, targets, lse, dloss, dH, dW, ws)
        return (None if dH is None else dH.to(ctx.dtypes[0])), (None if dW is None else dW.to(ctx.dtypes[1])), None


def _normed(x, residual, gain, eps):
    """The stream x + residual [M, K] (fp32; x, in bf16, may be None), 1 / rms,
    and the 8-bit form of its norm."""
    M, K = residual.shape
    stream, gain = _operand(residual), _operand(gain)
    buf = b.NormQuantBuffers.allocate(M, K, torch.bfloat16, torch.float32, gain.dtype, backward=False, device=gain.device)
    if x is None:
        b.bl_norm_quant_forward(stream, None, gain, eps, None, buf.rstd, buf.xq, buf.sx)
        buf.sum = stream
    else:
        b.bl_norm_quant_forward(_operand(x.to(torch.bfloat16)), stream, gain, eps, buf.sum, buf.rstd, buf.xq, buf.sx)
    return gain, buf


def _norm_gradients(dy, dsum, stream, gain, rstd, x_dtype):
    """Gradients of x (None where there is none), of the residual and of the gain."""
    dresidual, dgain = torch.empty_like(stream), torch.empty_like(gain)
    dx = None if x_dtype is None else torch.empty(stream.shape, dtype=torch.bfloat16, device=stream.device)
    ws = torch.empty(max(b.bl_norm_quant_backward_workspace_size(*stream.shape), 16), dtype=torch.uint8, device=stream.device)
    b.bl_norm_quant_backward(dy, None if dsum is None else _operand(dsum), stream, gain, rstd, dx, dresidual, dgain, ws)
    return (None if dx is None else dx.to(x_dtype)), dresidual, dgain


class NormProjectionsFunction(torch.autograd.Function):
    """(stream, y_1, ..., y_n): the stream x + residual [M, K] (fp32; x, the last
    projection's output, in bf16 precision, or None: the stream is the residual),
    and BitLinear of its RMS norm, quantised once, with each of the masters
    weights [N_i, K]."""

    @staticmethod
    def forward(ctx, x, residual, gain, eps, *weights):
        M, K = residual.shape
        dev = residual.device
        gain, buf = _normed(x, residual, gain, eps)
        saved, outs = [], []
        for w in weights:
            N = w.shape[0]
            w32 = _operand(w.detach().to(torch.float32))
            packed = torch.empty((N, K // 4), dtype=torch.uint8, device=dev)
            gamma = torch.empty(1, dtype=torch.float32, device=dev)
            ws = torch.empty(max(b.bl_quantize_weight_workspace_size(N, K), 16), dtype=torch.uint8, device=dev)
            y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
            b.bl_quantize_weight(w32, packed, gamma, ws)
            b.bl_forward(buf.xq, buf.sx, packed, gamma, y)
            saved += [packed, gamma]
            outs.append(y.to(residual.dtype))
        stream = buf.sum if x is not None else residual.clone()
        ctx.save_for_backward(buf.sum, gain, buf.rstd, buf.xq, buf.sx, *saved)
        ctx.x_dtype = None if x is None else x.dtype
        ctx.w_dtypes = [w.dtype for w in weights]
        return (stream, *outs)

    @staticmethod
    @once_differentiable
    def backward(ctx, dsum, *dys):
        stream, gain, rstd, xq, sx, *saved = ctx.saved_tensors
        M, K = xq.shape
        dy, dws = None, []
        for g, packed, gamma, dt in zip(dys, saved[::2], saved[1::2], ctx.w_dtypes):
            N = packed.shape[0]
            dX = torch.empty((M, K), dtype=torch.bfloat16, device=g.device)
            dW = torch.empty((N, K), dtype=torch.float32, device=g.device)
            ws = torch.empty(max(b.bl_backward_workspace_size(M, N, K), 16), dtype=torch.uint8, device=g.device)
            b.bl_backward(_operand(to_bf16_rn(g)), xq, sx, packed, gamma, dX, dW, workspace=ws)
            dy = dX.float() if dy is None else dy.add_(dX)
            dws.append(dW.to(dt))
        return (*_norm_gradients(dy, dsum, stream, gain, rstd, ctx.x_dtype), None, *dws)


class NormHead8Function(torch.autograd.Function):
    """Logits [M, V] (fp32) of a head [V, K] kept in 8 bits per row, from the RMS
    norm of the stream x + residual (as in NormProjectionsFunction) in 8 bits per
    token. The gradients' call takes a multiple of 8 channels: rows of zeros fill
    the head's codes up to that."""

    @staticmethod
    def forward(ctx, x, residual, gain, eps, head):
        (M, K), V = residual.shape, head.shape[0]
        gain, buf = _normed(x, residual, gain, eps)
        wq = torch.empty((-(-V // 8) * 8, K), dtype=torch.int8, device=head.device)
        sw = torch.empty(wq.shape[0], dtype=torch.float32, device=head.device)
        b.bl_quantize_act(_operand(head.detach().to(torch.bfloat16)), wq[:V], sw[:V])
        if len(wq) > V:
            wq[V:] = 0
            sw[V:] = 0
        logits = torch.empty((M, V), dtype=torch.float32, device=head.device)
        b.bl_int8_linear_forward(buf.xq, buf.sx, wq[:V], sw[:V], logits)
        ctx.save_for_backward(buf.sum, gain, buf.rstd, buf.xq, buf.sx, wq, sw)
        ctx.x_dtype = None if x is None else x.dtype
        ctx.w_dtype = head.dtype
        return logits

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        stream, gain, rstd, xq, sx, wq, sw = ctx.saved_tensors
        (M, K), V, V8 = xq.shape, g.shape[1], wq.shape[0]
        dX = torch.empty((M, K), dtype=torch.bfloat16, device=g.device)
        dW = torch.empty((V8, K), dtype=torch.float32, device=g.device)
        ws = torch.empty(max(b.bl_int8_linear_backward_workspace_size(M, V8, K), 16), dtype=torch.uint8, device=g.device)
        dY = g.to(torch.bfloat16)
        if V8 > V:
            dY = torch.nn.functional.pad(dY, (0, V8 - V))
        b.bl_int8_linear_backward(_operand(dY), xq, sx, wq, sw, dX, dW, workspace=ws)
        return (*_norm_gradients(dX, None, stream, gain, rstd, ctx.x_dtype), None, dW[:V].to(ctx.w_dtype))


def _left_out(targets, vocab):
    """targets with those outside the vocabulary as the one that the cross-entropy ignores."""
    return torch.where((targets >= 0) & (targets < vocab), targets, -100)


def _mean_loss(logits, targets):
    """Mean cross-entropy of logits [M, V] at targets [M], as HeadLossFunction's."""
    targets = _left_out(targets, logits.shape[1])
    total = torch.nn.functional.cross_entropy(logits, targets, ignore_index=-100, reduction="sum")
    return total / (targets >= 0).sum().clamp(min=1)


def _rmsnorm(x, g, eps):
    return x / torch.sqrt(torch.mean(x * x, dim=-1, keepdim=True) + eps) * g


def lm_loss(params: dict, ids: torch.Tensor, cfg, library_ops: bool = False, saved8: bool = False,
            fused_norms: bool = False, head8: bool = False) -> torch.Tensor:
    """Mean next-token cross-entropy of ids [B, S + 1] (parameters of one float
    dtype; fp32 with library_ops: the norms, the gating and the head's loss by
    the library, the norms' inputs kept in 8 bits with saved8). fused_norms, head8
    (with library_ops, without saved8): the module's docstring."""
    if library_ops and params["embed"].dtype != torch.float32:
        raise ValueError(f"library_ops takes fp32 parameters, got {params['embed'].dtype}")
    if (fused_norms or head8) and (not library_ops or saved8):
        raise ValueError("fused_norms and head8 go with library_ops and without saved8")

    def norm(x, g):
        if library_ops:
            return RMSNormFunction.apply(x.reshape(-1, d), g, cfg.norm_eps, saved8)
        return _rmsnorm(x, g, cfg.norm_eps).reshape(-1, d)

    def gated(gate, up):
        return SwigluFunction.apply(gate, up) if library_ops else torch.nn.functional.silu(gate) * up

    B, S1 = ids.shape
    S, d, H = S1 - 1, cfg.d, cfg.heads
    dh = d // H
    x_ids, y_ids = ids[:, :S], ids[:, 1:]
    embed = params["embed"]
    # an id outside the vocabulary (a padded batch: its targets are left out) embeds as zeros
    one_hot = (x_ids.reshape(-1, 1) == torch.arange(embed.shape[0], device=ids.device)).to(embed.dtype)
    h = (one_hot @ embed).reshape(B, S, d)
    causal = torch.ones(S, S, dtype=torch.bool, device=ids.device).tril()
    bl = BitLinearFunction.apply
    pending = None  # the last projection's output, still to be added to h (fused_norms)

    def normed_projections(gain, weights):
        """h with what is pending added, and the projections of its norm."""
        if fused_norms:
            stream, *ys = NormProjectionsFunction.apply(pending, h.reshape(-1, d), gain, cfg.norm_eps, *weights)
            return stream.reshape(B, S, d), ys
        a = norm(h, gain)
        return h, [bl(a, w) for w in weights]

    for i in range(cfg.layers):
        def p(n):
            return params[f"layer{i}.{n}"]
        h, qkv = normed_projections(p("attn_norm"), [p(n) for n in ("q", "k", "v")])
        q, k, v = (y.reshape(B, S, H, dh).transpose(1, 2) for y in qkv)
        scores = (q @ k.transpose(-1, -2)) / math.sqrt(dh)
        scores = scores.masked_fill(~causal, float("-inf"))
        o = (torch.softmax(scores, dim=-1) @ v).transpose(1, 2).reshape(B * S, d)
        pending = bl(o, p("o"))
        if not fused_norms:
            h = h + pending.reshape(B, S, d)
        h, (gate, up) = normed_projections(p("mlp_norm"), [p("gate"), p("up")])
        pending = bl(gated(gate, up), p("down"))
        if not fused_norms:
            h = h + pending.reshape(B, S, d)
    if head8:
        logits = NormHead8Function.apply(pending if fused_norms else None, h.reshape(-1, d), params["final_norm"],
                                         cfg.norm_eps, params["head"])
        return _mean_loss(logits, y_ids.reshape(-1))
    if fused_norms:
        h = h + pending.reshape(B, S, d)
    last = norm(h, params["final_norm"])
    if library_ops:
        return HeadLossFunction.apply(last, params["head"], y_ids.reshape(-1))
    return torch.nn.functional.cross_entropy(last @ params["head"].T, _left_out(y_ids.reshape(-1), params["head"].shape[0]))


def clip_gradients(grads, max_norm: float):
    """The gradients (tensors, bf16 or fp32), scaled down in place to a norm over
    all of them of max_norm at most, and that norm [1] before. A gradient that is
    not contiguous, or that shares memory with one before it (autograd may hand
    one tensor to two leaves), is replaced by a copy."""
    if not grads:
        raise ValueError("no gradients")
    out, begins, ends = [], [], []  # and the memory of those so far, by address
    for g in grads:
        g = g.contiguous()
        if g.numel():
            begin = g.data_ptr()
            i = bisect.bisect_right(ends, begin)
            if i < len(begins) and begins[i] < begin + g.numel() * g.element_size():
                g = g.clone()
                begin = g.data_ptr()
                i = bisect.bisect_right(ends, begin)
            begins.insert(i, begin)
            ends.insert(i, begin + g.numel() * g.element_size())
        out.append(g)
    norm = torch.empty(1, dtype=torch.float32, device=out[0].device)
    ws = torch.empty(max(b.bl_grad_norm_workspace_size(len(out)), 16), dtype=torch.uint8, device=norm.device)
    b.bl_clip_grads(out, max_norm, norm, ws)
    return out, norm


def adamw_step(params: dict, grads: dict, state: dict, step: int, cfg):
    """One AdamW step in place (step counts from 1); no decay on norm gains."""
    b1, b2 = cfg.beta1, cfg.beta2
    bc1, bc2 = 1.0 - b1 ** step, 1.0 - b2 ** step
    with torch.no_grad():
        for name, p in params.items():
            g = grads[name]
            m, v = state.setdefault(name, (torch.zeros_like(p), torch.zeros_like(p)))
            m.mul_(b1).add_(g, alpha=1.0 - b1)
            v.mul_(b2).addcmul_(g, g, value=1.0 - b2)
            if not name.endswith("norm"):
                p.mul_(1.0 - cfg.lr * cfg.weight_decay)
            p.sub_(cfg.lr * (m / bc1) / (torch.sqrt(v / bc2) + cfg.eps))


def train_lm(init: dict, batches: torch.Tensor, cfg, device, steps: int | None = None, timing: bool = False,
             dtype=torch.float64, library_ops: bool = False, saved8: bool = False, fused_norms: bool = False,
             head8: bool = False, max_norm: float | None = None):
    """Losses of `steps` AdamW steps from `init` on `batches` (token ids), with
    everything outside the BitLinear calls in ``dtype``; with ``timing``, also
    the mean device time per step in ms (CUDA events, first step excluded).
    library_ops, saved8, fused_norms, head8: as lm_loss (with dtype fp32). max_norm
    (dtype fp32): the gradients' norm over all parameters is cut to it before AdamW."""
    if max_norm is not None and dtype != torch.float32:
        raise ValueError(f"max_norm takes fp32 gradients, got {dtype}")
    params = {n: t.to(device=device, dtype=dtype).contiguous().requires_grad_(True) for n, t in init.items()}
    ids_all = batches.to(device)
    state: dict = {}
    losses, times = [], []
    for t in range(steps if steps is not None else batches.shape[0]):
        if timing:
            s, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            s.record()
        loss = lm_loss(params, ids_all[t], cfg, library_ops, saved8, fused_norms, head8)
        grads = torch.autograd.grad(loss, list(params.values()))
        if max_norm is not None:
            grads, _ = clip_gradients(grads, max_norm)
        adamw_step(params, dict(zip(params.keys(), grads)), state, t + 1, cfg)
        if timing:
            e.record()
        losses.append(loss.detach())
        if timing:
            torch.cuda.synchronize(device)
            times.append(s.elapsed_time(e))
    if b.bl_get_last_error() != 0:
        raise RuntimeError("device error word set")
    out = [float(x) for x in losses]
    return (out, sum(times[1:]) / max(len(times) - 1, 1)) if timing else out
