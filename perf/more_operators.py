"""Operators around 8-bit products, and the gradients' norm: what is measured, and their plain forms.

Three operators that a decoder LM with quantised layers runs next to the
ternary projections:

  norm    the residual's addition, RMS norm and the 8-bit form of its result
          (one scale per token), which is what the products take; forward
          alone (serving), or forward and backward with the gradients of the
          projection's output, of the residual stream and of the gain
  linear  the product of two 8-bit integer operands with a scale per token and
          per output channel; forward alone (serving, from one token), or
          forward and the straight-through gradients of both operands
  clip    the norm over all of a model's gradients, and the gradients scaled
          down to a largest norm

``run`` computes them in elementary torch operations in 32 bits; with ``own``
set it calls the framework's operators. Sizes are the repository's own: the
4-layer LM (2048 tokens, width 512, SwiGLU width 1408, vocabulary 8192) and
the 2560 / 6912 layers over 2048 and 4096 tokens, with generic vocabularies.
"""

import math

import torch

own = False

EPS = 1e-6         # of the norm
FLOOR = 1e-5       # least absmax of a token's 8-bit form
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token on its way into a layer of width 2560: launch latency
        {"name": "norm_serve_1_2560", "op": "norm", "M": 1, "K": 2560, "x": "bf16", "s": "bf16", "p": "bf16", "train": False},
        # the small LM's step: projections in bf16, residual stream in fp32
        {"name": "norm_train_2048_512", "op": "norm", "M": 2048, "K": 512, "x": "bf16", "s": "f32", "p": "f32", "train": True},
        # a layer of width 2560, 8 sequences of 512 tokens
        {"name": "norm_train_4096_2560", "op": "norm", "M": 4096, "K": 2560, "x": "bf16", "s": "bf16", "p": "bf16", "train": True},
        # an odd number of tokens, a width that fills no warp evenly, all in fp32
        {"name": "norm_train_777_1000_f32", "op": "norm", "M": 777, "K": 1000, "x": "f32", "s": "f32", "p": "f32", "train": True},
        # one decoded token through the up projection
        {"name": "linear_1_2560_6912", "op": "linear", "M": 1, "K": 2560, "N": 6912, "y": "bf16", "train": False},
        # the logits of 16 sequences that are decoded together, in fp32
        {"name": "linear_16_2560_32000_f32", "op": "linear", "M": 16, "K": 2560, "N": 32000, "y": "f32", "train": False},
        # a short prompt, odd sizes
        {"name": "linear_333_1040_5001", "op": "linear", "M": 333, "K": 1040, "N": 5001, "y": "bf16", "train": False},
        # the up projection of a long prompt
        {"name": "linear_4096_2560_6912", "op": "linear", "M": 4096, "K": 2560, "N": 6912, "y": "bf16", "train": False},
        # a training step of an 8-bit up projection
        {"name": "linear_train_4096_2560_6912", "op": "linear", "M": 4096, "K": 2560, "N": 6912, "y": "bf16", "train": True},
        # the small LM's gradients
        {"name": "clip_lm_4_512", "op": "clip", "layers": 4, "d": 512, "ffn": 1408, "vocab": 8192, "g": "f32", "packed": False, "most": 1.0},
        # six blocks of width 2560 with a vocabulary of 32000, gradients in bf16
        {"name": "clip_lm_6_2560", "op": "clip", "layers": 6, "d": 2560, "ffn": 6912, "vocab": 32000, "g": "bf16", "packed": False, "most": 1.0},
        # odd widths in one packed buffer: tensors that start at any element
        {"name": "clip_packed_3_333", "op": "clip", "layers": 3, "d": 333, "ffn": 901, "vocab": 1021, "g": "bf16", "packed": True, "most": 1.0},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "linear", "linear", "clip"])
    if op == "norm":
        while True:
            M, K = spread(1, 8192), 8 * spread(8, 1024)
            if M * K <= 4096 * 6912:
                break
        x, s = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        return {"op": op, "M": M, "K": K, "x": x, "s": s, "p": rng.choice(["bf16", "f32"]), "train": rng.random() < 0.6}
    if op == "linear":
        train = rng.random() < 0.4
        while True:
            M, K, N = spread(1, 8192), 16 * spread(4, 432), spread(64, 32000)
            if train:
                N = 8 * (N // 8)
            if M * K * N <= 4096 * 2560 * 6912:
                break
        return {"op": op, "M": M, "K": K, "N": N, "y": rng.choice(["bf16", "f32"]), "train": train}
    while True:
        case = {"op": op, "layers": rng.randint(1, 8), "d": spread(32, 2560), "ffn": spread(64, 6912),
                "vocab": spread(128, 32000), "g": rng.choice(["bf16", "f32"]), "packed": rng.random() < 0.4,
                "most": rng.choice([1.0, 1.0, 1e6])}
        if work(case)["bytes"] <= 2.6e9:
            return case


def shapes(case):
    """Shapes of a model's gradients: embedding, per block two gains and seven projections, last gain, head."""
    d, f, v = case["d"], case["ffn"], case["vocab"]
    block = [(d,), (d,)] + [(d, d)] * 4 + [(f, d)] * 2 + [(d, f)]
    return [(v, d)] + block * case["layers"] + [(d,), (v, d)]


def work(case):
    if case["op"] == "clip":
        e = 2 if case["g"] == "bf16" else 4
        n = sum(math.prod(s) * (e if len(s) == 2 else 4) for s in shapes(case))
        return {"bytes": 2 * n + 4, "flops": 3 * sum(map(math.prod, shapes(case)))}
    M, K = case["M"], case["K"]
    if case["op"] == "linear":
        N = case["N"]
        e = 2 if case["y"] == "bf16" else 4
        n = M * K + N * K + 4 * (M + N) + e * M * N
        flops = 2 * M * N * K
        if case["train"]:
            n += 2 * M * N + 2 * M * K + 2 * N * K           # dY; dX, dW
            flops *= 3
        return {"bytes": n, "flops": flops}
    x, s, p = (2 if case[k] == "bf16" else 4 for k in "xsp")
    n = M * K * (x + 2 * s + 1) + 8 * M + K * p              # x, residual -> sum, codes; scale, 1 / rms
    if case["train"]:
        # dy (bf16), the sum's gradient, the sum -> gradients of the residual and of x
        n += M * K * (2 + 2 * s + (s + x if x != s else s)) + 4 * M + 2 * K * p
    return {"bytes": n, "flops": (20 if case["train"] else 8) * M * K}


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = {"case": dict(case)}
    if case["op"] == "clip":
        # tensors side by side in one buffer per type, each on a 128-byte line of its own unless packed
        for name, dt, rank in (("matrices", DTYPES[case["g"]], 2), ("gains", torch.float32, 1)):
            sizes = [math.prod(t) for t in shapes(case) if len(t) == rank]
            steps = sizes if case["packed"] else [-(-n // 64) * 64 for n in sizes]
            flat = torch.zeros(sum(steps), device="cuda", dtype=dt)
            at, spans = 0, []
            for n, step in zip(sizes, steps):
                # tensors of a model differ in size by orders of magnitude
                size = 10.0 ** (-2.0 - 2.0 * torch.rand((), generator=gen, device="cuda"))
                flat[at:at + n] = (randn(n) * size).to(dt)
                spans.append((at, n))
                at += step
            out = torch.zeros_like(flat)
            s[name], s[name + "_out"] = flat, out
            s[name + "_list"] = [flat[a:a + n] for a, n in spans]
            s[name + "_outs"] = [out[a:a + n] for a, n in spans]
        if own:
            import ternary_weight_quantization_b200 as bl
            s["norm"] = torch.empty(1, device="cuda")
            n = bl.bl_grad_norm_workspace_size(len(shapes(case)))
            s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        return s
    M, K = case["M"], case["K"]
    if case["op"] == "linear":
        N = case["N"]
        # a few features much larger than the others
        x = randn(M, K) * (1.0 + 15.0 * (torch.rand(K, generator=gen, device="cuda") < 0.01))
        w = randn(N, K) * 0.02 * (0.5 + torch.rand(N, 1, generator=gen, device="cuda"))
        for code, scale, v in (("xq", "sx", x), ("wq", "sw", w)):
            a = v.abs().amax(dim=1, keepdim=True)
            s[code], s[scale] = torch.round(v * (127.0 / a)).to(torch.int8), (a / 127.0)[:, 0].contiguous()
        if case["train"]:
            s["dY"] = (randn(M, N) * 0.1).to(torch.bfloat16)
        if own:
            import ternary_weight_quantization_b200 as bl
            s["b"] = bl.Int8LinearBuffers.allocate(M, N, K, DTYPES[case["y"]], backward=case["train"])
        return s
    dx, ds, dp = (DTYPES[case[k]] for k in "xsp")
    s["x"] = randn(M, K).to(dx)
    # a residual stream: a few features much larger than the others
    s["residual"] = (randn(M, K) * (1.0 + 4.0 * (torch.rand(K, generator=gen, device="cuda") < 0.02)) + 0.25 * randn(K)).to(ds)
    s["weight"] = (1.0 + 0.2 * randn(K)).to(dp)
    if case["train"]:
        s["dy"] = (randn(M, K) * 0.1).to(torch.bfloat16)
        s["dsum"] = (randn(M, K) * 0.1).to(ds)
    if own:
        import ternary_weight_quantization_b200 as bl
        s["b"] = bl.NormQuantBuffers.allocate(M, K, dx, ds, dp, backward=case["train"])
        s["x_hat"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    return s


# ----------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    return {"norm": _norm, "linear": _linear, "clip": _clip}[case["op"]](s, case)


def _own(s, case):
    import ternary_weight_quantization_b200 as bl
    op = case["op"]
    if op == "clip":
        bl.bl_clip_grads(s["matrices_list"] + s["gains_list"], case["most"], s["norm"], s["workspace"],
                         out=s["matrices_outs"] + s["gains_outs"])
        return {"norm": s["norm"], "matrices": s["matrices_out"], "gains": s["gains_out"]}
    b = s["b"]
    if op == "linear":
        bl.bl_int8_linear_forward(s["xq"], s["sx"], s["wq"], s["sw"], b.y)
        if not case["train"]:
            return {"y": b.y}
        bl.bl_int8_linear_backward(s["dY"], s["xq"], s["sx"], s["wq"], s["sw"], b.dX, b.dW, workspace=b.workspace)
        return {"y": b.y, "dX": b.dX, "dW": b.dW}
    bl.bl_norm_quant_forward(s["x"], s["residual"], s["weight"], EPS, b.sum, b.rstd, b.xq, b.sx)
    # the values that the codes stand for
    out = {"sum": b.sum, "rstd": b.rstd, "sx": b.sx, "x_hat": torch.mul(b.xq, b.sx[:, None], out=s["x_hat"])}
    if case["train"]:
        bl.bl_norm_quant_backward(s["dy"], s["dsum"], b.sum, s["weight"], b.rstd, b.dx, b.dresidual, b.dweight, b.workspace)
        out.update(dresidual=b.dresidual, dweight=b.dweight)
        if case["x"] != case["s"]:
            out["dx"] = b.dx
    return out


# ----------------------------------------------------------------- plain forms (32 bits)

def _norm(s, case):
    total = s["x"].float() + s["residual"].float()
    total = total.to(s["residual"].dtype)          # the stream is kept in its own type
    r, w = total.float(), s["weight"].float()
    rstd = 1.0 / torch.sqrt((r * r).mean(dim=1, keepdim=True) + EPS)
    y = r * rstd * w
    a = y.abs().amax(dim=1, keepdim=True).clamp(min=FLOOR)
    codes, sx = torch.round(y * (127.0 / a)), a / 127.0
    out = {"sum": total, "rstd": rstd[:, 0], "sx": sx[:, 0], "x_hat": (codes * sx).to(torch.bfloat16)}
    if case["train"]:
        # the quantiser's Jacobian is taken as 1
        dy, n = s["dy"].float(), r * rstd
        g = dy * w
        d = s["dsum"].float() + rstd * (g - n * (g * n).mean(dim=1, keepdim=True))
        out.update(dresidual=d.to(total.dtype), dweight=(dy * n).sum(dim=0).to(s["weight"].dtype))
        if case["x"] != case["s"]:
            out["dx"] = d.to(s["x"].dtype)
    return out


def _linear(s, case):
    y = (s["xq"].float() @ s["wq"].float().t()) * (s["sx"][:, None] * s["sw"][None, :])
    out = {"y": y.to(DTYPES[case["y"]])}
    if case["train"]:
        # the operands' values in bf16, as the layers' products take them
        x_hat = (s["xq"].float() * s["sx"][:, None]).to(torch.bfloat16).float()
        w_hat = (s["wq"].float() * s["sw"][:, None]).to(torch.bfloat16).float()
        dY = s["dY"].float()
        out["dX"], out["dW"] = (dY @ w_hat).to(torch.bfloat16), (dY.t() @ x_hat).to(torch.bfloat16)
    return out


def _clip(s, case):
    both = s["matrices_list"] + s["gains_list"]
    total = torch.stack([g.float().square().sum(dtype=torch.float64) for g in both]).sum()
    norm = torch.sqrt(total)
    scale = torch.where(norm > case["most"], case["most"] / norm, 1.0).float()
    for g, out in zip(both, s["matrices_outs"] + s["gains_outs"]):
        out.copy_(g.float() * scale)
    return {"norm": norm.float().reshape(1), "matrices": s["matrices_out"], "gains": s["gains_out"]}


# ----------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        flat = torch.cat([s["matrices"].double(), s["gains"].double()])
        norm = torch.linalg.vector_norm(flat)
        factor = min(1.0, case["most"] / max(float(norm), 1e-300))
        return {"norm": norm.reshape(1), "matrices": s["matrices"].double() * factor, "gains": s["gains"].double() * factor}
    if case["op"] == "linear":
        xv = s["xq"].double() * s["sx"].double()[:, None]
        wv = s["wq"].double() * s["sw"].double()[:, None]
        out = {"y": torch.einsum("mk,nk->mn", xv, wv)}
        if case["train"]:
            # the gradients are defined on operands that were rounded to bf16 once: a product
            # of 8 and 24 bits has at most 32 and passes through fp32 only as its sum does
            xb, wb = _bf16(s["xq"], s["sx"]), _bf16(s["wq"], s["sw"])
            dY = s["dY"].double()
            out["dX"], out["dW"] = torch.einsum("mn,nk->mk", dY, wb), torch.einsum("mn,mk->nk", dY, xb)
        return out
    # the sum in the stream's type is an output, and what follows is defined on it
    total = s["x"].double() + s["residual"].double()
    kept = total.float().to(s["residual"].dtype).double()
    w = s["weight"].double()
    scale = torch.rsqrt(kept.pow(2).mean(1) + EPS)
    unit = kept * scale[:, None]
    y = unit * w
    top = torch.linalg.vector_norm(y, float("inf"), dim=1).clamp(min=FLOOR)
    value = torch.round(y / top[:, None] * 127) * (top[:, None] / 127)
    out = {"sum": total, "rstd": scale, "sx": top / 127, "x_hat": value}
    if case["train"]:
        g = s["dy"].double() * w
        along = (g * unit).sum(1, keepdim=True) / case["K"] * unit
        d = (g - along) * scale[:, None] + s["dsum"].double()
        out.update(dresidual=d, dweight=torch.einsum("mk,mk->k", s["dy"].double(), unit))
        if case["x"] != case["s"]:
            out["dx"] = d
    return out


def _bf16(codes, scales):
    """A code's value as the layers define it: fp32(code * scale), rounded to bf16."""
    return (codes.double() * scales.double()[:, None]).float().bfloat16().double()
