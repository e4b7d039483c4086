"""Training operators next to the BitLinear layer: what is measured, and their plain forms.

Four operators that a decoder LM trained with BitLinear layers runs outside
the ternary projections:

  xent    the LM head and its softmax cross-entropy over a large vocabulary,
          without keeping the logits: forward alone (evaluation), or forward
          and both gradients (training)
  norm    layer norm or RMS norm, forward and backward with the gradients of
          its gain and bias; the backward reads the saved input, or its 8-bit
          checkpoint
  swiglu  silu(gate) * up, whose backward reads 8-bit checkpoints of gate and
          up
  act8    an activation saved in 8 bits (one scale per 128 values of a row)
          and read back

``run`` computes them in elementary torch operations in 32 bits; with ``own``
set it calls the framework's operators. Sizes are the repository's own: the
4-layer LM (2048 tokens, width 512, SwiGLU width 1408, vocabulary 8192) and
the 2560 / 6912 layers over 2048 and 4096 tokens, with generic vocabularies.
"""

import math

import torch

own = False

GROUP = 128        # values of a row that share one scale of the 8-bit form
EPS = 1e-6         # of the norms
FLOOR = 1e-30      # least absmax of a group of the 8-bit form
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------- cases

def listed():
    return [
        # the loss of one decoded token under the small LM: launch latency
        {"name": "xent_eval_1_512_8192", "op": "xent", "M": 1, "K": 512, "V": 8192, "train": False, "left_out": 0.0, "dw": "bf16"},
        # perplexity of 2048 tokens over a large vocabulary
        {"name": "xent_eval_2048_2560_131072", "op": "xent", "M": 2048, "K": 2560, "V": 131072, "train": False, "left_out": 0.0, "dw": "bf16"},
        # the training step of the small LM (8 sequences of 256 tokens)
        {"name": "xent_train_2048_512_8192", "op": "xent", "M": 2048, "K": 512, "V": 8192, "train": True, "left_out": 0.0, "dw": "bf16"},
        # the training step of a model of width 2560, 8 sequences of 512 tokens
        {"name": "xent_train_4096_2560_32000", "op": "xent", "M": 4096, "K": 2560, "V": 32000, "train": True, "left_out": 0.0, "dw": "bf16"},
        # a padded batch of odd sizes, the head's gradient in fp32
        {"name": "xent_train_ragged_f32", "op": "xent", "M": 777, "K": 1000, "V": 50001, "train": True, "left_out": 0.3, "dw": "f32"},
        # the small LM's norm over its fp32 residual stream
        {"name": "norm_rms_f32_2048_512", "op": "norm", "M": 2048, "K": 512, "x": "f32", "p": "f32", "rms": True, "bias": False, "saved8": False},
        # layer norm of a layer of width 2560 with its input saved in 8 bits
        {"name": "norm_saved8_bf16_4096_2560", "op": "norm", "M": 4096, "K": 2560, "x": "bf16", "p": "bf16", "rms": False, "bias": False, "saved8": True},
        # odd sizes, gain and bias
        {"name": "norm_odd_f32_333_1001", "op": "norm", "M": 333, "K": 1001, "x": "f32", "p": "f32", "rms": False, "bias": True, "saved8": False},
        # the gate of the small LM's blocks
        {"name": "swiglu_bf16_2048_1408", "op": "swiglu", "M": 2048, "K": 1408, "x": "bf16"},
        # the gate of a block with 6912 hidden features
        {"name": "swiglu_bf16_4096_6912", "op": "swiglu", "M": 4096, "K": 6912, "x": "bf16"},
        # a layer's input saved and read back
        {"name": "act8_bf16_4096_6912", "op": "act8", "M": 4096, "K": 6912, "x": "bf16"},
        # odd sizes: rows that start anywhere, a last group of 5 values
        {"name": "act8_odd_f32_1021_2565", "op": "act8", "M": 1021, "K": 2565, "x": "f32"},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["xent", "xent", "norm", "swiglu", "act8"])
    if op == "xent":
        while True:
            M, K, V = spread(1, 4096), 8 * spread(8, 512), spread(1000, 131072)
            if 6 * M * K * V <= 2.0e12 and M * V <= 2048 * 131072:
                break
        return {"op": op, "M": M, "K": K, "V": V, "train": rng.random() < 0.7,
                "left_out": rng.choice([0.0, 0.1, 0.5]), "dw": rng.choice(["bf16", "f32"])}
    M, K = spread(1, 4096), spread(16, 6912)
    if rng.random() < 0.6:
        K = max(8, K // 8 * 8)
    case = {"op": op, "M": M, "K": K, "x": rng.choice(["bf16", "f32"])}
    if op == "norm":
        case.update(p=rng.choice(["bf16", "f32"]), rms=rng.random() < 0.5, bias=rng.random() < 0.5,
                    saved8=rng.random() < 0.5)
        case["bias"] = case["bias"] and not case["rms"]
    return case


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "xent":
        V = case["V"]
        e = 2 if case["dw"] == "bf16" else 4
        n = 2 * M * K + 2 * V * K + 8 * M + 8 * M            # h, W, targets; loss and lse
        flops = 2 * M * K * V
        if case["train"]:
            n += 4 * M + 2 * M * K + e * V * K               # dloss; dH, dW
            flops += 4 * M * K * V                           # the logits once, dH, dW
        return {"bytes": n, "flops": flops}
    b = 2 if case["x"] == "bf16" else 4
    g = -(-K // GROUP)
    if case["op"] == "act8":
        return {"bytes": M * K * (2 * b + 2) + 8 * M * g, "flops": 4 * M * K}
    if case["op"] == "swiglu":
        # forward: gate, up -> y and the two 8-bit forms; backward: dy and those -> dgate, dup
        return {"bytes": M * K * (6 * b + 4) + 16 * M * g, "flops": 20 * M * K}
    e = 2 if case["p"] == "bf16" else 4
    params = 1 + int(case["bias"])
    n = M * K * 4 * b + 8 * M * (1 if case["rms"] else 2) + 3 * params * K * e
    n += (2 * M * K + 8 * M * g) if case["saved8"] else M * K * b
    return {"bytes": n, "flops": 16 * M * K}


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    M, K = case["M"], case["K"]
    s = {"case": dict(case)}
    if case["op"] == "xent":
        V = case["V"]
        # the head at its initial scale, and tokens of which some are already predicted well
        W = randn(V, K) * 0.02
        t = torch.randint(0, V, (M,), generator=gen, device="cuda")
        sure = torch.rand(M, 1, generator=gen, device="cuda") * (8.0 / (0.02 * math.sqrt(K)))
        h = randn(M, K) + sure * W[t] / (0.02 * math.sqrt(K))
        out = torch.rand(M, generator=gen, device="cuda") < case["left_out"]
        t = torch.where(out, -100, t)
        s["h"], s["W"], s["targets"] = h.to(torch.bfloat16), W.to(torch.bfloat16), t
        # the mean over the tokens that count
        s["dloss"] = torch.full((M,), 1.0, device="cuda") / (t >= 0).sum().clamp(min=1)
        if own:
            import ternary_weight_quantization_b200 as bl
            s["b"] = bl.XentBuffers.allocate(M, V, K, DTYPES[case["dw"]], backward=case["train"])
        return s
    dt = DTYPES[case["x"]]
    if case["op"] == "swiglu":
        s["gate"], s["up"], s["dy"] = (randn(M, K).to(dt) for _ in range(3))
        if own:
            import ternary_weight_quantization_b200 as bl
            s["b"] = bl.SwigluBuffers.allocate(M, K, dt)
        return s
    # a residual stream: a few features much larger than the others
    x = randn(M, K) * (1.0 + 15.0 * (torch.rand(K, generator=gen, device="cuda") < 0.01)) + 0.25 * randn(K)
    s["x"] = x.to(dt)
    if case["op"] == "act8":
        if own:
            import ternary_weight_quantization_b200 as bl
            s["b"] = bl.Act8.allocate(M, K)
            s["out"] = torch.empty_like(s["x"])
        return s
    pt = DTYPES[case["p"]]
    s["dy"] = (randn(M, K) * 0.1).to(dt)
    s["weight"] = (1.0 + 0.2 * randn(K)).to(pt)
    s["bias"] = (0.2 * randn(K)).to(pt) if case["bias"] else None
    if own:
        import ternary_weight_quantization_b200 as bl
        s["b"] = bl.NormBuffers.allocate(M, K, dt, pt, rms=case["rms"], bias=case["bias"], saved8=case["saved8"])
    return s


# ----------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return _own(s, case)
    if op == "xent":
        return _xent(s, case)
    if op == "norm":
        return _norm(s, case)
    if op == "swiglu":
        return _swiglu(s)
    values, _ = _saved8(s["x"])
    return {"x": values.to(s["x"].dtype)}


def _own(s, case):
    import ternary_weight_quantization_b200 as bl
    op, b = case["op"], s["b"]
    if op == "xent":
        bl.bl_linear_xent_forward(s["h"], s["W"], s["targets"], b.loss, b.lse, b.workspace)
        if not case["train"]:
            return {"loss": b.loss, "lse": b.lse}
        bl.bl_linear_xent_backward(s["h"], s["W"], s["targets"], b.lse, s["dloss"], b.dH, b.dW, b.workspace)
        return {"loss": b.loss, "lse": b.lse, "dH": b.dH, "dW": b.dW}
    if op == "norm":
        rms = case["rms"]
        bl.bl_norm_forward(s["x"], s["weight"], s["bias"], EPS, b.y, b.mean, b.rstd, rms=rms, saved8=b.saved8)
        x = b.saved8 if case["saved8"] else s["x"]
        bl.bl_norm_backward(s["dy"], x, s["weight"], b.mean, b.rstd, b.dx, b.dweight, b.dbias, b.workspace, rms=rms)
        out = {"y": b.y, "rstd": b.rstd, "dx": b.dx, "dweight": b.dweight}
        if not rms:
            out["mean"] = b.mean
        if case["bias"]:
            out["dbias"] = b.dbias
        return out
    if op == "swiglu":
        bl.bl_swiglu_forward(s["gate"], s["up"], b.y, b.gate8, b.up8)
        bl.bl_swiglu_backward(s["dy"], b.gate8, b.up8, b.dgate, b.dup)
        return {"y": b.y, "dgate": b.dgate, "dup": b.dup}
    bl.bl_act8_encode(s["x"], b)
    bl.bl_act8_decode(b, s["out"])
    return {"x": s["out"]}


# ----------------------------------------------------------------- plain forms (32 bits)

def _xent(s, case):
    h, W, t = s["h"].float(), s["W"].float(), s["targets"]
    counts = t >= 0
    at = torch.where(counts, t, 0)[:, None]
    logits = h @ W.t()
    top = logits.max(dim=1, keepdim=True).values
    lse = top + torch.log(torch.exp(logits - top).sum(dim=1, keepdim=True))
    loss = torch.where(counts, (lse - logits.gather(1, at))[:, 0], 0.0)
    out = {"loss": loss, "lse": lse[:, 0]}
    if case["train"]:
        p = torch.exp(logits - lse)
        del logits
        p.scatter_add_(1, at, torch.full_like(lse, -1.0))
        p *= torch.where(counts, s["dloss"], 0.0)[:, None]
        out["dH"] = (p @ W).to(torch.bfloat16)
        out["dW"] = (p.t() @ h).to(DTYPES[case["dw"]])
    return out


def _saved8(x):
    """The values that the 8-bit form of x stands for (fp32), and its scales.

    Groups of 128 values of a row: a = max(absmax, 1e-30), codes
    rint(fp32(x * fp32(127 / a))), scale fp32(a / 127), value fp32(code * scale).
    """
    M, K = x.shape
    g = -(-K // GROUP)
    v = torch.zeros(M, g * GROUP, device=x.device)
    v[:, :K] = x
    v = v.view(M, g, GROUP)
    a = v.abs().amax(dim=2, keepdim=True).clamp(min=FLOOR)
    codes = torch.round(v * (127.0 / a))
    scale = a / 127.0
    return (codes * scale).view(M, g * GROUP)[:, :K], scale[:, :, 0]


def _norm(s, case):
    x, dy, w = s["x"].float(), s["dy"].float(), s["weight"].float()
    if case["rms"]:
        mean = torch.zeros(x.shape[0], 1, device=x.device)
    else:
        mean = x.mean(dim=1, keepdim=True)
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + EPS)
    y = d * rstd * w
    if case["bias"]:
        y = y + s["bias"].float()
    saved = _saved8(s["x"])[0] if case["saved8"] else x
    xhat = (saved - mean) * rstd
    g = dy * w
    c2 = (g * xhat).mean(dim=1, keepdim=True)
    c1 = torch.zeros_like(c2) if case["rms"] else g.mean(dim=1, keepdim=True)
    dx = rstd * (g - c1 - xhat * c2)
    pt = s["weight"].dtype
    out = {"y": y.to(s["x"].dtype), "rstd": rstd[:, 0], "dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(dim=0).to(pt)}
    if not case["rms"]:
        out["mean"] = mean[:, 0]
    if case["bias"]:
        out["dbias"] = dy.sum(dim=0).to(pt)
    return out


def _swiglu(s):
    dt = s["gate"].dtype
    gate, up, dy = s["gate"].float(), s["up"].float(), s["dy"].float()
    y = gate / (1.0 + torch.exp(-gate)) * up
    g8, u8 = _saved8(s["gate"])[0], _saved8(s["up"])[0]
    sig = 1.0 / (1.0 + torch.exp(-g8))
    return {"y": y.to(dt), "dgate": (dy * u8 * sig * (1.0 + g8 * (1.0 - sig))).to(dt), "dup": (dy * g8 * sig).to(dt)}


# ----------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "xent":
        h, W, t = s["h"].double(), s["W"].double(), s["targets"]
        z = h @ W.t()
        lse = torch.logsumexp(z, dim=1)
        rows = torch.arange(case["M"], device="cuda")
        counts = t >= 0
        out = {"loss": torch.where(counts, lse - z[rows, t.clamp(min=0)], 0.0), "lse": lse}
        if case["train"]:
            z.sub_(lse[:, None]).exp_()
            z[rows[counts], t[counts]] -= 1.0
            z.mul_(torch.where(counts, s["dloss"].double(), 0.0)[:, None])
            out["dH"], out["dW"] = z @ W, z.t() @ h
        return out
    if case["op"] == "act8":
        return {"x": _exact8(s["x"])}
    if case["op"] == "swiglu":
        gate, up, dy = s["gate"].double(), s["up"].double(), s["dy"].double()
        g8, u8 = _exact8(s["gate"]), _exact8(s["up"])
        sg = torch.sigmoid(g8)
        return {"y": gate * torch.sigmoid(gate) * up, "dgate": dy * u8 * (sg + g8 * sg * (1 - sg)), "dup": dy * g8 * sg}
    x, dy, w = s["x"].double(), s["dy"].double(), s["weight"].double()
    if case["rms"]:
        mu, var = torch.zeros_like(x[:, :1]), (x ** 2).mean(1, keepdim=True)
    else:
        var, mu = torch.var_mean(x, dim=1, keepdim=True, correction=0)
    r = torch.rsqrt(var + EPS)
    y = (x - mu) * r * w + (s["bias"].double() if case["bias"] else 0.0)
    n = ((_exact8(s["x"]) if case["saved8"] else x) - mu) * r
    g = dy * w
    along = (g * n).mean(1, keepdim=True) * n
    flat = 0.0 if case["rms"] else g.mean(1, keepdim=True)
    out = {"y": y, "rstd": r[:, 0], "dx": (g - flat - along) * r, "dweight": torch.einsum("mk,mk->k", dy, n)}
    if not case["rms"]:
        out["mean"] = mu[:, 0]
    if case["bias"]:
        out["dbias"] = dy.sum(0)
    return out


def _exact8(x):
    """The 8-bit form by its definition, which fixes where fp32 rounds: the
    products of an fp32 value and an fp32 factor are exact in 64 bits, and
    each is rounded once."""
    M, K = x.shape
    pad = -K % GROUP
    v = torch.nn.functional.pad(x.double(), (0, pad)).reshape(M, -1, GROUP)
    a = v.abs().amax(-1, keepdim=True).clamp(min=float(torch.tensor(FLOOR, dtype=torch.float32)))
    inv = (127.0 / a).float().double()
    code = torch.round((v * inv).float().double())
    value = (code * (a / 127.0).float().double()).float().double()
    return value.reshape(M, -1)[:, :K]
