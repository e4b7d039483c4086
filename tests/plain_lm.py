"""The decoder LM written out in plain torch, in 64 bits, from its formulas: ternary
projections of activations in 8 bits per token with straight-through gradients, and the
head in full or in 8 bits per row and token. It shares no code with the library's model."""

import math

import torch

NEGATIVE = float("-inf")


def _straight(x, value):
    return x + (value - x).detach()


def _eight(x):
    a = x.abs().amax(-1, keepdim=True).clamp(min=1e-5)
    return torch.round(x * (127 / a)) * (a / 127)


def _ternary(w):
    g = w.abs().mean()
    return torch.round(w / g).clamp(-1, 1) * g


def _norm(x, gain, eps):
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * gain


def gradients(init, ids, cfg, head8=False, mistake=None):
    """(loss, gradients by name). mistake: (what, k) spoils the k-th projection output on
    its way into the stream: "lost", "twice", or "late" (the norm behind it does not see it)."""
    p = {n: t.double().requires_grad_(True) for n, t in init.items()}
    B, S = ids.shape[0], ids.shape[1] - 1
    hd = cfg.d // cfg.heads
    count = 0

    def project(x8, name):
        return x8 @ _straight(p[name], _ternary(p[name])).t()

    def eight(x):
        return _straight(x, _eight(x))

    def add(h, out):
        nonlocal count
        what = mistake[0] if mistake and mistake[1] == count else None
        count += 1
        if what == "lost":
            return h, h
        if what == "twice":
            return h + 2 * out, h + 2 * out
        return h + out, (h if what == "late" else h + out)

    h = p["embed"][ids[:, :S]]
    seen = h
    mask = torch.full((S, S), NEGATIVE, dtype=torch.float64).triu(1)
    for i in range(cfg.layers):
        a = eight(_norm(seen, p[f"layer{i}.attn_norm"], cfg.norm_eps))
        q, k, v = (project(a, f"layer{i}.{n}").view(B, S, cfg.heads, hd).permute(0, 2, 1, 3) for n in "qkv")
        weights = torch.softmax(torch.einsum("bhid,bhjd->bhij", q, k) / math.sqrt(hd) + mask, -1)
        mixed = torch.einsum("bhij,bhjd->bihd", weights, v).reshape(B, S, cfg.d)
        h, seen = add(h, project(eight(mixed), f"layer{i}.o"))
        m = eight(_norm(seen, p[f"layer{i}.mlp_norm"], cfg.norm_eps))
        gate, up = project(m, f"layer{i}.gate"), project(m, f"layer{i}.up")
        h, seen = add(h, project(eight(gate * torch.sigmoid(gate) * up), f"layer{i}.down"))
    last = _norm(seen, p["final_norm"], cfg.norm_eps)
    if head8:
        z = eight(last) @ _straight(p["head"], _eight(p["head"])).t()
    else:
        z = last @ p["head"].t()
    z = torch.log_softmax(z, -1)
    loss = -z.gather(-1, ids[:, 1:, None]).mean()
    return loss.detach(), dict(zip(p, torch.autograd.grad(loss, list(p.values()), allow_unused=True, materialize_grads=True)))


def far(got, want):
    """The largest relative distance, in norm, of any parameter's gradient, and whose."""
    return max((float((got[n].double().cpu() - w).norm() / w.norm().clamp(min=1e-300)), n) for n, w in want.items())


# How far the library's model may be from this one: on the way from a parameter to the
# loss lie at most 9 operands in 8 bits (two layers' four and the head's), and as many on
# the gradients' way back. Next to a tie, or behind values rounded to bf16, a code is
# another one, so each is off by at most a step, and by half of one on average: 1 / 254
# of a row's largest value, 3.5 of its root mean square.
NEAR = 18 * 3.5 / 254


def case(cfg, seed):
    """Parameters with a head large enough that the loss depends on the stream, and ids."""
    from workloads.lm import lm_batches, lm_init
    init = lm_init(cfg, seed=seed)
    init["head"] = torch.randn(init["head"].shape, generator=torch.Generator().manual_seed(3)) * 0.2
    return init, lm_batches(cfg, seed=3)[0]


def of_library(init, ids, cfg, device, **how):
    """The same of the library's model."""
    from ternary_weight_quantization_b200 import lm
    params = {n: t.to(device).requires_grad_(True) for n, t in init.items()}
    loss = lm.lm_loss(params, ids.to(device), cfg, library_ops=True, **how)
    return loss.detach(), dict(zip(params, torch.autograd.grad(loss, list(params.values()))))
