"""The training operators next to the layer, without a GPU: the C ABI refuses
bad arguments before it enqueues anything, the binding refuses tensors that do
not fit, sizes of workspaces, and empty calls."""

import ctypes

import pytest
import torch

import ternary_weight_quantization_b200 as bl
from ternary_weight_quantization_b200 import bitlinear as b

F = ctypes.c_void_p(0x10000)        # never dereferenced: validation fails first
MIS = ctypes.c_void_p(0x10008)
BIG = 1 << 40


def _xf(h=F, W=F, t=F, M=4, V=100, K=64, loss=F, lse=F, ws=F, n=BIG):
    return lambda L: L.bl_linear_xent_forward(h, W, t, M, V, K, loss, lse, ws, n, None)


def _xb(h=F, W=F, t=F, lse=F, dl=F, M=4, V=100, K=64, dH=F, dW=F, dt=0, ws=F, n=BIG):
    return lambda L: L.bl_linear_xent_backward(h, W, t, lse, dl, M, V, K, dH, dW, dt, 0, ws, n, None)


def _nf(x=F, dt=0, w=F, bias=F, pdt=0, M=4, K=64, eps=1e-6, rms=0, y=F, mean=F, rstd=F, c=None, s=None):
    return lambda L: L.bl_norm_forward(x, dt, w, bias, pdt, M, K, eps, rms, y, mean, rstd, c, s, None)


def _nb(dy=F, x=F, c=None, s=None, dt=0, w=F, pdt=0, mean=F, rstd=F, M=4, K=64, rms=0, dx=F, dw=F, db=F, ws=F, n=BIG):
    return lambda L: L.bl_norm_backward(dy, x, c, s, dt, w, pdt, mean, rstd, M, K, rms, dx, dw, db, 0, ws, n, None)


def _sf(gate=F, up=F, dt=0, M=4, K=64, y=F, saved=(None,) * 4):
    return lambda L: L.bl_swiglu_forward(gate, up, dt, M, K, y, *saved, None)


def _sb(dy=F, saved=(F,) * 4, dt=0, M=4, K=64, dg=F, du=ctypes.c_void_p(0x20000)):
    return lambda L: L.bl_swiglu_backward(dy, *saved, dt, M, K, dg, du, None)


@pytest.mark.parametrize("call,expect", [
    (_xf(M=-1), 1), (_xf(V=0), 1), (_xf(K=60), 2), (_xf(K=0), 2), (_xf(K=65544), 2), (_xf(M=131073), 2),
    (_xf(V=(1 << 24) + 1), 2), (_xf(h=None), 1), (_xf(W=None), 1), (_xf(t=None), 1), (_xf(loss=None), 1),
    (_xf(lse=None), 1), (_xf(h=MIS), 4), (_xf(W=MIS), 4), (_xf(t=MIS), 4), (_xf(lse=MIS), 4),
    (_xf(ws=None), 8), (_xf(ws=MIS), 8), (_xf(n=64), 8),
    (_xb(M=-1), 1), (_xb(V=0), 1), (_xb(K=12), 2), (_xb(dt=2), 3), (_xb(h=None), 1), (_xb(lse=None), 1),
    (_xb(dl=None), 1), (_xb(t=None), 1), (_xb(dH=MIS), 4), (_xb(dW=MIS), 4), (_xb(dl=MIS), 4), (_xb(ws=None), 8),
    (_xb(n=1000), 8), (_xb(ws=MIS), 8),
    (lambda L: L.bl_act8_encode(F, 2, 4, 64, F, F, None), 3),
    (lambda L: L.bl_act8_encode(F, 0, -1, 64, F, F, None), 1),
    (lambda L: L.bl_act8_encode(F, 0, 4, 0, F, F, None), 2),
    (lambda L: L.bl_act8_encode(None, 0, 4, 64, F, F, None), 1),
    (lambda L: L.bl_act8_encode(F, 0, 4, 64, MIS, F, None), 4),
    (lambda L: L.bl_act8_decode(F, F, 4, 64, F, 7, None), 3),
    (lambda L: L.bl_act8_decode(F, None, 4, 64, F, 0, None), 1),
    (lambda L: L.bl_act8_decode(F, MIS, 4, 64, F, 0, None), 4),
    (lambda L: L.bl_act8_decode(F, F, 4, (1 << 30) + 1, F, 0, None), 2),
    (_nf(K=0), 2), (_nf(M=-1), 1), (_nf(dt=9), 3), (_nf(pdt=9), 3), (_nf(eps=float("nan")), 1),
    (_nf(eps=float("inf")), 1), (_nf(eps=-1.0), 1), (_nf(c=F), 1), (_nf(s=F), 1), (_nf(x=None), 1), (_nf(y=None), 1),
    (_nf(mean=None), 1), (_nf(rstd=None), 1), (_nf(w=MIS), 4), (_nf(bias=MIS), 4), (_nf(c=MIS, s=F), 4),
    (_nb(K=0), 2), (_nb(dt=9), 3), (_nb(pdt=9), 3), (_nb(c=F, s=F), 1), (_nb(x=None), 1), (_nb(x=None, c=F), 1),
    (_nb(dy=None), 1), (_nb(mean=None), 1), (_nb(rstd=None), 1), (_nb(dx=MIS), 4), (_nb(ws=None), 8), (_nb(n=100), 8),
    (_sf(K=0), 2), (_sf(dt=5), 3), (_sf(saved=(F, None, F, F)), 1), (_sf(gate=None), 1), (_sf(y=MIS), 4),
    (_sf(saved=(F, F, F, MIS)), 4),
    (_sb(dt=5), 3), (_sb(saved=(F, F, None, F)), 1), (_sb(dy=None), 1), (_sb(du=F), 1), (_sb(dg=MIS), 4),
])
def test_host_validation_without_gpu(call, expect):
    lib = b.load_library()
    assert call(lib) == expect
    assert lib.bl_last_error_message().decode()


def test_empty_work_is_ok_without_gpu():
    lib = b.load_library()
    N = None
    assert _xf(h=N, W=N, t=N, M=0, loss=N, lse=N, ws=N, n=0)(lib) == 0
    assert _xb(h=N, W=N, t=N, lse=N, dl=N, M=0, dH=N, dW=N, ws=N, n=0)(lib) == 0
    assert _xb(dH=N, dW=N, ws=N, n=0)(lib) == 0
    assert lib.bl_act8_encode(N, 0, 0, 64, N, N, N) == 0
    assert lib.bl_act8_decode(N, N, 0, 64, N, 0, N) == 0
    assert _nf(x=N, M=0, y=N, mean=N, rstd=N)(lib) == 0
    assert _nb(dy=N, x=N, M=0, mean=N, rstd=N, dw=N, db=N, ws=N, n=0)(lib) == 0
    assert _nb(dx=N, dw=N, db=N, ws=N, n=0)(lib) == 0
    assert _sf(gate=N, up=N, M=0, y=N)(lib) == 0
    assert _sb(dy=N, saved=(N,) * 4, M=0, dg=N, du=N)(lib) == 0


def test_workspace_sizes():
    # forward: a (maximum, sum) pair per token and 128 vocabulary entries (64
    # where the tiles are few), and the target's logit per token (twice)
    assert bl.bl_linear_xent_forward_workspace_size(2048, 8192, 512) == 64 * 2048 * 8 + 2048 * 8
    assert bl.bl_linear_xent_forward_workspace_size(1, 257, 8) == 256 + 256
    assert bl.bl_linear_xent_forward_workspace_size(256, 9472, 8) == 148 * 256 * 8 + 256 * 8
    assert bl.bl_linear_xent_forward_workspace_size(256, 9473, 8) == 2 * 38 * 256 * 8 + 256 * 8
    assert bl.bl_linear_xent_forward_workspace_size(0, 8192, 512) == 0
    assert bl.bl_linear_xent_forward_workspace_size(4, 8192, 60) == 0
    # backward: never the logits of the whole vocabulary (here 1 GiB in bf16)
    n = bl.bl_linear_xent_backward_workspace_size(4096, 131072, 2560)
    assert 0 < n <= (128 << 20) + 4096 * 2560 * 2 + 4096 * 2560 * 4 + 1024
    assert bl.bl_linear_xent_backward_workspace_size(4096, 131072, 2560, torch.float32) <= n + (1 << 20)
    assert bl.bl_linear_xent_backward_workspace_size(0, 131072, 2560) == 0
    assert bl.bl_norm_backward_workspace_size(4096, 2560) == 148 * 2 * 2560 * 4
    assert bl.bl_norm_backward_workspace_size(10, 10000) == 148 * 2 * 10000 * 4 + 10 * 8
    assert bl.bl_norm_backward_workspace_size(0, 2560) == 0


M, K, V = 4, 64, 100
bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)   # noqa: E731
f32 = lambda *s: torch.zeros(s, dtype=torch.float32)   # noqa: E731
i64 = lambda *s: torch.zeros(s, dtype=torch.int64)     # noqa: E731
u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)      # noqa: E731
a8 = lambda: bl.Act8.allocate(M, K, "cpu")             # noqa: E731

CALLS = {
    "bl_linear_xent_forward": lambda: bl.bl_linear_xent_forward(bf(M, K), bf(V, K), i64(M), f32(M), f32(M), u8(4096)),
    "bl_linear_xent_backward": lambda: bl.bl_linear_xent_backward(bf(M, K), bf(V, K), i64(M), f32(M), f32(M), bf(M, K),
                                                                  bf(V, K), u8(4096)),
    "bl_act8_encode": lambda: bl.bl_act8_encode(bf(M, K), a8()),
    "bl_act8_decode": lambda: bl.bl_act8_decode(a8(), bf(M, K)),
    "bl_norm_forward": lambda: bl.bl_norm_forward(bf(M, K), f32(K), f32(K), 1e-6, bf(M, K), f32(M), f32(M)),
    "bl_norm_backward": lambda: bl.bl_norm_backward(bf(M, K), bf(M, K), f32(K), f32(M), f32(M), bf(M, K), f32(K),
                                                    f32(K), u8(4096)),
    "bl_swiglu_forward": lambda: bl.bl_swiglu_forward(bf(M, K), bf(M, K), bf(M, K), a8(), a8()),
    "bl_swiglu_backward": lambda: bl.bl_swiglu_backward(bf(M, K), a8(), a8(), bf(M, K), bf(M, K)),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_cpu_tensors_are_refused(name):
    with pytest.raises(ValueError, match="CUDA tensor"):
        CALLS[name]()


class _Fake:
    """Stands in for a CUDA tensor on a machine without one: the binding's
    checks read only these attributes before they call the library."""

    def __init__(self, *shape, dtype=torch.bfloat16, index=0, contiguous=True):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device("cuda", index)
        self.is_cuda, self._contiguous = True, contiguous

    def is_contiguous(self):
        return self._contiguous

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty((), dtype=self.dtype).element_size()

    def data_ptr(self):
        return 0x10000


def _args(name):
    f, i = torch.float32, torch.int64
    t = _Fake
    s8 = lambda: bl.Act8(t(M, K, dtype=torch.int8), t(M, 1, dtype=f))   # noqa: E731
    return {
        "bl_linear_xent_forward": dict(h=t(M, K), W=t(V, K), targets=t(M, dtype=i), loss=t(M, dtype=f), lse=t(M, dtype=f),
                                       workspace=t(4096, dtype=torch.uint8)),
        "bl_linear_xent_backward": dict(h=t(M, K), W=t(V, K), targets=t(M, dtype=i), lse=t(M, dtype=f),
                                        dloss=t(M, dtype=f), dH=t(M, K), dW=t(V, K), workspace=t(4096, dtype=torch.uint8)),
        "bl_act8_encode": dict(x=t(M, K), saved=s8()),
        "bl_act8_decode": dict(saved=s8(), x=t(M, K)),
        "bl_norm_forward": dict(x=t(M, K), weight=t(K), bias=t(K), eps=1e-6, y=t(M, K), mean=t(M, dtype=f),
                                rstd=t(M, dtype=f), saved8=s8()),
        "bl_norm_backward": dict(dy=t(M, K), x=t(M, K), weight=t(K), mean=t(M, dtype=f), rstd=t(M, dtype=f), dx=t(M, K),
                                 dweight=t(K), dbias=t(K), workspace=t(4096, dtype=torch.uint8)),
        "bl_swiglu_forward": dict(gate=t(M, K), up=t(M, K), y=t(M, K), gate8=s8(), up8=s8()),
        "bl_swiglu_backward": dict(dy=t(M, K), gate8=s8(), up8=s8(), dgate=t(M, K), dup=t(M, K)),
    }[name]


def _tensors(name):
    for key, v in _args(name).items():
        if isinstance(v, bl.Act8):
            yield key, "codes"
            yield key, "scales"
        elif isinstance(v, _Fake):
            yield key, None


def _spoil(args, key, part, change):
    t = args[key] if part is None else getattr(args[key], part)
    t = change(t)
    if part is None:
        args[key] = t
    else:
        setattr(args[key], part, t)
    return args


EVERY = [(n, k, p) for n in sorted(CALLS) for k, p in _tensors(n)]


@pytest.fixture(autouse=True)
def _library_is_not_called(monkeypatch, request):
    if "refused" in request.node.name:
        def no(*a):
            raise AssertionError("the library must not be reached")
        monkeypatch.setattr(b, "load_library", lambda: type("L", (), {"__getattr__": lambda self, n: no})())


@pytest.mark.parametrize("name,key,part", EVERY)
def test_tensors_of_another_device_are_refused(monkeypatch, name, key, part):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    args = _spoil(_args(name), key, part, lambda t: _Fake(*t.shape, dtype=t.dtype, index=1))
    with pytest.raises(ValueError, match="current CUDA device"):
        getattr(bl, name)(**args)


@pytest.mark.parametrize("name,key,part", [e for e in EVERY if e[1] != "workspace"])
def test_wrong_tensors_are_refused(monkeypatch, name, key, part):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for change in (lambda t: _Fake(*t.shape, dtype=t.dtype, contiguous=False),
                   lambda t: _Fake(*t.shape, dtype=torch.float16),
                   lambda t: _Fake(*(n + 1 for n in t.shape), dtype=t.dtype)):
        with pytest.raises(ValueError):
            getattr(bl, name)(**_spoil(_args(name), key, part, change))


def test_mixed_parameter_types_and_halves_of_a_pair_are_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    a = _args("bl_norm_forward")
    a["bias"] = _Fake(K, dtype=torch.float32)
    with pytest.raises(ValueError, match="bias must be"):
        bl.bl_norm_forward(**a)
    a = _args("bl_swiglu_forward")
    a["up8"] = None
    with pytest.raises(ValueError, match="together"):
        bl.bl_swiglu_forward(**a)
