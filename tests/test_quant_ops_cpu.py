"""The norm with an INT8 result, the product of INT8 operands and the gradients'
norm and clipping, without a GPU: the C ABI refuses bad arguments before it
enqueues anything, the binding refuses tensors that do not fit, sizes of
workspaces, and empty calls."""

import ctypes

import pytest
import torch

import ternary_weight_quantization_b200 as bl
from ternary_weight_quantization_b200 import bitlinear as b
from tests.test_train_ops_cpu import _Fake

F = ctypes.c_void_p(0x10000)        # never dereferenced: validation fails first
G = ctypes.c_void_p(0x20000)
NORM = ctypes.c_void_p(0x50000)
MIS = ctypes.c_void_p(0x10008)
BIG = 1 << 50
INF, NAN = float("inf"), float("nan")


def _qf(x=F, xt=0, r=F, st=0, w=F, pt=0, M=4, K=64, eps=1e-6, s=F, rstd=F, xq=F, sx=F):
    return lambda L: L.bl_norm_quant_forward(x, xt, r, st, w, pt, M, K, eps, s, rstd, xq, sx, None)


def _qb(dy=F, dt=0, ds=F, s=F, st=0, w=F, pt=0, rstd=F, M=4, K=64, dr=F, dx=G, xt=0, dw=F, ws=F, n=BIG):
    return lambda L: L.bl_norm_quant_backward(dy, dt, ds, s, st, w, pt, rstd, M, K, dr, dx, xt, dw, 0, ws, n, None)


def _lf(xq=F, sx=F, wq=F, sw=F, M=4, N=24, K=64, y=F, yt=0):
    return lambda L: L.bl_int8_linear_forward(xq, sx, wq, sw, M, N, K, y, yt, None)


def _lb(dY=F, xq=F, sx=F, wq=F, sw=F, M=4, N=24, K=64, dX=F, dW=F, dt=0, ws=F, n=BIG):
    return lambda L: L.bl_int8_linear_backward(dY, xq, sx, wq, sw, M, N, K, dX, dW, dt, 0, ws, n, None)


def _list(items):
    out = (b._Tensor * max(len(items), 1))()
    for i, (data, n, dt) in enumerate(items):
        out[i] = b._Tensor(data, n, dt)
    return out


TWO = ((0x10000, 100, 0), (0x20000, 7, 1))


def _gn(items=TWO, count=None, norm=NORM, ws=F, n=BIG):
    return lambda L: L.bl_grad_norm(_list(items), len(items) if count is None else count, norm, ws, n, None)


def _gc(items=TWO, out=None, most=1.0, norm=NORM, ws=F, n=BIG, count=None):
    def call(L):
        to = None if out is None else (ctypes.c_void_p * len(out))(*out)
        return L.bl_clip_grads(_list(items), to, len(items) if count is None else count, most, norm, ws, n, None)
    return call


@pytest.mark.parametrize("call,expect", [
    (_qf(M=-1), 1), (_qf(K=0), 2), (_qf(K=60), 2), (_qf(K=8200), 2), (_qf(M=(1 << 30) + 1), 2), (_qf(xt=2), 3),
    (_qf(st=7), 3), (_qf(pt=-1), 3), (_qf(xt=1, st=0), 3), (_qf(eps=NAN), 1), (_qf(eps=INF), 1), (_qf(eps=-1.0), 1),
    (_qf(x=None), 1), (_qf(r=None), 1), (_qf(s=None), 1), (_qf(r=None, s=None, st=1), 3), (_qf(rstd=None), 1),
    (_qf(xq=None), 1), (_qf(sx=None), 1), (_qf(x=MIS), 4), (_qf(r=MIS), 4), (_qf(w=MIS), 4), (_qf(s=MIS), 4),
    (_qf(rstd=MIS), 4), (_qf(xq=MIS), 4), (_qf(sx=MIS), 4),
    (_qb(M=-1), 1), (_qb(K=12), 2), (_qb(K=8200), 2), (_qb(dt=2), 3), (_qb(st=2), 3), (_qb(pt=2), 3), (_qb(xt=2), 3),
    (_qb(xt=1, st=0), 3), (_qb(dy=None), 1), (_qb(s=None), 1), (_qb(rstd=None), 1), (_qb(dx=F), 1), (_qb(dy=MIS), 4),
    (_qb(ds=MIS), 4), (_qb(s=MIS), 4), (_qb(w=MIS), 4), (_qb(rstd=MIS), 4), (_qb(dr=MIS), 4), (_qb(dx=MIS), 4),
    (_qb(dw=MIS), 4), (_qb(ws=None), 8), (_qb(ws=MIS), 8), (_qb(n=1000), 8),
    (_lf(M=-1), 1), (_lf(N=0), 1), (_lf(K=0), 2), (_lf(K=24), 2), (_lf(K=65552), 2), (_lf(M=131073), 2),
    (_lf(N=(1 << 20) + 1), 2), (_lf(yt=2), 3), (_lf(xq=None), 1), (_lf(sx=None), 1), (_lf(wq=None), 1), (_lf(sw=None), 1),
    (_lf(y=None), 1), (_lf(xq=MIS), 4), (_lf(sx=MIS), 4), (_lf(wq=MIS), 4), (_lf(sw=MIS), 4), (_lf(y=MIS), 4),
    (_lb(M=-1), 1), (_lb(N=25), 2), (_lb(K=24), 2), (_lb(dt=2), 3), (_lb(dY=None), 1), (_lb(xq=None), 1), (_lb(sx=None), 1),
    (_lb(wq=None), 1), (_lb(sw=None), 1), (_lb(dY=MIS), 4), (_lb(xq=MIS), 4), (_lb(sx=MIS), 4), (_lb(wq=MIS), 4),
    (_lb(sw=MIS), 4), (_lb(dX=MIS), 4), (_lb(dW=MIS), 4), (_lb(ws=None), 8), (_lb(ws=MIS), 8), (_lb(n=1000), 8),
    (_gn(count=-1), 1), (_gn(norm=None), 1), (_gn(items=((0x10000, 4, 2),)), 3), (_gn(items=((0x10000, -1, 0),)), 1),
    (_gn(items=((None, 4, 0),)), 1), (_gn(items=((0x10001, 4, 0),)), 4), (_gn(items=((0x10002, 4, 1),)), 4),
    (_gn(ws=None), 8), (_gn(ws=MIS), 8), (_gn(n=16), 8), (_gn(norm=ctypes.c_void_p(0x10002)), 4),
    (_gn(items=((0x10000, (1 << 40) + 1, 0),)), 2), (_gn(items=((0x10000, 1 << 39, 0),) * 3), 2),
    (lambda L: L.bl_grad_norm(None, 3, NORM, F, BIG, None), 1),
    (lambda L: L.bl_grad_norm(_list(TWO), (1 << 20) + 1, NORM, F, BIG, None), 2),
    (_gc(most=NAN), 1), (_gc(most=-1.0), 1), (_gc(norm=None), 1), (_gc(ws=None), 8), (_gc(n=16), 8),
    (_gc(items=TWO + ((0x10000, 4, 0),)), 1),                       # one tensor twice, in place
    (_gc(items=((0x10000, 100, 0), (0x100C0, 100, 0))), 1),         # two that overlap
    (_gc(items=((0x10000, 100, 0), (0x10000 - 2, 2, 0))), 1),
    (_gc(out=(0x30000, 0x30000 + 196)), 1),                         # outputs that overlap
    (_gc(out=(0x30000, 0x10000 + 196)), 1),                         # an output in another's input
    (_gc(out=(0x10000 + 4, 0x40000)), 1),                           # an output in its own input, at another place
    (_gc(out=(0x20000, 0x10000)), 1),                               # outputs that change places
    (_gc(norm=ctypes.c_void_p(0x10000 + 196)), 1), (_gn(norm=ctypes.c_void_p(0x20000 + 24)), 1),   # norm in a tensor
    (_gc(out=(0x30000, 0x40000), norm=ctypes.c_void_p(0x30000)), 1), (_gc(out=(None, 0x40000)), 1), (_gc(out=(0x30001, 0x40000)), 4), (_gc(out=(0x30000, 0x40002)), 4),
])
def test_host_validation_without_gpu(call, expect):
    lib = b.load_library()
    assert call(lib) == expect
    assert lib.bl_last_error_message().decode()


@pytest.mark.parametrize("call", [
    _gc(out=(0x30000, 0x20000)), _gc(), _gc(out=(0x30000, 0x30000 + 200)),
    _gc(items=((0x10000, 100, 0), (0x10000 + 200, 4, 1), (None, 0, 0))),
])
def test_lists_that_are_allowed_reach_the_device(call):
    """Everything is checked before the device, which is not there."""
    assert call(b.load_library()) in (5, 6)


def test_empty_work_is_ok_without_gpu():
    lib = b.load_library()
    N = None
    assert _qf(x=N, r=N, s=N, rstd=N, xq=N, sx=N, M=0)(lib) == 0
    assert _qb(dy=N, ds=N, s=N, rstd=N, M=0, dr=N, dx=N, dw=N, ws=N, n=0)(lib) == 0
    assert _qb(dr=N, dx=N, dw=N, ws=N, n=0)(lib) == 0
    assert _lf(xq=N, sx=N, wq=N, sw=N, y=N, M=0)(lib) == 0
    assert _lb(dY=N, xq=N, sx=N, wq=N, sw=N, M=0, dX=N, dW=N, ws=N, n=0)(lib) == 0
    assert _lb(dX=N, dW=N, ws=N, n=0)(lib) == 0


def test_workspace_sizes():
    assert bl.bl_norm_quant_backward_workspace_size(4096, 2560) == 148 * 2560 * 4
    assert bl.bl_norm_quant_backward_workspace_size(1, 64) == bl.bl_norm_quant_backward_workspace_size(1 << 20, 64)
    assert bl.bl_norm_quant_backward_workspace_size(0, 64) == 0 and bl.bl_norm_quant_backward_workspace_size(4, 60) == 0
    assert bl.bl_grad_norm_workspace_size(0) == 0
    assert bl.bl_grad_norm_workspace_size(1) == bl.bl_grad_norm_workspace_size(1024) < bl.bl_grad_norm_workspace_size(1025)
    # both operands in bf16, and dX's partial sums for the numbers of tokens with
    # few tiles: 1.5 * 74 tiles of 256 x 256 at most, and a row of 10 of them
    n = bl.bl_int8_linear_backward_workspace_size(4096, 6912, 2560)
    assert 0 < n - (4096 + 6912) * 2560 * 2 <= 1024 + (111 + 74) * 256 * 256 * 4
    assert bl.bl_int8_linear_backward_workspace_size(0, 64, 64) == 0
    assert bl.bl_int8_linear_backward_workspace_size(4, 60, 64) == 0


@pytest.mark.parametrize("N,K", [(6912, 2560), (32000, 80), (1 << 20, 512), (512, 16), (264, 65536)])
def test_int8_backward_workspaces_never_shrink_as_tokens_are_added(N, K):
    sizes = [bl.bl_int8_linear_backward_workspace_size(M, N, K) for M in
             (1, 16, 100, 256, 257, 511, 512, 513, 1000, 1024, 2048, 3000, 4096, 9999, 20000, 65536, 131072)]
    assert sizes == sorted(sizes) and sizes[0] > 0


# ----------------------------------------------------------------- the binding
M, K, N = 4, 64, 24
f32, i8, u8 = torch.float32, torch.int8, torch.uint8


def _args(name, t=_Fake):
    return {
        "bl_norm_quant_forward": dict(x=t(M, K), residual=t(M, K), weight=t(K), eps=1e-6, sum=t(M, K), rstd=t(M, dtype=f32),
                                      xq=t(M, K, dtype=i8), sx=t(M, dtype=f32)),
        "bl_norm_quant_backward": dict(dy=t(M, K), dsum=t(M, K), sum=t(M, K), weight=t(K), rstd=t(M, dtype=f32), dx=t(M, K),
                                       dresidual=t(M, K), dweight=t(K), workspace=t(1 << 20, dtype=u8)),
        "bl_int8_linear_forward": dict(xq=t(M, K, dtype=i8), sx=t(M, dtype=f32), wq=t(N, K, dtype=i8), sw=t(N, dtype=f32), y=t(M, N)),
        "bl_int8_linear_backward": dict(dY=t(M, N), xq=t(M, K, dtype=i8), sx=t(M, dtype=f32), wq=t(N, K, dtype=i8),
                                        sw=t(N, dtype=f32), dX=t(M, K), dW=t(N, K), workspace=t(1 << 20, dtype=u8)),
        "bl_grad_norm": dict(grads=[t(3, 5), t(7, dtype=f32)], norm=t(1, dtype=f32), workspace=t(1 << 20, dtype=u8)),
        "bl_clip_grads": dict(grads=[t(3, 5), t(7, dtype=f32)], max_norm=1.0, norm=t(1, dtype=f32),
                              workspace=t(1 << 20, dtype=u8), out=[t(3, 5), t(7, dtype=f32)]),
    }[name]


NAMES = ["bl_norm_quant_forward", "bl_norm_quant_backward", "bl_int8_linear_forward", "bl_int8_linear_backward",
         "bl_grad_norm", "bl_clip_grads"]


def _each(name):
    for key, v in _args(name).items():
        if isinstance(v, list):
            yield from ((key, i) for i in range(len(v)))
        elif isinstance(v, _Fake):
            yield key, None


def _spoil(args, key, i, change):
    if i is None:
        args[key] = change(args[key])
    else:
        args[key][i] = change(args[key][i])
    return args


EVERY = [(n, k, i) for n in NAMES for k, i in _each(n)]


@pytest.fixture(autouse=True)
def _library_is_not_called(monkeypatch, request):
    if "refused" in request.node.name:
        def no(*a):
            raise AssertionError("the library must not be reached")
        monkeypatch.setattr(b, "load_library", lambda: type("L", (), {"__getattr__": lambda self, n: no})())


@pytest.mark.parametrize("name", NAMES)
def test_cpu_tensors_are_refused(name):
    def cpu(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype)
    with pytest.raises(ValueError, match="CUDA tensor"):
        getattr(bl, name)(**_args(name, cpu))


@pytest.mark.parametrize("name,key,i", EVERY)
def test_tensors_of_another_device_are_refused(monkeypatch, name, key, i):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    args = _spoil(_args(name), key, i, lambda t: _Fake(*t.shape, dtype=t.dtype, index=1))
    with pytest.raises(ValueError, match="current CUDA device"):
        getattr(bl, name)(**args)


@pytest.mark.parametrize("name,key,i", [e for e in EVERY if e[1] != "workspace"])
def test_wrong_tensors_are_refused(monkeypatch, name, key, i):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    changes = [lambda t: _Fake(*t.shape, dtype=t.dtype, contiguous=False), lambda t: _Fake(*t.shape, dtype=torch.float16)]
    if key != "grads" or name == "bl_clip_grads":
        changes.append(lambda t: _Fake(*(n + 1 for n in t.shape), dtype=t.dtype))
    for change in changes:
        with pytest.raises(ValueError):
            getattr(bl, name)(**_spoil(_args(name), key, i, change))


def test_lists_of_other_lengths_and_mixed_types_are_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    a = _args("bl_clip_grads")
    a["out"].pop()
    with pytest.raises(ValueError, match="out has 1"):
        bl.bl_clip_grads(**a)
    a = _args("bl_norm_quant_forward")
    a["sum"] = _Fake(M, K, dtype=f32)
    with pytest.raises(ValueError, match="sum must be"):
        bl.bl_norm_quant_forward(**a)
    a = _args("bl_norm_quant_backward")
    a["dweight"] = _Fake(K, dtype=f32)
    with pytest.raises(ValueError, match="dweight must be"):
        bl.bl_norm_quant_backward(**a)
