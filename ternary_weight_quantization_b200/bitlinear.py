"""Thin Python binding of libbitlinear.so (argument marshalling only).

The training operators next to the layer go through the extension module
_binding (csrc/binding.cpp), which makes the same checks and the call in one
step; where it finds an argument that does not fit, the checks here say which.

Each function has the name of the C entry point it calls, takes torch CUDA
tensors, checks dtype / shape / contiguity, passes raw device pointers and
the current CUDA stream, and raises :class:`BitLinearError` on any status
other than BL_OK. Every step of the computation runs in the library's CUDA
kernels; there is no CPU or PyTorch fallback, and importing the library fails
loudly when the shared object is missing.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbitlinear.so")

BL_BF16 = 0
BL_F32 = 1

STATUS = {
    0: "BL_OK", 1: "BL_ERR_INVALID_ARG", 2: "BL_ERR_UNSUPPORTED_SHAPE", 3: "BL_ERR_DTYPE",
    4: "BL_ERR_ALIGNMENT", 5: "BL_ERR_ARCH", 6: "BL_ERR_CUDA", 7: "BL_ERR_TIMEOUT", 8: "BL_ERR_WORKSPACE",
}

# (name, restype, argtypes) of every symbol include/bitlinear.h declares
_VP, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
SIGNATURES = {
    "bl_version": (_I32, []),
    "bl_status_string": (ctypes.c_char_p, [_I32]),
    "bl_last_error_message": (ctypes.c_char_p, []),
    "bl_quantize_weight_workspace_size": (_SZ, [_I64, _I64]),
    "bl_quantize_weight": (_I32, [_VP, _I32, _I64, _I64, _VP, _VP, _VP, _SZ, _VP]),
    "bl_quantize_weight_noalloc": (_I32, [_VP, _I32, _I64, _I64, _VP, _VP, _VP]),
    "bl_quantize_act": (_I32, [_VP, _I64, _I64, _VP, _VP, _VP]),
    "bl_quantize": (_I32, [_VP, _I32, _I64, _I64, _VP, _I64, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "bl_forward": (_I32, [_VP, _VP, _VP, _VP, _I64, _I64, _I64, _VP, _VP, _VP]),
    "bl_backward": (_I32, [_VP, _VP, _VP, _VP, _VP, _I64, _I64, _I64, _VP, _VP, _I32, _I32, _VP]),
    "bl_backward_signs": (_I32, [_VP, _VP, _VP, _VP, _VP, _I64, _I64, _I64, _VP, _VP, _VP]),
    "bl_backward_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "bl_backward_ws": (_I32, [_VP, _VP, _VP, _VP, _VP, _I64, _I64, _I64, _VP, _VP, _I32, _I32, _VP, _SZ, _VP]),
    "bl_backward_signs_ws": (_I32, [_VP, _VP, _VP, _VP, _VP, _I64, _I64, _I64, _VP, _VP, _VP, _SZ, _VP]),
    "bl_export_weights": (_I32, [_VP, _VP, _I64, _I64, _VP, _VP, _VP]),
    "bl_get_last_error": (_I32, []),
    "bl_reset_error": (_I32, []),
    "bl_selftest_timeout": (_I32, [_VP]),
    "bl_sign_pack": (_I32, [_VP, _I32, _I64, _I64, _VP, _VP]),
    "bl_sign_vote": (_I32, [_VP, _I32, _I64, _I64, _VP, _VP]),
    "bl_signsgd_update": (_I32, [_VP, _I32, _I64, _I64, _VP, ctypes.c_float, _VP]),
    "bl_signsgd_apply": (_I32, [_VP, _I32, _VP, _I32, _I64, _I64, ctypes.c_float, _VP, _VP, _VP, _SZ, _VP]),
    "bl_linear_xent_forward_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "bl_linear_xent_forward": (_I32, [_VP, _VP, _VP, _I64, _I64, _I64, _VP, _VP, _VP, _SZ, _VP]),
    "bl_linear_xent_backward_workspace_size": (_SZ, [_I64, _I64, _I64, _I32]),
    "bl_linear_xent_backward": (_I32, [_VP, _VP, _VP, _VP, _VP, _I64, _I64, _I64, _VP, _VP, _I32, _I32, _VP, _SZ, _VP]),
    "bl_act8_encode": (_I32, [_VP, _I32, _I64, _I64, _VP, _VP, _VP]),
    "bl_act8_decode": (_I32, [_VP, _VP, _I64, _I64, _VP, _I32, _VP]),
    "bl_norm_forward": (_I32, [_VP, _I32, _VP, _VP, _I32, _I64, _I64, ctypes.c_float, _I32, _VP, _VP, _VP, _VP, _VP, _VP]),
    "bl_norm_backward_workspace_size": (_SZ, [_I64, _I64]),
    "bl_norm_backward": (_I32, [_VP, _VP, _VP, _VP, _I32, _VP, _I32, _VP, _VP, _I64, _I64, _I32, _VP, _VP, _VP, _I32, _VP,
                                _SZ, _VP]),
    "bl_swiglu_forward": (_I32, [_VP, _VP, _I32, _I64, _I64, _VP, _VP, _VP, _VP, _VP, _VP]),
    "bl_swiglu_backward": (_I32, [_VP, _VP, _VP, _VP, _VP, _I32, _I64, _I64, _VP, _VP, _VP]),
    "bl_norm_quant_forward": (_I32, [_VP, _I32, _VP, _I32, _VP, _I32, _I64, _I64, ctypes.c_float, _VP, _VP, _VP, _VP, _VP]),
    "bl_norm_quant_backward_workspace_size": (_SZ, [_I64, _I64]),
    "bl_norm_quant_backward": (_I32, [_VP, _I32, _VP, _VP, _I32, _VP, _I32, _VP, _I64, _I64, _VP, _VP, _I32, _VP, _I32, _VP,
                                      _SZ, _VP]),
    "bl_int8_linear_forward": (_I32, [_VP, _VP, _VP, _VP, _I64, _I64, _I64, _VP, _I32, _VP]),
    "bl_int8_linear_backward_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "bl_int8_linear_backward": (_I32, [_VP, _VP, _VP, _VP, _VP, _I64, _I64, _I64, _VP, _VP, _I32, _I32, _VP, _SZ, _VP]),
    "bl_grad_norm_workspace_size": (_SZ, [_I64]),
    "bl_grad_norm": (_I32, [_VP, _I64, _VP, _VP, _SZ, _VP]),
    "bl_clip_grads": (_I32, [_VP, _VP, _I64, ctypes.c_double, _VP, _VP, _SZ, _VP]),
}


class BitLinearError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}: {detail}")
        self.status = status


_LIB = None
_QUICK = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libbitlinear.so and declare its C signatures (raises if absent)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m ternary_weight_quantization_b200.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = lib
    return lib


def _quick():
    """The extension module (raises if absent)."""
    global _QUICK
    if _QUICK is None:
        load_library()
        if not os.path.exists(os.path.join(_PKG, "_binding.so")):
            raise RuntimeError(f"{_PKG}/_binding.so is missing: build it with "
                               "`python -m ternary_weight_quantization_b200.build`")
        from . import _binding
        _QUICK = _binding
    return _QUICK


def _check(status: int, where: str):
    if status != 0:
        lib = load_library()
        detail = lib.bl_last_error_message().decode(errors="replace")
        raise BitLinearError(status, where, detail)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    elif stream.device.index != torch.cuda.current_device():
        raise ValueError(f"stream of {stream.device} but the current CUDA device is cuda:{torch.cuda.current_device()}")
    return ctypes.c_void_p(stream.cuda_stream)


def _on_current_device(*tensors):
    """Every tensor argument must live on the current CUDA device: the library
    launches on the current device (and the stream passed is that device's),
    so a tensor of another GPU would hand its kernels foreign pointers."""
    cur = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.device.index != cur:
            raise ValueError(f"tensor on {t.device} but the current CUDA device is cuda:{cur}; "
                             "call under torch.cuda.device(...) of the tensors' device")


def _need(t, dtype, shape, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ----------------------------------------------------------------- entry points

def bl_version() -> int:
    return load_library().bl_version()


def bl_quantize_weight_workspace_size(N: int, K: int) -> int:
    return load_library().bl_quantize_weight_workspace_size(N, K)


def bl_quantize_weight(W, w_packed, gamma, workspace, stream=None):
    """S1: W [N,K] bf16|f32 -> w_packed [N,K/4] uint8, gamma [1] f32."""
    N, K = W.shape
    if W.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("W must be bf16 or f32")
    _need(W, W.dtype, (N, K), "W")
    _need(w_packed, torch.uint8, (N, K // 4), "w_packed")
    _need(gamma, torch.float32, (1,), "gamma")
    _on_current_device(W, w_packed, gamma, workspace)
    wdt = BL_F32 if W.dtype == torch.float32 else BL_BF16
    _check(load_library().bl_quantize_weight(_ptr(W), wdt, N, K, _ptr(w_packed), _ptr(gamma), _ptr(workspace),
                                             workspace.numel() * workspace.element_size(), _stream(stream)),
           "bl_quantize_weight")


def bl_quantize_act(x, xq, sx, stream=None):
    """S2: x [M,K] bf16 -> xq [M,K] int8, sx [M] f32."""
    M, K = x.shape
    _need(x, torch.bfloat16, (M, K), "x")
    _need(xq, torch.int8, (M, K), "xq")
    _need(sx, torch.float32, (M,), "sx")
    _on_current_device(x, xq, sx)
    _check(load_library().bl_quantize_act(_ptr(x), M, K, _ptr(xq), _ptr(sx), _stream(stream)), "bl_quantize_act")


def bl_quantize(W, x, w_packed, gamma, xq, sx, workspace, stream=None):
    """S1 + S2 in one call (same outputs as bl_quantize_weight then bl_quantize_act)."""
    N, K = W.shape
    M = x.shape[0]
    if W.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("W must be bf16 or f32")
    _need(W, W.dtype, (N, K), "W")
    _need(x, torch.bfloat16, (M, K), "x")
    _need(w_packed, torch.uint8, (N, K // 4), "w_packed")
    _need(gamma, torch.float32, (1,), "gamma")
    _need(xq, torch.int8, (M, K), "xq")
    _need(sx, torch.float32, (M,), "sx")
    _on_current_device(W, x, w_packed, gamma, xq, sx, workspace)
    wdt = BL_F32 if W.dtype == torch.float32 else BL_BF16
    _check(load_library().bl_quantize(_ptr(W), wdt, N, K, _ptr(x), M, _ptr(w_packed), _ptr(gamma), _ptr(xq),
                                      _ptr(sx), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                      _stream(stream)),
           "bl_quantize")


def bl_forward(xq, sx, w_packed, gamma, y, debug_acc=None, stream=None):
    """S3: y [M,N] bf16 = xq . codes^T * sx * gamma (debug_acc [M,N] int32 optional)."""
    M, K = xq.shape
    N = w_packed.shape[0]
    _need(xq, torch.int8, (M, K), "xq")
    _need(sx, torch.float32, (M,), "sx")
    _need(w_packed, torch.uint8, (N, K // 4), "w_packed")
    _need(gamma, torch.float32, (1,), "gamma")
    _need(y, torch.bfloat16, (M, N), "y")
    if debug_acc is not None:
        _need(debug_acc, torch.int32, (M, N), "debug_acc")
    _on_current_device(xq, sx, w_packed, gamma, y, debug_acc)
    _check(load_library().bl_forward(_ptr(xq), _ptr(sx), _ptr(w_packed), _ptr(gamma), M, N, K, _ptr(y),
                                     _ptr(debug_acc), _stream(stream)), "bl_forward")


def bl_backward_workspace_size(M: int, N: int, K: int) -> int:
    return load_library().bl_backward_workspace_size(M, N, K)


def bl_backward(dY, xq, sx, w_packed, gamma, dX=None, dW=None, accumulate_dW=False, stream=None, workspace=None):
    """S4: dX [M,K] bf16 = gamma * dY . codes; dW [N,K] (bf16|f32) = dY^T . x_hat.
    workspace (bl_backward_workspace_size bytes): x_hat is made once there
    (bl_backward_ws) instead of rebuilt in every dW tile; same results."""
    M, N = dY.shape
    K = xq.shape[1]
    _need(dY, torch.bfloat16, (M, N), "dY")
    _need(xq, torch.int8, (M, K), "xq")
    _need(sx, torch.float32, (M,), "sx")
    _need(w_packed, torch.uint8, (N, K // 4), "w_packed")
    _need(gamma, torch.float32, (1,), "gamma")
    dwdt = BL_BF16
    if dX is not None:
        _need(dX, torch.bfloat16, (M, K), "dX")
    if dW is not None:
        if dW.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("dW must be bf16 or f32")
        _need(dW, dW.dtype, (N, K), "dW")
        dwdt = BL_F32 if dW.dtype == torch.float32 else BL_BF16
    _on_current_device(dY, xq, sx, w_packed, gamma, dX, dW, workspace)
    lib = load_library()
    if workspace is None:
        _check(lib.bl_backward(_ptr(dY), _ptr(xq), _ptr(sx), _ptr(w_packed), _ptr(gamma), M, N, K,
                               _ptr(dX), _ptr(dW), dwdt, int(bool(accumulate_dW)), _stream(stream)),
               "bl_backward")
    else:
        _check(lib.bl_backward_ws(_ptr(dY), _ptr(xq), _ptr(sx), _ptr(w_packed), _ptr(gamma), M, N, K,
                                  _ptr(dX), _ptr(dW), dwdt, int(bool(accumulate_dW)), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream)),
               "bl_backward_ws")


def bl_backward_signs(dY, xq, sx, w_packed, gamma, dX, dw_sign_words, stream=None, workspace=None):
    """S4 with G1 fused: dX [M,K] bf16 (or None) as bl_backward, and the sign
    words of dW, dw_sign_words [N, K/32] int32 (bit patterns), instead of dW.
    workspace: as bl_backward's."""
    M, N = dY.shape
    K = xq.shape[1]
    _need(dY, torch.bfloat16, (M, N), "dY")
    _need(xq, torch.int8, (M, K), "xq")
    _need(sx, torch.float32, (M,), "sx")
    _need(w_packed, torch.uint8, (N, K // 4), "w_packed")
    _need(gamma, torch.float32, (1,), "gamma")
    if dX is not None:
        _need(dX, torch.bfloat16, (M, K), "dX")
    _need(dw_sign_words, torch.int32, (N, K // 32), "dw_sign_words")
    _on_current_device(dY, xq, sx, w_packed, gamma, dX, dw_sign_words, workspace)
    lib = load_library()
    if workspace is None:
        _check(lib.bl_backward_signs(_ptr(dY), _ptr(xq), _ptr(sx), _ptr(w_packed), _ptr(gamma), M, N, K,
                                     _ptr(dX), _ptr(dw_sign_words), _stream(stream)),
               "bl_backward_signs")
    else:
        _check(lib.bl_backward_signs_ws(_ptr(dY), _ptr(xq), _ptr(sx), _ptr(w_packed), _ptr(gamma), M, N, K,
                                        _ptr(dX), _ptr(dw_sign_words), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _stream(stream)),
               "bl_backward_signs_ws")


def bl_sign_pack(dW, sign_words, stream=None):
    """G1: sign_words [N, K/32] int32 (bit patterns) <- sign bits of dW [N, K] (bf16|f32)."""
    N, K = dW.shape
    if dW.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("dW must be bf16 or f32")
    _need(dW, dW.dtype, (N, K), "dW")
    _need(sign_words, torch.int32, (N, K // 32), "sign_words")
    _on_current_device(dW, sign_words)
    dt = BL_F32 if dW.dtype == torch.float32 else BL_BF16
    _check(load_library().bl_sign_pack(_ptr(dW), dt, N, K, _ptr(sign_words), _stream(stream)), "bl_sign_pack")


def bl_sign_vote(sign_words, direction, stream=None):
    """G2: direction [N, K/4] uint8 (2-bit packed) <- majority of sign_words [R, N, K/32] int32."""
    R, N, KW = sign_words.shape
    _need(sign_words, torch.int32, (R, N, KW), "sign_words")
    _need(direction, torch.uint8, (N, KW * 8), "direction")
    _on_current_device(sign_words, direction)
    _check(load_library().bl_sign_vote(_ptr(sign_words), R, N, KW * 32, _ptr(direction), _stream(stream)),
           "bl_sign_vote")


def bl_signsgd_update(W, direction, lr, stream=None):
    """G3: W [N, K] (bf16|f32) <- dtype_rn(fp32(W) - lr * direction), in place."""
    N, K = W.shape
    if W.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("W must be bf16 or f32")
    _need(W, W.dtype, (N, K), "W")
    _need(direction, torch.uint8, (N, K // 4), "direction")
    _on_current_device(W, direction)
    dt = BL_F32 if W.dtype == torch.float32 else BL_BF16
    _check(load_library().bl_signsgd_update(_ptr(W), dt, N, K, _ptr(direction), float(lr), _stream(stream)),
           "bl_signsgd_update")


def bl_signsgd_apply(sign_words, W, lr, w_packed, gamma, workspace, stream=None):
    """G2 + G3 + S1 fused on the holder: the majority direction of sign_words
    [R, N, K/32] int32 applied to W [N, K] (bf16|f32) in place, then W's new
    w_packed [N, K/4] uint8 and gamma [1] f32 (two launches)."""
    R, N, KW = sign_words.shape
    K = KW * 32
    if W.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("W must be bf16 or f32")
    _need(sign_words, torch.int32, (R, N, KW), "sign_words")
    _need(W, W.dtype, (N, K), "W")
    _need(w_packed, torch.uint8, (N, K // 4), "w_packed")
    _need(gamma, torch.float32, (1,), "gamma")
    _on_current_device(sign_words, W, w_packed, gamma, workspace)
    dt = BL_F32 if W.dtype == torch.float32 else BL_BF16
    _check(load_library().bl_signsgd_apply(_ptr(sign_words), R, _ptr(W), dt, N, K, float(lr), _ptr(w_packed),
                                           _ptr(gamma), _ptr(workspace),
                                           workspace.numel() * workspace.element_size(), _stream(stream)),
           "bl_signsgd_apply")


def bl_export_weights(w_packed, gamma, stream=None):
    """Copy (w_packed, gamma) to host: returns (uint8 [N,K/4] CPU tensor, float gamma)."""
    N, Kq = w_packed.shape
    host = torch.empty((N, Kq), dtype=torch.uint8, pin_memory=True)
    hg = torch.empty(1, dtype=torch.float32, pin_memory=True)
    _check(load_library().bl_export_weights(_ptr(w_packed), _ptr(gamma), N, Kq * 4, _ptr(host), _ptr(hg),
                                            _stream(stream)), "bl_export_weights")
    return host, float(hg[0])


def bl_get_last_error() -> int:
    return load_library().bl_get_last_error()


def bl_reset_error() -> int:
    return load_library().bl_reset_error()


# ----------------------------------------------------------------- training operators next to the layer

def _dtype_code(t, name):
    if t.dtype == torch.bfloat16:
        return BL_BF16
    if t.dtype == torch.float32:
        return BL_F32
    raise ValueError(f"{name} must be bf16 or f32")


def _device(t, name):
    """The current CUDA device, for a call whose first tensor is t."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return torch.cuda.current_device()


def _pointers(cur, specs):
    """Addresses of the tensors of specs, (tensor or None, dtype, shape, name)
    each, after the checks of _need and _on_current_device in one pass."""
    out = []
    for t, dtype, shape, name in specs:
        if t is None:
            out.append(None)
            continue
        if t.dtype is not dtype or t.shape != shape or t.device.index != cur or not t.is_contiguous():
            _need(t, dtype, shape, name)
            _on_current_device(t)
        out.append(t.data_ptr())
    return out


def _scratch(cur, workspace):
    """(address, bytes) of a workspace (None: none)."""
    if workspace is None:
        return None, 0
    if workspace.device.index != cur:
        _on_current_device(workspace)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _stream_of(stream, cur):
    # the address alone: no Stream object per call
    return torch._C._cuda_getCurrentRawStream(cur) if stream is None else _stream(stream)


def bl_linear_xent_forward_workspace_size(M: int, V: int, K: int) -> int:
    return load_library().bl_linear_xent_forward_workspace_size(M, V, K)


def bl_linear_xent_backward_workspace_size(M: int, V: int, K: int, dw_dtype=torch.bfloat16) -> int:
    code = BL_F32 if dw_dtype == torch.float32 else BL_BF16
    return load_library().bl_linear_xent_backward_workspace_size(M, V, K, code)


def bl_linear_xent_forward(h, W, targets, loss, lse, workspace, stream=None):
    """X1: loss [M], lse [M] f32 of the softmax cross-entropy of h [M,K] . W [V,K]^T
    (bf16) at targets [M] int64; a target outside 0..V-1 leaves its token out."""
    status = _quick().xent_forward(h, W, targets, loss, lse, workspace, stream)
    if status is not None:
        return _check(status, "bl_linear_xent_forward")
    M, K = h.shape
    V = W.shape[0]
    cur = _device(h, "h")
    p = _pointers(cur, ((h, torch.bfloat16, (M, K), "h"), (W, torch.bfloat16, (V, K), "W"),
                        (targets, torch.int64, (M,), "targets"), (loss, torch.float32, (M,), "loss"),
                        (lse, torch.float32, (M,), "lse")))
    ws, n = _scratch(cur, workspace)
    _check(load_library().bl_linear_xent_forward(p[0], p[1], p[2], M, V, K, p[3], p[4], ws, n, _stream_of(stream, cur)),
           "bl_linear_xent_forward")


def bl_linear_xent_backward(h, W, targets, lse, dloss, dH=None, dW=None, workspace=None, accumulate_dW=False,
                            stream=None):
    """X2: dH [M,K] bf16 and dW [V,K] (bf16|f32) of X1 (each may be None), given
    dloss [M] f32, the gradient of each token's loss, and X1's lse. Without dW a
    workspace sized for either type of dW will do."""
    status = _quick().xent_backward(h, W, targets, lse, dloss, dH, dW, workspace, accumulate_dW, stream)
    if status is not None:
        return _check(status, "bl_linear_xent_backward")
    M, K = h.shape
    V = W.shape[0]
    cur = _device(h, "h")
    dwdt = BL_BF16 if dW is None else _dtype_code(dW, "dW")
    p = _pointers(cur, ((h, torch.bfloat16, (M, K), "h"), (W, torch.bfloat16, (V, K), "W"),
                        (targets, torch.int64, (M,), "targets"), (lse, torch.float32, (M,), "lse"),
                        (dloss, torch.float32, (M,), "dloss"), (dH, torch.bfloat16, (M, K), "dH"),
                        (dW, None if dW is None else dW.dtype, (V, K), "dW")))
    ws, n = _scratch(cur, workspace)
    _check(load_library().bl_linear_xent_backward(*p[:5], M, V, K, p[5], p[6], dwdt, 1 if accumulate_dW else 0, ws, n,
                                                  _stream_of(stream, cur)), "bl_linear_xent_backward")


@dataclass
class Act8:
    """The 8-bit form of an activation [M,K]: codes [M,K] int8 and one scale per
    128 values of a row, scales [M, ceil(K / 128)] f32."""
    codes: torch.Tensor
    scales: torch.Tensor

    @staticmethod
    def allocate(M, K, device="cuda"):
        return Act8(codes=torch.empty((M, K), dtype=torch.int8, device=device),
                    scales=torch.empty((M, -(-K // 128)), dtype=torch.float32, device=device))


def _act8_specs(a, M, K, name):
    if a is None:
        return (None,) * 4, (None,) * 4
    return ((a.codes, torch.int8, (M, K), f"{name}.codes"),
            (a.scales, torch.float32, (M, -(-K // 128)), f"{name}.scales"))


def bl_act8_encode(x, saved: Act8, stream=None):
    """A1: saved <- the 8-bit form of x [M,K] (bf16|f32)."""
    status = _quick().act8_encode(x, saved.codes, saved.scales, stream)
    if status is not None:
        return _check(status, "bl_act8_encode")
    M, K = x.shape
    cur = _device(x, "x")
    dt = _dtype_code(x, "x")
    p = _pointers(cur, ((x, x.dtype, (M, K), "x"), *_act8_specs(saved, M, K, "saved")))
    _check(load_library().bl_act8_encode(p[0], dt, M, K, p[1], p[2], _stream_of(stream, cur)), "bl_act8_encode")


def bl_act8_decode(saved: Act8, x, stream=None):
    """A2: x [M,K] (bf16|f32) <- the saved values."""
    status = _quick().act8_decode(saved.codes, saved.scales, x, stream)
    if status is not None:
        return _check(status, "bl_act8_decode")
    M, K = x.shape
    cur = _device(x, "x")
    dt = _dtype_code(x, "x")
    p = _pointers(cur, (*_act8_specs(saved, M, K, "saved"), (x, x.dtype, (M, K), "x")))
    _check(load_library().bl_act8_decode(p[0], p[1], M, K, p[2], dt, _stream_of(stream, cur)), "bl_act8_decode")


def bl_norm_forward(x, weight, bias, eps, y, mean, rstd, rms=False, saved8: Act8 | None = None, stream=None):
    """N1: y [M,K] = layer norm (rms: RMS norm) of x [M,K] (bf16|f32) with weight,
    bias [K] (bf16|f32, each may be None); mean (None with rms), rstd [M] f32;
    saved8 receives the 8-bit form of x."""
    codes, scales = (None, None) if saved8 is None else (saved8.codes, saved8.scales)
    status = _quick().norm_forward(x, weight, bias, eps, y, mean, rstd, rms, codes, scales, stream)
    if status is not None:
        return _check(status, "bl_norm_forward")
    M, K = x.shape
    cur = _device(x, "x")
    dt = _dtype_code(x, "x")
    param = weight if weight is not None else bias
    pdt, ptype = (BL_F32, None) if param is None else (_dtype_code(param, "weight or bias"), param.dtype)
    p = _pointers(cur, ((x, x.dtype, (M, K), "x"), (weight, ptype, (K,), "weight"), (bias, ptype, (K,), "bias"),
                        (y, x.dtype, (M, K), "y"), (mean, torch.float32, (M,), "mean"),
                        (rstd, torch.float32, (M,), "rstd"), *_act8_specs(saved8, M, K, "saved8")))
    _check(load_library().bl_norm_forward(p[0], dt, p[1], p[2], pdt, M, K, eps, 1 if rms else 0, *p[3:8],
                                          _stream_of(stream, cur)), "bl_norm_forward")


def bl_norm_backward_workspace_size(M: int, K: int) -> int:
    return load_library().bl_norm_backward_workspace_size(M, K)


def bl_norm_backward(dy, x, weight, mean, rstd, dx=None, dweight=None, dbias=None, workspace=None, rms=False,
                     accumulate=False, stream=None):
    """N2: dx [M,K], dweight, dbias [K] (each may be None) of N1. x: the forward's
    input, or the Act8 that the forward saved."""
    saved8, x = (x, None) if isinstance(x, Act8) else (None, x)
    codes, scales = (None, None) if saved8 is None else (saved8.codes, saved8.scales)
    status = _quick().norm_backward(dy, x, codes, scales, weight, mean, rstd, dx, dweight, dbias, workspace, rms,
                                    accumulate, stream)
    if status is not None:
        return _check(status, "bl_norm_backward")
    M, K = dy.shape
    cur = _device(dy, "dy")
    dt = _dtype_code(dy, "dy")
    param = weight if weight is not None else dweight if dweight is not None else dbias
    pdt, ptype = (BL_F32, None) if param is None else (_dtype_code(param, "weight, dweight or dbias"), param.dtype)
    p = _pointers(cur, ((dy, dy.dtype, (M, K), "dy"), (x, dy.dtype, (M, K), "x"), *_act8_specs(saved8, M, K, "x"),
                        (weight, ptype, (K,), "weight"), (mean, torch.float32, (M,), "mean"),
                        (rstd, torch.float32, (M,), "rstd"), (dx, dy.dtype, (M, K), "dx"),
                        (dweight, ptype, (K,), "dweight"), (dbias, ptype, (K,), "dbias")))
    ws, n = _scratch(cur, workspace)
    _check(load_library().bl_norm_backward(*p[:4], dt, p[4], pdt, p[5], p[6], M, K, 1 if rms else 0, *p[7:10],
                                           1 if accumulate else 0, ws, n, _stream_of(stream, cur)),
           "bl_norm_backward")


def bl_swiglu_forward(gate, up, y, gate8: Act8 | None = None, up8: Act8 | None = None, stream=None):
    """U1: y [M,K] = silu(gate) * up (bf16|f32); gate8, up8 (both or neither)
    receive the 8-bit forms of gate and up."""
    if (gate8 is None) != (up8 is None):
        raise ValueError("gate8 and up8 go together")
    saved = (None,) * 4 if gate8 is None else (gate8.codes, gate8.scales, up8.codes, up8.scales)
    status = _quick().swiglu_forward(gate, up, y, *saved, stream)
    if status is not None:
        return _check(status, "bl_swiglu_forward")
    M, K = gate.shape
    cur = _device(gate, "gate")
    dt = _dtype_code(gate, "gate")
    p = _pointers(cur, ((gate, gate.dtype, (M, K), "gate"), (up, gate.dtype, (M, K), "up"), (y, gate.dtype, (M, K), "y"),
                        *_act8_specs(gate8, M, K, "gate8"), *_act8_specs(up8, M, K, "up8")))
    _check(load_library().bl_swiglu_forward(p[0], p[1], dt, M, K, *p[2:7], _stream_of(stream, cur)),
           "bl_swiglu_forward")


def bl_swiglu_backward(dy, gate8: Act8, up8: Act8, dgate, dup, stream=None):
    """U2: dgate, dup [M,K] of U1 from the 8-bit forms of gate and up."""
    status = _quick().swiglu_backward(dy, gate8.codes, gate8.scales, up8.codes, up8.scales, dgate, dup, stream)
    if status is not None:
        return _check(status, "bl_swiglu_backward")
    M, K = dy.shape
    cur = _device(dy, "dy")
    dt = _dtype_code(dy, "dy")
    p = _pointers(cur, ((dy, dy.dtype, (M, K), "dy"), *_act8_specs(gate8, M, K, "gate8"),
                        *_act8_specs(up8, M, K, "up8"), (dgate, dy.dtype, (M, K), "dgate"),
                        (dup, dy.dtype, (M, K), "dup")))
    _check(load_library().bl_swiglu_backward(*p[:5], dt, M, K, p[5], p[6], _stream_of(stream, cur)),
           "bl_swiglu_backward")


# ----------------------------------------------------------------- around the 8-bit products; the gradients' norm

def bl_norm_quant_forward(x, residual, weight, eps, sum, rstd, xq, sx, stream=None):
    """Q1: sum [M,K] = x + residual (of the residual's type; both None: x is the
    stream), then xq [M,K] int8 and sx [M] f32, the 8-bit form of the RMS norm of
    sum with gain weight [K] (bf16|f32, may be None); rstd [M] f32 for Q2."""
    status = _quick().norm_quant_forward(x, residual, weight, eps, sum, rstd, xq, sx, stream)
    if status is not None:
        return _check(status, "bl_norm_quant_forward")
    M, K = x.shape
    cur = _device(x, "x")
    dt = _dtype_code(x, "x")
    stype, sdt = (x.dtype, dt) if residual is None else (residual.dtype, _dtype_code(residual, "residual"))
    pdt, ptype = (BL_F32, None) if weight is None else (_dtype_code(weight, "weight"), weight.dtype)
    p = _pointers(cur, ((x, x.dtype, (M, K), "x"), (residual, stype, (M, K), "residual"), (weight, ptype, (K,), "weight"),
                        (sum, stype, (M, K), "sum"), (rstd, torch.float32, (M,), "rstd"), (xq, torch.int8, (M, K), "xq"),
                        (sx, torch.float32, (M,), "sx")))
    _check(load_library().bl_norm_quant_forward(p[0], dt, p[1], sdt, p[2], pdt, M, K, eps, *p[3:], _stream_of(stream, cur)),
           "bl_norm_quant_forward")


def bl_norm_quant_backward_workspace_size(M: int, K: int) -> int:
    return load_library().bl_norm_quant_backward_workspace_size(M, K)


def bl_norm_quant_backward(dy, dsum, sum, weight, rstd, dx=None, dresidual=None, dweight=None, workspace=None,
                           accumulate=False, stream=None):
    """Q2: dx [M,K] (of x's type), dresidual [M,K] (of the stream's) and dweight
    [K] of Q1 (each may be None), given dy [M,K] (bf16|f32) and dsum [M,K], the
    gradient of the stream behind the addition (None: zero)."""
    status = _quick().norm_quant_backward(dy, dsum, sum, weight, rstd, dx, dresidual, dweight, workspace, accumulate,
                                          stream)
    if status is not None:
        return _check(status, "bl_norm_quant_backward")
    M, K = dy.shape
    cur = _device(dy, "dy")
    ddt, sdt = _dtype_code(dy, "dy"), _dtype_code(sum, "sum")
    xdt, xtype = (sdt, None) if dx is None else (_dtype_code(dx, "dx"), dx.dtype)
    param = weight if weight is not None else dweight
    pdt, ptype = (BL_F32, None) if param is None else (_dtype_code(param, "weight or dweight"), param.dtype)
    p = _pointers(cur, ((dy, dy.dtype, (M, K), "dy"), (dsum, sum.dtype, (M, K), "dsum"), (sum, sum.dtype, (M, K), "sum"),
                        (weight, ptype, (K,), "weight"), (rstd, torch.float32, (M,), "rstd"), (dx, xtype, (M, K), "dx"),
                        (dresidual, sum.dtype, (M, K), "dresidual"), (dweight, ptype, (K,), "dweight")))
    ws, n = _scratch(cur, workspace)
    _check(load_library().bl_norm_quant_backward(p[0], ddt, p[1], p[2], sdt, p[3], pdt, p[4], M, K, p[6], p[5], xdt, p[7],
                                                 1 if accumulate else 0, ws, n, _stream_of(stream, cur)),
           "bl_norm_quant_backward")


def bl_int8_linear_forward(xq, sx, wq, sw, y, stream=None):
    """L1: y [M,N] (bf16|f32) = (xq [M,K] . wq [N,K]^T) * sx [M] * sw [N], the codes int8."""
    status = _quick().int8_linear_forward(xq, sx, wq, sw, y, stream)
    if status is not None:
        return _check(status, "bl_int8_linear_forward")
    M, K = xq.shape
    N = wq.shape[0]
    cur = _device(xq, "xq")
    dt = _dtype_code(y, "y")
    p = _pointers(cur, ((xq, torch.int8, (M, K), "xq"), (sx, torch.float32, (M,), "sx"), (wq, torch.int8, (N, K), "wq"),
                        (sw, torch.float32, (N,), "sw"), (y, y.dtype, (M, N), "y")))
    _check(load_library().bl_int8_linear_forward(*p[:4], M, N, K, p[4], dt, _stream_of(stream, cur)),
           "bl_int8_linear_forward")


def bl_int8_linear_backward_workspace_size(M: int, N: int, K: int) -> int:
    return load_library().bl_int8_linear_backward_workspace_size(M, N, K)


def bl_int8_linear_backward(dY, xq, sx, wq, sw, dX=None, dW=None, accumulate_dW=False, stream=None, workspace=None):
    """L2: dX [M,K] bf16 and dW [N,K] (bf16|f32) of L1 (each may be None), given
    dY [M,N] bf16; the operands' codes taken straight through as their values."""
    status = _quick().int8_linear_backward(dY, xq, sx, wq, sw, dX, dW, accumulate_dW, stream, workspace)
    if status is not None:
        return _check(status, "bl_int8_linear_backward")
    M, N = dY.shape
    K = xq.shape[1]
    cur = _device(dY, "dY")
    dwdt, wtype = (BL_BF16, None) if dW is None else (_dtype_code(dW, "dW"), dW.dtype)
    p = _pointers(cur, ((dY, torch.bfloat16, (M, N), "dY"), (xq, torch.int8, (M, K), "xq"), (sx, torch.float32, (M,), "sx"),
                        (wq, torch.int8, (N, K), "wq"), (sw, torch.float32, (N,), "sw"),
                        (dX, torch.bfloat16, (M, K), "dX"), (dW, wtype, (N, K), "dW")))
    ws, n = _scratch(cur, workspace)
    _check(load_library().bl_int8_linear_backward(*p[:5], M, N, K, p[5], p[6], dwdt, 1 if accumulate_dW else 0, ws, n,
                                                  _stream_of(stream, cur)), "bl_int8_linear_backward")


class _Tensor(ctypes.Structure):
    _fields_ = [("data", _VP), ("numel", _I64), ("dtype", _I32)]


def bl_grad_norm_workspace_size(count: int) -> int:
    return load_library().bl_grad_norm_workspace_size(count)


def _tensor_list(cur, tensors, name):
    """The bl_tensor array of a list of tensors of any shapes (bf16|f32)."""
    out = (_Tensor * max(len(tensors), 1))()
    for i, t in enumerate(tensors):
        dt = _dtype_code(t, f"{name}[{i}]")
        address, = _pointers(cur, ((t, t.dtype, t.shape, f"{name}[{i}]"),))
        out[i] = _Tensor(address, t.numel(), dt)
    return out


def bl_grad_norm(grads, norm, workspace, stream=None):
    """C1: norm [1] f32 = the 2-norm over all of grads, a list of tensors of any
    shapes (bf16|f32, mixed at will)."""
    status = _quick().grad_norm(grads, norm, workspace, stream)
    if status is not None:
        return _check(status, "bl_grad_norm")
    grads = list(grads)
    cur = _device(norm, "norm")
    p = _pointers(cur, ((norm, torch.float32, (1,), "norm"),))
    ws, n = _scratch(cur, workspace)
    _check(load_library().bl_grad_norm(_tensor_list(cur, grads, "grads"), len(grads), p[0], ws, n, _stream_of(stream, cur)),
           "bl_grad_norm")


def bl_clip_grads(grads, max_norm, norm, workspace, out=None, stream=None):
    """C2: norm [1] f32 as C1, and grads scaled by max_norm / norm where norm is
    above max_norm: in place, or into out, a list of tensors like grads."""
    status = _quick().clip_grads(grads, max_norm, norm, workspace, out, stream)
    if status is not None:
        return _check(status, "bl_clip_grads")
    grads = list(grads)
    cur = _device(norm, "norm")
    p = _pointers(cur, ((norm, torch.float32, (1,), "norm"),))
    ws, n = _scratch(cur, workspace)
    tensors, to = _tensor_list(cur, grads, "grads"), None
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError(f"out has {len(out)} tensors, grads {len(grads)}")
        to = (_VP * max(len(out), 1))(*_pointers(cur, [(o, g.dtype, g.shape, f"out[{i}]")
                                                       for i, (o, g) in enumerate(zip(out, grads))]))
    _check(load_library().bl_clip_grads(tensors, to, len(grads), max_norm, p[0], ws, n, _stream_of(stream, cur)),
           "bl_clip_grads")


@dataclass
class XentBuffers:
    """Device buffers of X1 and (backward) X2 (caller-owned, reused); one
    workspace serves both calls, in either order on one stream. A call of fewer
    tokens takes their first rows and the same workspace and dW."""
    loss: torch.Tensor
    lse: torch.Tensor
    workspace: torch.Tensor
    dH: torch.Tensor | None = None
    dW: torch.Tensor | None = None

    @staticmethod
    def allocate(M, V, K, dw_dtype=torch.bfloat16, backward=True, device="cuda"):
        ws = bl_linear_xent_forward_workspace_size(M, V, K)
        if backward:
            ws = max(ws, bl_linear_xent_backward_workspace_size(M, V, K, dw_dtype))
        return XentBuffers(
            loss=torch.empty(M, dtype=torch.float32, device=device),
            lse=torch.empty(M, dtype=torch.float32, device=device),
            workspace=torch.empty(max(ws, 16), dtype=torch.uint8, device=device),
            dH=torch.empty((M, K), dtype=torch.bfloat16, device=device) if backward else None,
            dW=torch.empty((V, K), dtype=dw_dtype, device=device) if backward else None,
        )


@dataclass
class NormBuffers:
    """Device buffers of N1 and N2 (caller-owned, reused)."""
    y: torch.Tensor
    mean: torch.Tensor | None
    rstd: torch.Tensor
    saved8: Act8 | None
    dx: torch.Tensor
    dweight: torch.Tensor
    dbias: torch.Tensor | None
    workspace: torch.Tensor

    @staticmethod
    def allocate(M, K, dtype=torch.bfloat16, p_dtype=torch.float32, rms=False, bias=False, saved8=False,
                 device="cuda"):
        def empty(shape, dt):
            return torch.empty(shape, dtype=dt, device=device)
        return NormBuffers(
            y=empty((M, K), dtype), mean=None if rms else empty(M, torch.float32), rstd=empty(M, torch.float32),
            saved8=Act8.allocate(M, K, device) if saved8 else None,
            dx=empty((M, K), dtype), dweight=empty(K, p_dtype), dbias=empty(K, p_dtype) if bias else None,
            workspace=empty(max(bl_norm_backward_workspace_size(M, K), 16), torch.uint8))


@dataclass
class SwigluBuffers:
    """Device buffers of U1 and U2 (caller-owned, reused)."""
    y: torch.Tensor
    gate8: Act8
    up8: Act8
    dgate: torch.Tensor
    dup: torch.Tensor

    @staticmethod
    def allocate(M, K, dtype=torch.bfloat16, device="cuda"):
        def empty():
            return torch.empty((M, K), dtype=dtype, device=device)
        return SwigluBuffers(y=empty(), gate8=Act8.allocate(M, K, device), up8=Act8.allocate(M, K, device),
                             dgate=empty(), dup=empty())


@dataclass
class NormQuantBuffers:
    """Device buffers of Q1 and (backward) Q2 (caller-owned, reused). dx is there
    where x has another type than the stream; else dresidual serves both."""
    sum: torch.Tensor
    rstd: torch.Tensor
    xq: torch.Tensor
    sx: torch.Tensor
    dx: torch.Tensor | None = None
    dresidual: torch.Tensor | None = None
    dweight: torch.Tensor | None = None
    workspace: torch.Tensor | None = None

    @staticmethod
    def allocate(M, K, x_dtype=torch.bfloat16, s_dtype=torch.bfloat16, p_dtype=torch.float32, backward=True,
                 device="cuda"):
        def empty(shape, dt):
            return torch.empty(shape, dtype=dt, device=device)
        b = NormQuantBuffers(sum=empty((M, K), s_dtype), rstd=empty(M, torch.float32), xq=empty((M, K), torch.int8),
                             sx=empty(M, torch.float32))
        if backward:
            b.dx = empty((M, K), x_dtype) if x_dtype != s_dtype else None
            b.dresidual, b.dweight = empty((M, K), s_dtype), empty(K, p_dtype)
            b.workspace = empty(max(bl_norm_quant_backward_workspace_size(M, K), 16), torch.uint8)
        return b


@dataclass
class Int8LinearBuffers:
    """Device buffers of L1 and (backward) L2 (caller-owned, reused)."""
    y: torch.Tensor
    dX: torch.Tensor | None = None
    dW: torch.Tensor | None = None
    workspace: torch.Tensor | None = None

    @staticmethod
    def allocate(M, N, K, y_dtype=torch.bfloat16, dw_dtype=torch.bfloat16, backward=True, device="cuda"):
        def empty(shape, dt):
            return torch.empty(shape, dtype=dt, device=device)
        b = Int8LinearBuffers(y=empty((M, N), y_dtype))
        if backward:
            b.dX, b.dW = empty((M, K), torch.bfloat16), empty((N, K), dw_dtype)
            b.workspace = empty(max(bl_int8_linear_backward_workspace_size(M, N, K), 16), torch.uint8)
        return b


# ----------------------------------------------------------------- one whole step

@dataclass
class StepBuffers:
    """Device buffers of one BitLinear fwd+bwd (caller-owned, reused)."""
    w_packed: torch.Tensor
    gamma: torch.Tensor
    workspace: torch.Tensor
    xq: torch.Tensor
    sx: torch.Tensor
    y: torch.Tensor
    dX: torch.Tensor
    dW: torch.Tensor
    bwd_workspace: torch.Tensor | None = None  # x_hat scratch of the backward (bl_backward_ws)

    @staticmethod
    def allocate(M, N, K, dw_dtype=torch.bfloat16, device="cuda"):
        ws = bl_quantize_weight_workspace_size(N, K)
        return StepBuffers(
            w_packed=torch.empty((N, K // 4), dtype=torch.uint8, device=device),
            gamma=torch.empty(1, dtype=torch.float32, device=device),
            workspace=torch.empty(max(ws, 16), dtype=torch.uint8, device=device),
            xq=torch.empty((M, K), dtype=torch.int8, device=device),
            sx=torch.empty(M, dtype=torch.float32, device=device),
            y=torch.empty((M, N), dtype=torch.bfloat16, device=device),
            dX=torch.empty((M, K), dtype=torch.bfloat16, device=device),
            dW=torch.empty((N, K), dtype=dw_dtype, device=device),
            bwd_workspace=torch.empty(max(bl_backward_workspace_size(M, N, K), 16), dtype=torch.uint8, device=device),
        )


def bitlinear_step(x, W, dY, bufs: StepBuffers, stream=None):
    """One BitLinear forward + backward: S1 + S2 (bl_quantize) -> S3 -> S4 (four kernel launches)."""
    bl_quantize(W, x, bufs.w_packed, bufs.gamma, bufs.xq, bufs.sx, bufs.workspace, stream)
    bl_forward(bufs.xq, bufs.sx, bufs.w_packed, bufs.gamma, bufs.y, None, stream)
    bl_backward(dY, bufs.xq, bufs.sx, bufs.w_packed, bufs.gamma, bufs.dX, bufs.dW, False, stream,
                workspace=bufs.bwd_workspace)
