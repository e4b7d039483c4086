// C ABI of the BitLinear library: argument validation on the host, dispatch
// to the kernels, and the per-device error word that bounded device waits
// write on timeout. See include/bitlinear.h for the contract of each call.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <memory>
#include <new>

#include "../../include/bitlinear.h"
#include "bl_internal.h"

namespace {

__device__ int g_device_error = 0;

thread_local char g_msg[256] = "";

bl_status fail(bl_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return s;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Device address of the error word on the current device. Looked up on every
// call (a host-side table lookup once the module is loaded): a cached address
// would go stale if the caller reset the device and the module were loaded
// again at another address.
int* device_error_ptr() {
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) return nullptr;
  return static_cast<int*>(p);
}

// Checks the current device is sm_100 and returns its error word.
bl_status current_device(int** err) {
  static int arch_ok[64] = {};  // 0 unknown, 1 ok, 2 bad
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(BL_ERR_CUDA, "cudaGetDevice failed");
  if (dev < 0 || dev >= 64) return fail(BL_ERR_CUDA, "device index %d out of range", dev);
  if (arch_ok[dev] == 0) {
    int major = 0, minor = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    arch_ok[dev] = (major == 10 && minor == 0) ? 1 : 2;
  }
  if (arch_ok[dev] != 1) return fail(BL_ERR_ARCH, "device %d is not sm_100", dev);
  *err = device_error_ptr();
  if (!*err) return fail(BL_ERR_CUDA, "cannot resolve the device error word");
  return BL_OK;
}

bl_status check_k(int64_t K) {
  if (K < 32 || K % 32 != 0) return fail(BL_ERR_UNSUPPORTED_SHAPE, "K=%lld must be a positive multiple of 32", (long long)K);
  if (K > (int64_t(1) << 30)) return fail(BL_ERR_UNSUPPORTED_SHAPE, "K=%lld too large", (long long)K);
  return BL_OK;
}

bl_status cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return BL_OK;
  const char* detail = bl::launch_detail();
  bl_status s = fail(BL_ERR_CUDA, "%s: %s%s%s", what, cudaGetErrorString(e), detail[0] ? "; " : "", detail);
  bl::clear_launch_detail();
  return s;
}

// Memory that a clipped gradient is written to.
struct Span {
  uintptr_t b, e;
  bool operator<(const Span& o) const { return b < o.b; }
};

// The list as the launches take it. `host_out` null: in place.
bl_status tensor_list(const bl_tensor* x, void* const* host_out, int64_t count, bool write, bl::ClipTensor* out, Span* spans) {
  int64_t total = 0, nspans = 0;
  bool moved = false;
  for (int64_t i = 0; i < count; ++i) {
    const bl_tensor& t = x[i];
    if (t.dtype != BL_BF16 && t.dtype != BL_F32) return fail(BL_ERR_DTYPE, "dtype %d of tensor %lld", (int)t.dtype, (long long)i);
    if (t.numel < 0) return fail(BL_ERR_INVALID_ARG, "tensor %lld has %lld elements", (long long)i, (long long)t.numel);
    if (t.numel > (int64_t(1) << 40) - total)
      return fail(BL_ERR_UNSUPPORTED_SHAPE, "more than 2^40 elements (at tensor %lld)", (long long)i);
    total += t.numel;
    void* to = !write ? nullptr : host_out ? host_out[i] : t.data;
    out[i] = {t.data, to, t.numel, t.dtype == BL_F32};
    if (t.numel == 0) continue;
    const uintptr_t size = t.dtype == BL_F32 ? 4 : 2;
    if (!t.data || (write && !to)) return fail(BL_ERR_INVALID_ARG, "null pointer (tensor %lld)", (long long)i);
    if (reinterpret_cast<uintptr_t>(t.data) % size != 0 || reinterpret_cast<uintptr_t>(to) % size != 0)
      return fail(BL_ERR_ALIGNMENT, "tensor %lld starts inside an element", (long long)i);
    if (!write) continue;
    moved = moved || to != t.data;
    const uintptr_t b = reinterpret_cast<uintptr_t>(to);
    spans[nspans++] = {b, b + static_cast<uintptr_t>(t.numel) * size};
  }
  if (!write) return BL_OK;
  std::sort(spans, spans + nspans);
  for (int64_t i = 1; i < nspans; ++i)
    if (spans[i].b < spans[i - 1].e) return fail(BL_ERR_INVALID_ARG, "two tensors are written to the same memory");
  // an input may share memory with its own output, from the same place, and with no other
  for (int64_t i = 0; moved && i < count; ++i) {
    if (x[i].numel == 0) continue;
    const uintptr_t b = reinterpret_cast<uintptr_t>(x[i].data), e = b + static_cast<uintptr_t>(x[i].numel) * (out[i].f32 ? 4 : 2);
    const Span* s = std::upper_bound(spans, spans + nspans, Span{b, e});
    if (s > spans && s[-1].e > b) --s;
    for (; s < spans + nspans && s->b < e; ++s)
      if (out[i].in != out[i].out || s->b != b)
        return fail(BL_ERR_INVALID_ARG, "tensor %lld overlaps what is written", (long long)i);
  }
  return BL_OK;
}

bl_status clip(const bl_tensor* host_grads, void* const* host_out, int64_t count, bool write, double most, float* norm,
               void* workspace, size_t workspace_bytes, void* stream, const char* what) {
  if (count < 0 || (count > 0 && !host_grads)) return fail(BL_ERR_INVALID_ARG, "count=%lld, or no list", (long long)count);
  if (count > (int64_t(1) << 20)) return fail(BL_ERR_UNSUPPORTED_SHAPE, "more than 2^20 tensors");
  if (write && !(most >= 0.0)) return fail(BL_ERR_INVALID_ARG, "max_norm must be >= 0");
  if (!norm) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (reinterpret_cast<uintptr_t>(norm) % 4 != 0) return fail(BL_ERR_ALIGNMENT, "norm must be 4-byte aligned");
  std::unique_ptr<bl::ClipTensor[]> list(new (std::nothrow) bl::ClipTensor[count + 1]);
  std::unique_ptr<Span[]> spans(new (std::nothrow) Span[write ? count + 1 : 1]);
  if (!list || !spans) return fail(BL_ERR_INVALID_ARG, "no host memory for a list of %lld", (long long)count);
  if (bl_status s = tensor_list(host_grads, host_out, count, write, list.get(), spans.get())) return s;
  for (int64_t i = 0; i < count; ++i) {
    const uintptr_t n = reinterpret_cast<uintptr_t>(norm), bytes = static_cast<uintptr_t>(list[i].n) * (list[i].f32 ? 4 : 2);
    for (const void* t : {list[i].in, static_cast<const void*>(list[i].out)}) {
      const uintptr_t b = reinterpret_cast<uintptr_t>(t);
      if (t && b < n + 4 && n < b + bytes) return fail(BL_ERR_INVALID_ARG, "norm lies in tensor %lld", (long long)i);
    }
  }
  const size_t need = bl::grad_norm_workspace_bytes(count);
  if (count > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return fail(BL_ERR_WORKSPACE, "workspace needs %zu bytes, 16-byte aligned", need);
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_clip(list.get(), count, norm, most, write, workspace, static_cast<cudaStream_t>(stream)), what);
}

}  // namespace

extern "C" {

int bl_version(void) { return (1 << 16) | 0; }

const char* bl_status_string(bl_status s) {
  switch (s) {
    case BL_OK: return "BL_OK";
    case BL_ERR_INVALID_ARG: return "BL_ERR_INVALID_ARG";
    case BL_ERR_UNSUPPORTED_SHAPE: return "BL_ERR_UNSUPPORTED_SHAPE";
    case BL_ERR_DTYPE: return "BL_ERR_DTYPE";
    case BL_ERR_ALIGNMENT: return "BL_ERR_ALIGNMENT";
    case BL_ERR_ARCH: return "BL_ERR_ARCH";
    case BL_ERR_CUDA: return "BL_ERR_CUDA";
    case BL_ERR_TIMEOUT: return "BL_ERR_TIMEOUT";
    case BL_ERR_WORKSPACE: return "BL_ERR_WORKSPACE";
  }
  return "BL_ERR_UNKNOWN";
}

const char* bl_last_error_message(void) { return g_msg; }

size_t bl_quantize_weight_workspace_size(int64_t N, int64_t K) {
  if (N <= 0 || K <= 0) return 0;
  return bl::quantize_workspace_bytes();
}

bl_status bl_quantize_weight(const void* W, bl_dtype w_dtype, int64_t N, int64_t K, uint8_t* w_packed,
                             float* gamma, void* workspace, size_t workspace_bytes, void* stream) {
  g_msg[0] = 0;
  if (N < 1) return fail(BL_ERR_INVALID_ARG, "N=%lld must be >= 1", (long long)N);
  if (bl_status s = check_k(K)) return s;
  if (w_dtype != BL_BF16 && w_dtype != BL_F32) return fail(BL_ERR_DTYPE, "w_dtype %d", (int)w_dtype);
  if (!W || !w_packed || !gamma) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(W) || !aligned16(w_packed) || !aligned16(gamma))
    return fail(BL_ERR_ALIGNMENT, "W, w_packed and gamma must be 16-byte aligned");
  const size_t need = bl_quantize_weight_workspace_size(N, K);
  if (!workspace || workspace_bytes < need || !aligned16(workspace))
    return fail(BL_ERR_WORKSPACE, "workspace needs %zu bytes, 16-byte aligned", need);
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_quantize_weight(W, w_dtype == BL_F32, N, K, w_packed, gamma, workspace, err,
                                                static_cast<cudaStream_t>(stream)),
                     "bl_quantize_weight launch");
}

bl_status bl_quantize_weight_noalloc(const void* W, bl_dtype w_dtype, int64_t N, int64_t K, uint8_t* w_packed,
                                     float* gamma, void* stream) {
  g_msg[0] = 0;
  if (N < 1) return fail(BL_ERR_INVALID_ARG, "N=%lld must be >= 1", (long long)N);
  if (bl_status s = check_k(K)) return s;
  if (w_dtype != BL_BF16 && w_dtype != BL_F32) return fail(BL_ERR_DTYPE, "w_dtype %d", (int)w_dtype);
  if (!W || !w_packed || !gamma) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(W) || !aligned16(w_packed) || !aligned16(gamma))
    return fail(BL_ERR_ALIGNMENT, "W, w_packed and gamma must be 16-byte aligned");
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_quantize_weight_noalloc(W, w_dtype == BL_F32, N, K, w_packed, gamma, err,
                                                        static_cast<cudaStream_t>(stream)),
                     "bl_quantize_weight_noalloc launch");
}

bl_status bl_quantize_act(const void* x, int64_t M, int64_t K, int8_t* xq, float* sx, void* stream) {
  g_msg[0] = 0;
  if (M < 0) return fail(BL_ERR_INVALID_ARG, "M=%lld must be >= 0", (long long)M);
  if (bl_status s = check_k(K)) return s;
  if (M == 0) return BL_OK;
  if (!x || !xq || !sx) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(x) || !aligned16(xq) || !aligned16(sx))
    return fail(BL_ERR_ALIGNMENT, "x, xq and sx must be 16-byte aligned");
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_quantize_act(x, M, K, xq, sx, static_cast<cudaStream_t>(stream)),
                     "bl_quantize_act launch");
}

bl_status bl_quantize(const void* W, bl_dtype w_dtype, int64_t N, int64_t K, const void* x, int64_t M,
                      uint8_t* w_packed, float* gamma, int8_t* xq, float* sx, void* workspace,
                      size_t workspace_bytes, void* stream) {
  g_msg[0] = 0;
  if (N < 1) return fail(BL_ERR_INVALID_ARG, "N=%lld must be >= 1", (long long)N);
  if (M < 0) return fail(BL_ERR_INVALID_ARG, "M=%lld must be >= 0", (long long)M);
  if (bl_status s = check_k(K)) return s;
  if (w_dtype != BL_BF16 && w_dtype != BL_F32) return fail(BL_ERR_DTYPE, "w_dtype %d", (int)w_dtype);
  if (!W || !w_packed || !gamma) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (M > 0 && (!x || !xq || !sx)) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(W) || !aligned16(w_packed) || !aligned16(gamma) || (x && !aligned16(x)) ||
      (xq && !aligned16(xq)) || (sx && !aligned16(sx)))
    return fail(BL_ERR_ALIGNMENT, "tensors must be 16-byte aligned");
  const size_t need = bl_quantize_weight_workspace_size(N, K);
  if (!workspace || workspace_bytes < need || !aligned16(workspace))
    return fail(BL_ERR_WORKSPACE, "workspace needs %zu bytes, 16-byte aligned", need);
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_quantize(W, w_dtype == BL_F32, N, K, x, M, w_packed, gamma, workspace, xq, sx, err,
                                         static_cast<cudaStream_t>(stream)),
                     "bl_quantize launch");
}

bl_status bl_forward(const int8_t* xq, const float* sx, const uint8_t* w_packed, const float* gamma, int64_t M,
                     int64_t N, int64_t K, void* y, int32_t* debug_acc, void* stream) {
  g_msg[0] = 0;
  if (M < 0 || N < 1) return fail(BL_ERR_INVALID_ARG, "M=%lld, N=%lld", (long long)M, (long long)N);
  if (bl_status s = check_k(K)) return s;
  if (M > (int64_t(1) << 30) || N > (int64_t(1) << 30)) return fail(BL_ERR_UNSUPPORTED_SHAPE, "M or N too large");
  if (M == 0) return BL_OK;
  if (!xq || !sx || !w_packed || !gamma || !y) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(xq) || !aligned16(sx) || !aligned16(w_packed) || !aligned16(gamma) || !aligned16(y) ||
      (debug_acc && !aligned16(debug_acc)))
    return fail(BL_ERR_ALIGNMENT, "tensors must be 16-byte aligned");
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_forward(xq, sx, w_packed, gamma, M, N, K, y, debug_acc, err,
                                        static_cast<cudaStream_t>(stream)),
                     "bl_forward launch");
}

// The checks and the launch shared by bl_backward, bl_backward_signs and
// their workspace forms. dw_signs: dW receives sign words.
static bl_status backward_common(const void* dY, const int8_t* xq, const float* sx, const uint8_t* w_packed,
                                 const float* gamma, int64_t M, int64_t N, int64_t K, void* dX, void* dW,
                                 bl_dtype dw_dtype, int accumulate_dW, int dw_signs, void* workspace,
                                 size_t workspace_bytes, void* stream, const char* what) {
  g_msg[0] = 0;
  if (M < 0 || N < 1) return fail(BL_ERR_INVALID_ARG, "M=%lld, N=%lld", (long long)M, (long long)N);
  if (bl_status s = check_k(K)) return s;
  if (N % 8 != 0) return fail(BL_ERR_UNSUPPORTED_SHAPE, "N=%lld must be a multiple of 8", (long long)N);
  if (M > (int64_t(1) << 30) || N > (int64_t(1) << 30)) return fail(BL_ERR_UNSUPPORTED_SHAPE, "M or N too large");
  if (dw_signs) {
    if (!dW) return fail(BL_ERR_INVALID_ARG, "null dw_sign_words");
  } else {
    if (dW && dw_dtype != BL_BF16 && dw_dtype != BL_F32) return fail(BL_ERR_DTYPE, "dw_dtype %d", (int)dw_dtype);
    if (!dX && !dW) return BL_OK;
  }
  if (M > 0 && !dY) return fail(BL_ERR_INVALID_ARG, "null dY");
  if (dX && (!w_packed || !gamma)) return fail(BL_ERR_INVALID_ARG, "dX needs w_packed and gamma");
  if (dW && M > 0 && (!xq || !sx)) return fail(BL_ERR_INVALID_ARG, "dW needs xq and sx");
  if ((dY && !aligned16(dY)) || (xq && !aligned16(xq)) || (sx && !aligned16(sx)) ||
      (w_packed && !aligned16(w_packed)) || (gamma && !aligned16(gamma)) || (dX && !aligned16(dX)) ||
      (dW && !aligned16(dW)))
    return fail(BL_ERR_ALIGNMENT, "tensors must be 16-byte aligned");
  if (workspace && bl::backward_uses_xhat(N)) {
    const size_t need = bl_backward_workspace_size(M, N, K);
    if (workspace_bytes < need || !aligned16(workspace))
      return fail(BL_ERR_WORKSPACE, "workspace needs %zu bytes, 16-byte aligned", need);
  }
  // x_hat is only made when dW is computed from tokens and worth it
  void* xhat = (workspace && dW && M > 0 && bl::backward_uses_xhat(N)) ? workspace : nullptr;
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_backward(dY, xq, sx, w_packed, gamma, M, N, K, dX, dW,
                                         dw_signs ? 0 : dw_dtype == BL_F32, dw_signs ? 0 : accumulate_dW != 0,
                                         dw_signs, xhat, err, static_cast<cudaStream_t>(stream)),
                     what);
}

size_t bl_backward_workspace_size(int64_t M, int64_t N, int64_t K) {
  return (M > 0 && K > 0 && bl::backward_uses_xhat(N)) ? static_cast<size_t>(M) * static_cast<size_t>(K) * 2 : 0;
}

bl_status bl_backward(const void* dY, const int8_t* xq, const float* sx, const uint8_t* w_packed,
                      const float* gamma, int64_t M, int64_t N, int64_t K, void* dX, void* dW, bl_dtype dw_dtype,
                      int accumulate_dW, void* stream) {
  return backward_common(dY, xq, sx, w_packed, gamma, M, N, K, dX, dW, dw_dtype, accumulate_dW, 0, nullptr, 0,
                         stream, "bl_backward launch");
}

bl_status bl_backward_ws(const void* dY, const int8_t* xq, const float* sx, const uint8_t* w_packed,
                         const float* gamma, int64_t M, int64_t N, int64_t K, void* dX, void* dW, bl_dtype dw_dtype,
                         int accumulate_dW, void* workspace, size_t workspace_bytes, void* stream) {
  return backward_common(dY, xq, sx, w_packed, gamma, M, N, K, dX, dW, dw_dtype, accumulate_dW, 0, workspace,
                         workspace_bytes, stream, "bl_backward_ws launch");
}

bl_status bl_backward_signs(const void* dY, const int8_t* xq, const float* sx, const uint8_t* w_packed,
                            const float* gamma, int64_t M, int64_t N, int64_t K, void* dX, uint32_t* dw_sign_words,
                            void* stream) {
  return backward_common(dY, xq, sx, w_packed, gamma, M, N, K, dX, dw_sign_words, BL_BF16, 0, 1, nullptr, 0, stream,
                         "bl_backward_signs launch");
}

bl_status bl_backward_signs_ws(const void* dY, const int8_t* xq, const float* sx, const uint8_t* w_packed,
                               const float* gamma, int64_t M, int64_t N, int64_t K, void* dX,
                               uint32_t* dw_sign_words, void* workspace, size_t workspace_bytes, void* stream) {
  return backward_common(dY, xq, sx, w_packed, gamma, M, N, K, dX, dw_sign_words, BL_BF16, 0, 1, workspace,
                         workspace_bytes, stream, "bl_backward_signs_ws launch");
}

bl_status bl_export_weights(const uint8_t* w_packed, const float* gamma, int64_t N, int64_t K,
                            uint8_t* host_packed, float* host_gamma, void* stream) {
  g_msg[0] = 0;
  if (N < 1) return fail(BL_ERR_INVALID_ARG, "N=%lld must be >= 1", (long long)N);
  if (bl_status s = check_k(K)) return s;
  if (!w_packed || !gamma || !host_packed || !host_gamma) return fail(BL_ERR_INVALID_ARG, "null pointer");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (bl_status s = cuda_status(cudaMemcpyAsync(host_packed, w_packed, static_cast<size_t>(N * (K / 4)),
                                                cudaMemcpyDeviceToHost, st),
                                "export packed"))
    return s;
  if (bl_status s = cuda_status(cudaMemcpyAsync(host_gamma, gamma, sizeof(float), cudaMemcpyDeviceToHost, st),
                                "export gamma"))
    return s;
  return cuda_status(cudaStreamSynchronize(st), "export sync");
}

bl_status bl_sign_pack(const void* dW, bl_dtype dw_dtype, int64_t N, int64_t K, uint32_t* sign_words, void* stream) {
  g_msg[0] = 0;
  if (N < 1) return fail(BL_ERR_INVALID_ARG, "N=%lld must be >= 1", (long long)N);
  if (bl_status s = check_k(K)) return s;
  if (dw_dtype != BL_BF16 && dw_dtype != BL_F32) return fail(BL_ERR_DTYPE, "dw_dtype %d", (int)dw_dtype);
  if (!dW || !sign_words) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(dW) || !aligned16(sign_words)) return fail(BL_ERR_ALIGNMENT, "dW and sign_words must be 16-byte aligned");
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_sign_pack(dW, dw_dtype == BL_F32, N, K, sign_words, static_cast<cudaStream_t>(stream)),
                     "bl_sign_pack");
}

bl_status bl_sign_vote(const uint32_t* sign_words, int ranks, int64_t N, int64_t K, uint8_t* direction,
                       void* stream) {
  g_msg[0] = 0;
  if (N < 1) return fail(BL_ERR_INVALID_ARG, "N=%lld must be >= 1", (long long)N);
  if (bl_status s = check_k(K)) return s;
  if (ranks < 1 || ranks > 127) return fail(BL_ERR_INVALID_ARG, "ranks=%d must be in 1..127", ranks);
  if (!sign_words || !direction) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(sign_words) || !aligned16(direction))
    return fail(BL_ERR_ALIGNMENT, "sign_words and direction must be 16-byte aligned");
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_sign_vote(sign_words, ranks, N, K, direction, static_cast<cudaStream_t>(stream)),
                     "bl_sign_vote");
}

bl_status bl_signsgd_update(void* W, bl_dtype w_dtype, int64_t N, int64_t K, const uint8_t* direction, float lr,
                            void* stream) {
  g_msg[0] = 0;
  if (N < 1) return fail(BL_ERR_INVALID_ARG, "N=%lld must be >= 1", (long long)N);
  if (bl_status s = check_k(K)) return s;
  if (w_dtype != BL_BF16 && w_dtype != BL_F32) return fail(BL_ERR_DTYPE, "w_dtype %d", (int)w_dtype);
  if (!(lr - lr == 0.0f)) return fail(BL_ERR_INVALID_ARG, "lr must be finite");
  if (!W || !direction) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(W) || !aligned16(direction)) return fail(BL_ERR_ALIGNMENT, "W and direction must be 16-byte aligned");
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_signsgd_update(W, w_dtype == BL_F32, N, K, direction, lr,
                                               static_cast<cudaStream_t>(stream)),
                     "bl_signsgd_update");
}

bl_status bl_signsgd_apply(const uint32_t* sign_words, int ranks, void* W, bl_dtype w_dtype, int64_t N, int64_t K,
                           float lr, uint8_t* w_packed, float* gamma, void* workspace, size_t workspace_bytes,
                           void* stream) {
  g_msg[0] = 0;
  if (N < 1) return fail(BL_ERR_INVALID_ARG, "N=%lld must be >= 1", (long long)N);
  if (bl_status s = check_k(K)) return s;
  if (ranks < 1 || ranks > 127) return fail(BL_ERR_INVALID_ARG, "ranks=%d must be in 1..127", ranks);
  if (w_dtype != BL_BF16 && w_dtype != BL_F32) return fail(BL_ERR_DTYPE, "w_dtype %d", (int)w_dtype);
  if (!(lr - lr == 0.0f)) return fail(BL_ERR_INVALID_ARG, "lr must be finite");
  if (!sign_words || !W || !w_packed || !gamma) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(sign_words) || !aligned16(W) || !aligned16(w_packed) || !aligned16(gamma))
    return fail(BL_ERR_ALIGNMENT, "sign_words, W, w_packed and gamma must be 16-byte aligned");
  const size_t need = bl_quantize_weight_workspace_size(N, K);
  if (!workspace || workspace_bytes < need || !aligned16(workspace))
    return fail(BL_ERR_WORKSPACE, "workspace needs %zu bytes, 16-byte aligned", need);
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_signsgd_apply(sign_words, ranks, W, w_dtype == BL_F32, N, K, lr, w_packed, gamma,
                                              workspace, err, static_cast<cudaStream_t>(stream)),
                     "bl_signsgd_apply");
}

// Shape limits of the head cross-entropy (its tile counts and tensor-map
// coordinates fit in 32 bits within them).
static bl_status check_xent(int64_t M, int64_t V, int64_t K) {
  if (M < 0 || V < 1) return fail(BL_ERR_INVALID_ARG, "M=%lld, V=%lld", (long long)M, (long long)V);
  if (K < 8 || K % 8 != 0 || K > 65536)
    return fail(BL_ERR_UNSUPPORTED_SHAPE, "K=%lld must be a multiple of 8 from 8 to 65536", (long long)K);
  if (M > 131072 || V > (int64_t(1) << 24))
    return fail(BL_ERR_UNSUPPORTED_SHAPE, "M=%lld above 131072 or V=%lld above 2^24", (long long)M, (long long)V);
  return BL_OK;
}

size_t bl_linear_xent_forward_workspace_size(int64_t M, int64_t V, int64_t K) {
  g_msg[0] = 0;
  if (M == 0 || check_xent(M, V, K) != BL_OK) return 0;
  return bl::xent_forward_workspace_bytes(M, V, K);
}

size_t bl_linear_xent_backward_workspace_size(int64_t M, int64_t V, int64_t K, bl_dtype dw_dtype) {
  g_msg[0] = 0;
  if (M == 0 || check_xent(M, V, K) != BL_OK || (dw_dtype != BL_BF16 && dw_dtype != BL_F32)) return 0;
  return bl::xent_backward_workspace_bytes(M, V, K, dw_dtype == BL_F32);
}

bl_status bl_linear_xent_forward(const void* h, const void* W, const int64_t* targets, int64_t M, int64_t V,
                                 int64_t K, float* loss, float* lse, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  g_msg[0] = 0;
  if (bl_status s = check_xent(M, V, K)) return s;
  if (M == 0) return BL_OK;
  if (!h || !W || !targets || !loss || !lse) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(h) || !aligned16(W) || !aligned16(targets) || !aligned16(loss) || !aligned16(lse))
    return fail(BL_ERR_ALIGNMENT, "tensors must be 16-byte aligned");
  const size_t need = bl_linear_xent_forward_workspace_size(M, V, K);
  if (!workspace || workspace_bytes < need || !aligned16(workspace))
    return fail(BL_ERR_WORKSPACE, "workspace needs %zu bytes, 16-byte aligned", need);
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_xent_forward(h, W, targets, M, V, K, loss, lse, workspace, err,
                                             static_cast<cudaStream_t>(stream)),
                     "bl_linear_xent_forward launch");
}

bl_status bl_linear_xent_backward(const void* h, const void* W, const int64_t* targets, const float* lse,
                                  const float* dloss, int64_t M, int64_t V, int64_t K, void* dH, void* dW,
                                  bl_dtype dw_dtype, int accumulate_dW, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  g_msg[0] = 0;
  if (bl_status s = check_xent(M, V, K)) return s;
  if (dw_dtype != BL_BF16 && dw_dtype != BL_F32) return fail(BL_ERR_DTYPE, "dw_dtype %d", (int)dw_dtype);
  if (!dH && !dW) return BL_OK;
  if (M == 0 && (!dW || accumulate_dW)) return BL_OK;
  if (M > 0 && (!h || !W || !targets || !lse || !dloss)) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if ((h && !aligned16(h)) || (W && !aligned16(W)) || (targets && !aligned16(targets)) || (lse && !aligned16(lse)) ||
      (dloss && !aligned16(dloss)) || (dH && !aligned16(dH)) || (dW && !aligned16(dW)))
    return fail(BL_ERR_ALIGNMENT, "tensors must be 16-byte aligned");
  const size_t need = bl_linear_xent_backward_workspace_size(M, V, K, dw_dtype);
  if (M > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return fail(BL_ERR_WORKSPACE, "workspace needs %zu bytes, 16-byte aligned", need);
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_xent_backward(h, W, targets, lse, dloss, M, V, K, dH, dW, dw_dtype == BL_F32,
                                              accumulate_dW != 0, workspace, err, static_cast<cudaStream_t>(stream)),
                     "bl_linear_xent_backward launch");
}

// Shapes and type of the row operators (A1, A2, N1, N2, U1, U2).
static bl_status check_rows(int64_t M, int64_t K, bl_dtype dtype) {
  if (M < 0) return fail(BL_ERR_INVALID_ARG, "M=%lld must be >= 0", (long long)M);
  if (K < 1 || K > (int64_t(1) << 30))
    return fail(BL_ERR_UNSUPPORTED_SHAPE, "K=%lld must be from 1 to 2^30", (long long)K);
  if (M > (int64_t(1) << 30)) return fail(BL_ERR_UNSUPPORTED_SHAPE, "M=%lld too large", (long long)M);
  if (dtype != BL_BF16 && dtype != BL_F32) return fail(BL_ERR_DTYPE, "dtype %d", (int)dtype);
  return BL_OK;
}

bl_status bl_act8_encode(const void* x, bl_dtype x_dtype, int64_t M, int64_t K, int8_t* codes, float* scales,
                         void* stream) {
  g_msg[0] = 0;
  if (bl_status s = check_rows(M, K, x_dtype)) return s;
  if (M == 0) return BL_OK;
  if (!x || !codes || !scales) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales))
    return fail(BL_ERR_ALIGNMENT, "x, codes and scales must be 16-byte aligned");
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_act8_encode(x, x_dtype == BL_F32, M, K, codes, scales,
                                            static_cast<cudaStream_t>(stream)),
                     "bl_act8_encode launch");
}

bl_status bl_act8_decode(const int8_t* codes, const float* scales, int64_t M, int64_t K, void* x, bl_dtype x_dtype,
                         void* stream) {
  g_msg[0] = 0;
  if (bl_status s = check_rows(M, K, x_dtype)) return s;
  if (M == 0) return BL_OK;
  if (!x || !codes || !scales) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales))
    return fail(BL_ERR_ALIGNMENT, "x, codes and scales must be 16-byte aligned");
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_act8_decode(codes, scales, M, K, x, x_dtype == BL_F32,
                                            static_cast<cudaStream_t>(stream)),
                     "bl_act8_decode launch");
}

bl_status bl_norm_forward(const void* x, bl_dtype x_dtype, const void* weight, const void* bias, bl_dtype p_dtype,
                          int64_t M, int64_t K, float eps, int rms, void* y, float* mean, float* rstd, int8_t* codes,
                          float* scales, void* stream) {
  g_msg[0] = 0;
  if (bl_status s = check_rows(M, K, x_dtype)) return s;
  if (p_dtype != BL_BF16 && p_dtype != BL_F32) return fail(BL_ERR_DTYPE, "p_dtype %d", (int)p_dtype);
  if (!(eps - eps == 0.0f) || eps < 0.0f) return fail(BL_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if ((codes == nullptr) != (scales == nullptr)) return fail(BL_ERR_INVALID_ARG, "codes and scales go together");
  if (M == 0) return BL_OK;
  if (!x || !y || !rstd || (!rms && !mean)) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(x) || !aligned16(y) || !aligned16(rstd) || (mean && !aligned16(mean)) ||
      (weight && !aligned16(weight)) || (bias && !aligned16(bias)) || (codes && !aligned16(codes)) ||
      (scales && !aligned16(scales)))
    return fail(BL_ERR_ALIGNMENT, "tensors must be 16-byte aligned");
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_norm_forward(x, x_dtype == BL_F32, weight, bias, p_dtype == BL_F32, M, K, eps,
                                             rms != 0, y, mean, rstd, codes, scales,
                                             static_cast<cudaStream_t>(stream)),
                     "bl_norm_forward launch");
}

size_t bl_norm_backward_workspace_size(int64_t M, int64_t K) {
  g_msg[0] = 0;
  if (M == 0 || check_rows(M, K, BL_BF16) != BL_OK) return 0;
  return bl::norm_backward_workspace_bytes(M, K);
}

bl_status bl_norm_backward(const void* dy, const void* x, const int8_t* codes, const float* scales, bl_dtype x_dtype,
                           const void* weight, bl_dtype p_dtype, const float* mean, const float* rstd, int64_t M,
                           int64_t K, int rms, void* dx, void* dweight, void* dbias, int accumulate, void* workspace,
                           size_t workspace_bytes, void* stream) {
  g_msg[0] = 0;
  if (bl_status s = check_rows(M, K, x_dtype)) return s;
  if (p_dtype != BL_BF16 && p_dtype != BL_F32) return fail(BL_ERR_DTYPE, "p_dtype %d", (int)p_dtype);
  if ((codes == nullptr) != (scales == nullptr)) return fail(BL_ERR_INVALID_ARG, "codes and scales go together");
  if (x && codes) return fail(BL_ERR_INVALID_ARG, "x or its 8-bit form, not both");
  if (M == 0 && ((!dweight && !dbias) || accumulate)) return BL_OK;
  if (!dx && !dweight && !dbias) return BL_OK;
  if (M > 0 && (!dy || (!x && !codes) || !rstd || (!rms && !mean))) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if ((dy && !aligned16(dy)) || (x && !aligned16(x)) || (codes && !aligned16(codes)) ||
      (scales && !aligned16(scales)) || (weight && !aligned16(weight)) || (mean && !aligned16(mean)) ||
      (rstd && !aligned16(rstd)) || (dx && !aligned16(dx)) || (dweight && !aligned16(dweight)) ||
      (dbias && !aligned16(dbias)))
    return fail(BL_ERR_ALIGNMENT, "tensors must be 16-byte aligned");
  const size_t need = bl_norm_backward_workspace_size(M, K);
  if (M > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return fail(BL_ERR_WORKSPACE, "workspace needs %zu bytes, 16-byte aligned", need);
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_norm_backward(dy, x, codes, scales, x_dtype == BL_F32, weight, p_dtype == BL_F32,
                                              mean, rstd, M, K, rms != 0, dx, dweight, dbias, accumulate != 0,
                                              workspace, static_cast<cudaStream_t>(stream)),
                     "bl_norm_backward launch");
}

bl_status bl_swiglu_forward(const void* gate, const void* up, bl_dtype x_dtype, int64_t M, int64_t K, void* y,
                            int8_t* gate_codes, float* gate_scales, int8_t* up_codes, float* up_scales,
                            void* stream) {
  g_msg[0] = 0;
  if (bl_status s = check_rows(M, K, x_dtype)) return s;
  const int saved = (gate_codes != nullptr) + (gate_scales != nullptr) + (up_codes != nullptr) + (up_scales != nullptr);
  if (saved != 0 && saved != 4) return fail(BL_ERR_INVALID_ARG, "the four code and scale arrays go together");
  if (M == 0) return BL_OK;
  if (!gate || !up || !y) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(gate) || !aligned16(up) || !aligned16(y) ||
      (saved && (!aligned16(gate_codes) || !aligned16(gate_scales) || !aligned16(up_codes) || !aligned16(up_scales))))
    return fail(BL_ERR_ALIGNMENT, "tensors must be 16-byte aligned");
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_swiglu_forward(gate, up, x_dtype == BL_F32, M, K, y, gate_codes, gate_scales, up_codes,
                                               up_scales, static_cast<cudaStream_t>(stream)),
                     "bl_swiglu_forward launch");
}

bl_status bl_swiglu_backward(const void* dy, const int8_t* gate_codes, const float* gate_scales,
                             const int8_t* up_codes, const float* up_scales, bl_dtype x_dtype, int64_t M, int64_t K,
                             void* dgate, void* dup, void* stream) {
  g_msg[0] = 0;
  if (bl_status s = check_rows(M, K, x_dtype)) return s;
  if (M == 0) return BL_OK;
  if (!dy || !gate_codes || !gate_scales || !up_codes || !up_scales || !dgate || !dup)
    return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (dgate == dup) return fail(BL_ERR_INVALID_ARG, "dgate and dup are the same memory");
  if (!aligned16(dy) || !aligned16(gate_codes) || !aligned16(gate_scales) || !aligned16(up_codes) ||
      !aligned16(up_scales) || !aligned16(dgate) || !aligned16(dup))
    return fail(BL_ERR_ALIGNMENT, "tensors must be 16-byte aligned");
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_swiglu_backward(dy, gate_codes, gate_scales, up_codes, up_scales, x_dtype == BL_F32, M,
                                                K, dgate, dup, static_cast<cudaStream_t>(stream)),
                     "bl_swiglu_backward launch");
}

// Shapes and types of the norm with an INT8 result (Q1, Q2).
static bl_status check_norm_quant(int64_t M, int64_t K, bl_dtype x_dtype, bl_dtype s_dtype, bl_dtype p_dtype) {
  if (M < 0) return fail(BL_ERR_INVALID_ARG, "M=%lld must be >= 0", (long long)M);
  if (K < 8 || K % 8 != 0 || K > bl::kNormQuantMaxK)
    return fail(BL_ERR_UNSUPPORTED_SHAPE, "K=%lld must be a multiple of 8 from 8 to %lld", (long long)K,
                (long long)bl::kNormQuantMaxK);
  if (M > (int64_t(1) << 30)) return fail(BL_ERR_UNSUPPORTED_SHAPE, "M=%lld too large", (long long)M);
  if (x_dtype != BL_BF16 && x_dtype != BL_F32) return fail(BL_ERR_DTYPE, "x_dtype %d", (int)x_dtype);
  if (s_dtype != BL_BF16 && s_dtype != BL_F32) return fail(BL_ERR_DTYPE, "s_dtype %d", (int)s_dtype);
  if (p_dtype != BL_BF16 && p_dtype != BL_F32) return fail(BL_ERR_DTYPE, "p_dtype %d", (int)p_dtype);
  if (x_dtype == BL_F32 && s_dtype == BL_BF16) return fail(BL_ERR_DTYPE, "an fp32 x with a bf16 residual stream");
  return BL_OK;
}

bl_status bl_norm_quant_forward(const void* x, bl_dtype x_dtype, const void* residual, bl_dtype s_dtype,
                                const void* weight, bl_dtype p_dtype, int64_t M, int64_t K, float eps, void* sum,
                                float* rstd, int8_t* xq, float* sx, void* stream) {
  g_msg[0] = 0;
  if (bl_status s = check_norm_quant(M, K, x_dtype, s_dtype, p_dtype)) return s;
  if (!(eps - eps == 0.0f) || eps < 0.0f) return fail(BL_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (M == 0) return BL_OK;
  if (!x || !rstd || !xq || !sx) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if ((residual == nullptr) != (sum == nullptr)) return fail(BL_ERR_INVALID_ARG, "residual and sum go together");
  if (!residual && x_dtype != s_dtype) return fail(BL_ERR_DTYPE, "without a residual x is the stream: s_dtype must be x_dtype");
  if (!aligned16(x) || (residual && !aligned16(residual)) || (weight && !aligned16(weight)) || (sum && !aligned16(sum)) ||
      !aligned16(rstd) || !aligned16(xq) || !aligned16(sx))
    return fail(BL_ERR_ALIGNMENT, "tensors must be 16-byte aligned");
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_norm_quant_forward(x, x_dtype == BL_F32, residual, s_dtype == BL_F32, weight,
                                                   p_dtype == BL_F32, M, K, eps, sum, rstd, xq, sx,
                                                   static_cast<cudaStream_t>(stream)),
                     "bl_norm_quant_forward launch");
}

size_t bl_norm_quant_backward_workspace_size(int64_t M, int64_t K) {
  g_msg[0] = 0;
  if (M == 0 || check_norm_quant(M, K, BL_BF16, BL_BF16, BL_BF16) != BL_OK) return 0;
  return bl::norm_quant_backward_workspace_bytes(K);
}

bl_status bl_norm_quant_backward(const void* dy, bl_dtype dy_dtype, const void* dsum, const void* sum, bl_dtype s_dtype,
                                 const void* weight, bl_dtype p_dtype, const float* rstd, int64_t M, int64_t K,
                                 void* dresidual, void* dx, bl_dtype x_dtype, void* dweight, int accumulate,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  g_msg[0] = 0;
  if (bl_status s = check_norm_quant(M, K, x_dtype, s_dtype, p_dtype)) return s;
  if (dy_dtype != BL_BF16 && dy_dtype != BL_F32) return fail(BL_ERR_DTYPE, "dy_dtype %d", (int)dy_dtype);
  if (!dresidual && !dx && !dweight) return BL_OK;
  if (M == 0 && (!dweight || accumulate)) return BL_OK;
  if (M > 0 && (!dy || !sum || !rstd)) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (M > 0 && dx && dx == dresidual) return fail(BL_ERR_INVALID_ARG, "dx and dresidual are the same memory");
  if ((dy && !aligned16(dy)) || (dsum && !aligned16(dsum)) || (sum && !aligned16(sum)) ||
      (weight && !aligned16(weight)) || (rstd && !aligned16(rstd)) || (dresidual && !aligned16(dresidual)) ||
      (dx && !aligned16(dx)) || (dweight && !aligned16(dweight)))
    return fail(BL_ERR_ALIGNMENT, "tensors must be 16-byte aligned");
  const size_t need = bl_norm_quant_backward_workspace_size(M, K);
  if (M > 0 && dweight && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return fail(BL_ERR_WORKSPACE, "workspace needs %zu bytes, 16-byte aligned", need);
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_norm_quant_backward(dy, dy_dtype == BL_F32, dsum, sum, s_dtype == BL_F32, weight,
                                                    p_dtype == BL_F32, rstd, M, K, dresidual, dx, x_dtype == BL_F32,
                                                    dweight, accumulate != 0, workspace,
                                                    static_cast<cudaStream_t>(stream)),
                     "bl_norm_quant_backward launch");
}

// Shape limits of the product of INT8 operands (its INT32 sums, tile counts and
// tensor-map coordinates fit within them).
static bl_status check_int8(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 1) return fail(BL_ERR_INVALID_ARG, "M=%lld, N=%lld", (long long)M, (long long)N);
  if (K < 16 || K % 16 != 0 || K > 65536)
    return fail(BL_ERR_UNSUPPORTED_SHAPE, "K=%lld must be a multiple of 16 from 16 to 65536", (long long)K);
  if (M > 131072 || N > (int64_t(1) << 20))
    return fail(BL_ERR_UNSUPPORTED_SHAPE, "M=%lld above 131072 or N=%lld above 2^20", (long long)M, (long long)N);
  return BL_OK;
}

bl_status bl_int8_linear_forward(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw, int64_t M,
                                 int64_t N, int64_t K, void* y, bl_dtype y_dtype, void* stream) {
  g_msg[0] = 0;
  if (bl_status s = check_int8(M, N, K)) return s;
  if (y_dtype != BL_BF16 && y_dtype != BL_F32) return fail(BL_ERR_DTYPE, "y_dtype %d", (int)y_dtype);
  if (M == 0) return BL_OK;
  if (!xq || !sx || !wq || !sw || !y) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(xq) || !aligned16(sx) || !aligned16(wq) || !aligned16(sw) || !aligned16(y))
    return fail(BL_ERR_ALIGNMENT, "tensors must be 16-byte aligned");
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_int8_forward(xq, sx, wq, sw, M, N, K, y, y_dtype == BL_F32, err,
                                             static_cast<cudaStream_t>(stream)),
                     "bl_int8_linear_forward launch");
}

size_t bl_int8_linear_backward_workspace_size(int64_t M, int64_t N, int64_t K) {
  g_msg[0] = 0;
  if (M == 0 || N % 8 != 0 || check_int8(M, N, K) != BL_OK) return 0;
  return bl::int8_backward_workspace_bytes(M, N, K);
}

bl_status bl_int8_linear_backward(const void* dY, const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                                  int64_t M, int64_t N, int64_t K, void* dX, void* dW, bl_dtype dw_dtype,
                                  int accumulate_dW, void* workspace, size_t workspace_bytes, void* stream) {
  g_msg[0] = 0;
  if (bl_status s = check_int8(M, N, K)) return s;
  if (N % 8 != 0) return fail(BL_ERR_UNSUPPORTED_SHAPE, "N=%lld must be a multiple of 8 in the backward", (long long)N);
  if (dw_dtype != BL_BF16 && dw_dtype != BL_F32) return fail(BL_ERR_DTYPE, "dw_dtype %d", (int)dw_dtype);
  if (!dX && !dW) return BL_OK;
  if (M == 0 && (!dW || accumulate_dW)) return BL_OK;
  if (M > 0 && (!dY || !xq || !sx || !wq || !sw)) return fail(BL_ERR_INVALID_ARG, "null pointer");
  if ((dY && !aligned16(dY)) || (xq && !aligned16(xq)) || (sx && !aligned16(sx)) || (wq && !aligned16(wq)) ||
      (sw && !aligned16(sw)) || (dX && !aligned16(dX)) || (dW && !aligned16(dW)))
    return fail(BL_ERR_ALIGNMENT, "tensors must be 16-byte aligned");
  const size_t need = bl_int8_linear_backward_workspace_size(M, N, K);
  if (M > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return fail(BL_ERR_WORKSPACE, "workspace needs %zu bytes, 16-byte aligned", need);
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_int8_backward(dY, xq, sx, wq, sw, M, N, K, dX, dW, dw_dtype == BL_F32,
                                              accumulate_dW != 0, workspace, err, static_cast<cudaStream_t>(stream)),
                     "bl_int8_linear_backward launch");
}

size_t bl_grad_norm_workspace_size(int64_t count) {
  g_msg[0] = 0;
  return count < 1 || count > (int64_t(1) << 20) ? 0 : bl::grad_norm_workspace_bytes(count);
}

bl_status bl_grad_norm(const bl_tensor* host_grads, int64_t count, float* norm, void* workspace, size_t workspace_bytes,
                       void* stream) {
  g_msg[0] = 0;
  return clip(host_grads, nullptr, count, false, 0.0, norm, workspace, workspace_bytes, stream, "bl_grad_norm launch");
}

bl_status bl_clip_grads(const bl_tensor* host_grads, void* const* host_out, int64_t count, double max_norm, float* norm,
                        void* workspace, size_t workspace_bytes, void* stream) {
  g_msg[0] = 0;
  return clip(host_grads, host_out, count, true, max_norm, norm, workspace, workspace_bytes, stream, "bl_clip_grads launch");
}

bl_status bl_selftest_timeout(void* stream) {
  g_msg[0] = 0;
  int* err = nullptr;
  if (bl_status s = current_device(&err)) return s;
  return cuda_status(bl::launch_selftest_timeout(err, static_cast<cudaStream_t>(stream)), "bl_selftest_timeout");
}

bl_status bl_get_last_error(void) {
  g_msg[0] = 0;
  if (cudaError_t e = cudaDeviceSynchronize(); e != cudaSuccess) return cuda_status(e, "cudaDeviceSynchronize");
  int v = 0;
  if (cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int)); e != cudaSuccess)
    return cuda_status(e, "read device error word");
  if (v == BL_ERR_TIMEOUT) return fail(BL_ERR_TIMEOUT, "a device pipeline wait exceeded its bound");
  return v == 0 ? BL_OK : fail(static_cast<bl_status>(v), "device error %d", v);
}

bl_status bl_reset_error(void) {
  g_msg[0] = 0;
  const int zero = 0;
  return cuda_status(cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int)), "reset device error word");
}

}  // extern "C"
