// C ABI of the linear, gated and 8-bit integer products: argument validation and the
// choice of kernels.  See include/flint_moe.h.
#include <initializer_list>
#include <map>
#include <mutex>

#include "flint_internal.h"
#include "flint_moe.h"

namespace flint {

namespace {

constexpr int MAX_ROWS = 1 << 24;
constexpr int MAX_WIDTH = 1 << 17;  // of N, of 2 I and of K

int to_status(cudaError_t e) { return e == cudaSuccess ? FLINT_MOE_OK : FLINT_MOE_ERR_CUDA; }
bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

struct Range {
  const void* p;
  size_t n;
};
bool overlap(const Range& a, const Range& b) {
  if (a.p == nullptr || b.p == nullptr || a.n == 0 || b.n == 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  return pa < pb + b.n && pb < pa + a.n;
}
// A required pointer that is null or misaligned, an optional one that is misaligned, or an
// output that shares a byte with another buffer.
bool bad_buffers(std::initializer_list<Range> outs, std::initializer_list<Range> ins,
                 std::initializer_list<Range> optional_outs = {}, std::initializer_list<Range> optional_ins = {}) {
  Range all[12];
  int n = 0;
  for (const auto& list : {outs, ins})
    for (const Range& r : list)
      if (r.p == nullptr) return true;
  for (const auto& list : {outs, optional_outs})
    for (const Range& r : list) all[n++] = r;
  const int n_out = n;
  for (const auto& list : {ins, optional_ins})
    for (const Range& r : list) all[n++] = r;
  for (int i = 0; i < n; ++i)
    if (!aligned16(all[i].p)) return true;
  for (int i = 0; i < n_out; ++i)
    for (int j = i + 1; j < n; ++j)
      if (overlap(all[i], all[j])) return true;
  return false;
}

// Limits of a product of M rows with [experts][N][K]; gated: N is 2 I.
int check_shape(int M, int N, int K, int E, bool grouped, bool gated) {
  if (M < 1 || N < 1 || K < 1 || E < 1) return FLINT_MOE_ERR_INVALID_ARG;
  if (M > MAX_ROWS || E > ROUTE_MAX_E || N > MAX_WIDTH || N % (gated ? 32 : 8) != 0 || K > MAX_WIDTH || K % 16 != 0)
    return FLINT_MOE_ERR_UNSUPPORTED;
  if (!grouped && E != 1) return FLINT_MOE_ERR_INVALID_ARG;
  return FLINT_MOE_OK;
}
bool act_ok(int act) { return act == FLINT_MOE_ACT_SILU || act == FLINT_MOE_ACT_GELU; }
bool type_ok(int type) { return type == FLINT_MOE_T_BF16 || type == FLINT_MOE_T_F32; }
size_t type_size(int type) { return type == FLINT_MOE_T_BF16 ? 2 : 4; }
size_t offset_bytes(int E) { return (size_t)(E + 1) * 4; }

static_assert((int)FFN_NONE == (int)FLINT_MOE_ACT_NONE && (int)FFN_SILU == (int)FLINT_MOE_ACT_SILU &&
                  (int)FFN_GELU == (int)FLINT_MOE_ACT_GELU,
              "activations");

// A failure of the tensor-core kernels' set-up that another try cannot change.
bool lasting(cudaError_t e) {
  return e == cudaErrorNotSupported || e == cudaErrorInvalidConfiguration || e == cudaErrorInvalidValue ||
         e == cudaErrorNoKernelImageForDevice || e == cudaErrorInvalidDeviceFunction || e == cudaErrorSymbolNotFound;
}

// The current device's set-up: the library's, and that of the tensor-core kernels, once or, after a
// failure that may pass, on the next call again.  Without those kernels most_ks is 0.
int set_up(PairDevice* d) try {
  const int st = device_info(&d->sms, &d->err);
  if (st != FLINT_MOE_OK) return st;
  static std::mutex mu;
  static std::map<int, int> most;  // pairs of a cluster, 0: the kernels are not to be had
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return FLINT_MOE_ERR_CUDA;
  std::lock_guard<std::mutex> lk(mu);
  const auto it = most.find(dev);
  if (it != most.end()) {
    d->most_ks = it->second;
    return FLINT_MOE_OK;
  }
  const cudaError_t e = pair_gemm_kernels_init(&d->most_ks);
  if (e != cudaSuccess) {
    d->most_ks = 0;
    (void)cudaGetLastError();
  }
  if (e == cudaSuccess || lasting(e)) most.emplace(dev, d->most_ks);
  return FLINT_MOE_OK;
} catch (...) {  // no memory for the map, no mutex
  return FLINT_MOE_ERR_CUDA;
}

// The library's set-up alone.
int library_set_up() try {
  int sms = 0;
  unsigned* err = nullptr;
  return device_info(&sms, &err);
} catch (...) {
  return FLINT_MOE_ERR_CUDA;
}

int product(const ProductArgs& p, bool int8, flint_moe_stream_t stream) {
  PairDevice d;
  const int rc = set_up(&d);
  if (rc != FLINT_MOE_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (few_rows_take(p, int8, d)) return to_status(launch_few_rows(p, int8, st));
  if (d.most_ks == 0) return FLINT_MOE_ERR_CUDA;
  return to_status(launch_pair_forward(p, int8, d, st));
}

int gradients(const void* dy, const void* x, int M, const void* w, int E, const int32_t* offsets, int N, int K,
              void* dx, void* dw, int dw_type, const PairDevice& d, cudaStream_t st) {
  const GradArgs p = {dy, x, w, offsets, dx, dw, M, N, K, E, dw_type == FLINT_MOE_T_F32};
  if (dx == nullptr && dw == nullptr) return FLINT_MOE_OK;
  return to_status(launch_pair_backward(p, d, st));
}

}  // namespace

}  // namespace flint

using namespace flint;

extern "C" {

int flint_moe_linear(const void* x, int M, const void* w, int n_experts, const int32_t* offsets, int N, int K, void* y,
                     int y_type, flint_moe_stream_t stream) {
  if (!type_ok(y_type)) return FLINT_MOE_ERR_UNSUPPORTED;
  const int st = check_shape(M, N, K, n_experts, offsets != nullptr, false);
  if (st != FLINT_MOE_OK) return st;
  if (bad_buffers({{y, (size_t)M * N * type_size(y_type)}},
                  {{x, (size_t)M * K * 2}, {w, (size_t)n_experts * N * K * 2}}, {}, {{offsets, offset_bytes(n_experts)}}))
    return FLINT_MOE_ERR_INVALID_ARG;
  const ProductArgs p = {x, w, offsets, y, nullptr, nullptr, nullptr, M, N, K, n_experts, FFN_NONE,
                         y_type == FLINT_MOE_T_F32};
  return product(p, false, stream);
}

int flint_moe_gated_linear(const void* x, int M, const void* w, int n_experts, const int32_t* offsets, int I, int K,
                           int act, void* h, void* gu, flint_moe_stream_t stream) {
  if (!act_ok(act)) return FLINT_MOE_ERR_UNSUPPORTED;
  if (I < 1) return FLINT_MOE_ERR_INVALID_ARG;
  if (I > MAX_WIDTH / 2) return FLINT_MOE_ERR_UNSUPPORTED;
  const int st = check_shape(M, 2 * I, K, n_experts, offsets != nullptr, true);
  if (st != FLINT_MOE_OK) return st;
  if (bad_buffers({{h, (size_t)M * I * 2}}, {{x, (size_t)M * K * 2}, {w, (size_t)n_experts * 2 * I * K * 2}},
                  {{gu, (size_t)M * 2 * I * 2}}, {{offsets, offset_bytes(n_experts)}}))
    return FLINT_MOE_ERR_INVALID_ARG;
  const ProductArgs p = {x, w, offsets, h, gu, nullptr, nullptr, M, 2 * I, K, n_experts, act, 0};
  return product(p, false, stream);
}

int flint_moe_linear_backward(const void* dy, const void* x, int M, const void* w, int n_experts,
                              const int32_t* offsets, int N, int K, void* dx, void* dw, int dw_type,
                              flint_moe_stream_t stream) {
  if (!type_ok(dw_type)) return FLINT_MOE_ERR_UNSUPPORTED;
  int st = check_shape(M, N, K, n_experts, offsets != nullptr, false);
  if (st != FLINT_MOE_OK) return st;
  if (dx == nullptr && dw == nullptr) return FLINT_MOE_ERR_INVALID_ARG;
  const size_t weights = (size_t)n_experts * N * K;
  if (bad_buffers({}, {{dy, (size_t)M * N * 2}, {x, (size_t)M * K * 2}, {w, weights * 2}},
                  {{dx, (size_t)M * K * 2}, {dw, weights * type_size(dw_type)}}, {{offsets, offset_bytes(n_experts)}}))
    return FLINT_MOE_ERR_INVALID_ARG;
  PairDevice d;
  if ((st = set_up(&d)) != FLINT_MOE_OK) return st;
  if (d.most_ks == 0) return FLINT_MOE_ERR_CUDA;
  return gradients(dy, x, M, w, n_experts, offsets, N, K, dx, dw, dw_type, d,
                   reinterpret_cast<cudaStream_t>(stream));
}

int flint_moe_gated_linear_backward(const void* dh, const void* gu, const void* x, int M, const void* w, int n_experts,
                                    const int32_t* offsets, int I, int K, int act, void* dgu, void* dx, void* dw,
                                    int dw_type, flint_moe_stream_t stream) {
  if (!act_ok(act) || !type_ok(dw_type)) return FLINT_MOE_ERR_UNSUPPORTED;
  if (I < 1) return FLINT_MOE_ERR_INVALID_ARG;
  if (I > MAX_WIDTH / 2) return FLINT_MOE_ERR_UNSUPPORTED;
  int st = check_shape(M, 2 * I, K, n_experts, offsets != nullptr, true);
  if (st != FLINT_MOE_OK) return st;
  const size_t weights = (size_t)n_experts * 2 * I * K, sums = (size_t)M * 2 * I * 2;
  if (bad_buffers({{dgu, sums}}, {{dh, (size_t)M * I * 2}, {gu, sums}, {x, (size_t)M * K * 2}, {w, weights * 2}},
                  {{dx, (size_t)M * K * 2}, {dw, weights * type_size(dw_type)}}, {{offsets, offset_bytes(n_experts)}}))
    return FLINT_MOE_ERR_INVALID_ARG;
  PairDevice d;
  if ((st = set_up(&d)) != FLINT_MOE_OK) return st;
  if (d.most_ks == 0) return FLINT_MOE_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (launch_gate_backward(dh, gu, offsets, M, I, n_experts, act, dgu, s) != cudaSuccess) return FLINT_MOE_ERR_CUDA;
  return gradients(dgu, x, M, w, n_experts, offsets, 2 * I, K, dx, dw, dw_type, d, s);
}

int flint_moe_integer_quantize_rows(const void* x, int x_type, long long row_stride, int rows, int K,
                                    const int32_t* pos, int top_k, int places, int8_t* q, float* scales,
                                    flint_moe_stream_t stream) {
  if (!type_ok(x_type)) return FLINT_MOE_ERR_UNSUPPORTED;
  if (rows < 1 || K < 1 || places < 1 || (pos != nullptr && top_k < 1)) return FLINT_MOE_ERR_INVALID_ARG;
  if (rows > MAX_ROWS || places > MAX_ROWS || K % 16 != 0 || K > MAX_WIDTH || (pos != nullptr && top_k > ROUTE_MAX_K))
    return FLINT_MOE_ERR_UNSUPPORTED;
  if (pos == nullptr && places != rows) return FLINT_MOE_ERR_INVALID_ARG;
  if (row_stride < K || row_stride > (1LL << 31)) return FLINT_MOE_ERR_INVALID_ARG;
  const size_t size = type_size(x_type);
  if ((size_t)row_stride * size % 16 != 0) return FLINT_MOE_ERR_UNSUPPORTED;
  if (bad_buffers({{q, (size_t)places * K}, {scales, (size_t)places * 4}},
                  {{x, ((size_t)(rows - 1) * (size_t)row_stride + K) * size}}, {},
                  {{pos, (size_t)rows * (pos ? top_k : 0) * 4}}))
    return FLINT_MOE_ERR_INVALID_ARG;
  const int st = library_set_up();
  if (st != FLINT_MOE_OK) return st;
  return to_status(launch_integer_rows(x, x_type == FLINT_MOE_T_BF16, row_stride, rows, K, pos, top_k, places, q,
                                       scales, reinterpret_cast<cudaStream_t>(stream)));
}

int flint_moe_integer_gemm(const int8_t* a, const float* a_scales, int M, const int8_t* b, const float* b_scales,
                           int n_experts, const int32_t* offsets, int N, int K, int act, void* y, int y_type,
                           flint_moe_stream_t stream) {
  if (!type_ok(y_type) || (act != FLINT_MOE_ACT_NONE && !act_ok(act))) return FLINT_MOE_ERR_UNSUPPORTED;
  const bool gated = act != FLINT_MOE_ACT_NONE;
  const int st = check_shape(M, N, K, n_experts, offsets != nullptr, gated);
  if (st != FLINT_MOE_OK) return st;
  if (K == MAX_WIDTH) return FLINT_MOE_ERR_UNSUPPORTED;  // 2^17 products of 2^14 would pass an int
  if (bad_buffers({{y, (size_t)M * (gated ? N / 2 : N) * type_size(y_type)}},
                  {{a, (size_t)M * K},
                   {a_scales, (size_t)M * 4},
                   {b, (size_t)n_experts * N * K},
                   {b_scales, (size_t)n_experts * N * 4}},
                  {}, {{offsets, offset_bytes(n_experts)}}))
    return FLINT_MOE_ERR_INVALID_ARG;
  const ProductArgs p = {a, b, offsets, y, nullptr, a_scales, b_scales, M, N, K, n_experts, act,
                         y_type == FLINT_MOE_T_F32};
  return product(p, true, stream);
}

}  // extern "C"
