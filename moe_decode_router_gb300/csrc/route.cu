// Routing to experts from given logits, and grouping of the chosen pairs by
// expert, for any number of experts (the sublayer calls have both built in for
// their one shape).
//
// Routing, one warp per token.  With s = sigmoid(logit) or softmax over the
// row, an expert is chosen by its key: the logit itself without a bias (both
// scores grow with it, so the order is exact), s + bias with one.  Ties go to
// the lower index.  Where neighbouring keys or group scores are closer in fp32
// than fp32 can tell apart, the row is decided again in fp64: a selection is a
// whole number and has no "almost".
#include "flint_common.cuh"
#include "flint_internal.h"

namespace flint {

namespace {

constexpr unsigned FULL = 0xffffffffu;

// Order-preserving key of a float, never 0 for a value above -inf; -0 and +0
// share a key.
__device__ __forceinline__ uint32_t ord_key(float f) {
  const uint32_t b = __float_as_uint(__fadd_rn(f, 0.0f));
  return (b >> 31) ? ~b : (b | 0x80000000u);
}

struct RouteParams {
  const void* logits;
  long long stride;  // elements between rows
  const float* bias;
  int32_t* ids;
  float* w;
  int T, E, top_k, n_groups, top_groups;
  int softmax, top2, renorm;
  float scale;
};

// The two largest of the values that the lanes hold as (a, b), a >= b, -inf
// where there is none; every lane gets the result.
template <typename F>
__device__ __forceinline__ void warp_top2(F& a, F& b) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const F oa = __shfl_xor_sync(FULL, a, off), ob = __shfl_xor_sync(FULL, b, off);
    if (oa > a) {
      b = a > ob ? a : ob;
      a = oa;
    } else {
      b = b > oa ? b : oa;
    }
  }
}

// Score of every group: lane g of the result holds group g's, -inf for a group
// without candidates and for lanes without a group.
template <typename F, int EPL>
__device__ __forceinline__ F group_scores(const F (&v)[EPL], int lane, int E, int G, bool top2) {
  const int size = E / G;
  F mine = -(F)INFINITY;
  for (int g = 0; g < G; ++g) {
    F a = -(F)INFINITY, b = -(F)INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      if (e >= g * size && e < (g + 1) * size) {
        if (v[i] > a) {
          b = a;
          a = v[i];
        } else if (v[i] > b) {
          b = v[i];
        }
      }
    }
    warp_top2(a, b);
    const F s = (top2 && b > -(F)INFINITY) ? a + b : a;
    if (lane == g) mine = s;
  }
  return mine;
}

// Bit g of the result: group g is among the `top` best (ties to the lower
// group).  `unsure` is set when a kept and a dropped score are within `tol` of
// each other.
template <typename F>
__device__ __forceinline__ uint32_t keep_groups(F score, int lane, int G, int top, F tol, bool& unsure) {
  int rank = 0;
  for (int g = 0; g < G; ++g) {
    const F o = __shfl_sync(FULL, score, g);
    if (o > score || (o == score && g < lane)) ++rank;
  }
  const bool kept = lane < G && rank < top;
  const uint32_t mask = __ballot_sync(FULL, kept);
  // weakest kept score and strongest dropped one
  F lo = kept ? score : (F)INFINITY, hi = (lane < G && !kept) ? score : -(F)INFINITY;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const F l = __shfl_xor_sync(FULL, lo, off), h = __shfl_xor_sync(FULL, hi, off);
    lo = l < lo ? l : lo;
    hi = h > hi ? h : hi;
  }
  unsure = hi > -(F)INFINITY && !(lo - hi > tol);
  return mask;
}

template <typename F, int EPL>
__device__ __forceinline__ void softmax_scores(const float (&x)[EPL], F (&s)[EPL]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; ++i) m = x[i] > m ? x[i] : m;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, off));
  F z = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    s[i] = x[i] > -INFINITY ? (x[i] == m ? (F)1 : exp((F)x[i] - (F)m)) : (F)0;
    z += s[i];
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(FULL, z, off);
#pragma unroll
  for (int i = 0; i < EPL; ++i) s[i] = z > 0 ? s[i] / z : (F)0;
}

template <typename F, int EPL>
__device__ __forceinline__ void all_scores(const RouteParams& p, const float (&x)[EPL], F (&s)[EPL]) {
  if (p.softmax) {
    softmax_scores<F, EPL>(x, s);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] = x[i] > -INFINITY ? (F)1 / ((F)1 + exp(-(F)x[i])) : (F)0;
  }
}

// Keys (choice) and values (groups) of the row in type F; -inf: not a candidate.
template <typename F, int EPL>
__device__ __forceinline__ void keys_of(const RouteParams& p, const float (&x)[EPL], const F (&s)[EPL], int lane,
                                        F (&key)[EPL]) {
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    F k = -(F)INFINITY;
    if (x[i] > -INFINITY) {
      k = (p.bias != nullptr && e < p.E) ? s[i] + (F)__ldg(p.bias + e) : (F)x[i];
      if (!(k > -(F)INFINITY)) k = -(F)INFINITY;
    }
    key[i] = k;
  }
}

// Takes the groups that are out away from the keys.
template <typename F, int EPL>
__device__ __forceinline__ void drop_groups(F (&key)[EPL], int lane, int size, uint32_t kept) {
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int g = (lane + 32 * i) / size;
    if (g >= 32 || !((kept >> g) & 1u)) key[i] = -(F)INFINITY;
  }
}

// The `n` best keys in order: lane k ends with the k-th's expert (-1: none
// left) and key.
template <typename F, int EPL>
__device__ __forceinline__ void select_best(const F (&key)[EPL], int lane, int n, int& my_e, F& my_key) {
  uint32_t taken = 0u;
  my_e = -1;
  my_key = -(F)INFINITY;
  for (int k = 0; k < n; ++k) {
    F best = -(F)INFINITY;
    int at = 1 << 20;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (!((taken >> i) & 1u) && key[i] > best) {
        best = key[i];
        at = lane + 32 * i;
      }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const F ob = __shfl_xor_sync(FULL, best, off);
      const int oa = __shfl_xor_sync(FULL, at, off);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
      }
    }
    if (!(best > -(F)INFINITY)) break;
    if ((at & 31) == lane) taken |= 1u << (at >> 5);
    if (lane == k) {
      my_e = at;
      my_key = best;
    }
  }
}

// The row in fp64.
template <int EPL>
__device__ __noinline__ void route_row_f64(const RouteParams& p, const float (&x)[EPL], int lane, int& my_e) {
  double s[EPL], key[EPL], my_key;
  all_scores<double, EPL>(p, x, s);
  keys_of<double, EPL>(p, x, s, lane, key);
  if (p.n_groups > 1) {
    uint32_t kept;
    bool unsure;
    if (p.bias == nullptr && p.top2) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (!(x[i] > -INFINITY)) s[i] = -INFINITY;
      kept = keep_groups<double>(group_scores<double, EPL>(s, lane, p.E, p.n_groups, true), lane, p.n_groups,
                                 p.top_groups, 0.0, unsure);
    } else {
      kept = keep_groups<double>(group_scores<double, EPL>(key, lane, p.E, p.n_groups, p.top2 != 0), lane, p.n_groups,
                                 p.top_groups, 0.0, unsure);
    }
    drop_groups<double, EPL>(key, lane, p.E / p.n_groups, kept);
  }
  select_best<double, EPL>(key, lane, p.top_k, my_e, my_key);
}

template <int EPL, bool BF16>
__global__ void __launch_bounds__(128) route_kernel(const RouteParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (t >= p.T) return;
  float x[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    x[i] = -INFINITY;
    if (e < p.E) {
      const size_t at = (size_t)t * (size_t)p.stride + (size_t)e;
      x[i] = BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.logits)[at])
                  : static_cast<const float*>(p.logits)[at];
    }
  }
  int my_e;
  route_row_f64<EPL>(p, x, lane, my_e);

  // Weights from the selected logits.  u is the score times a factor common to
  // the row that keeps the largest near 1, so that renormalising never divides
  // by zero, however low the logits are.
  float xs = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const float v = __shfl_sync(FULL, x[i], my_e & 31);
    if (my_e >= 0 && (my_e >> 5) == i) xs = v;
  }
  const bool on = my_e >= 0;
  float ref = on ? (p.softmax ? xs : fminf(xs, 0.f)) : -INFINITY;
  if (p.renorm) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ref = fmaxf(ref, __shfl_xor_sync(FULL, ref, off));
  }
  float u = 0.f, den = 1.f;
  if (p.softmax) {
    if (!p.renorm) {
      float m = -INFINITY, z = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) m = x[i] > m ? x[i] : m;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, off));
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (x[i] > -INFINITY) z += x[i] == m ? 1.f : expf(x[i] - m);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(FULL, z, off);
      ref = m;
      den = z;
    }
    if (on) u = xs == ref ? 1.f : expf(xs - ref);
  } else if (on) {
    const float m = fminf(xs, 0.f);
    const float r = p.renorm ? ref : 0.f;
    u = (m == r ? 1.f : expf(m - r)) / (1.f + expf(-fabsf(xs)));
  }
  if (p.renorm) {
    den = u;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) den += __shfl_xor_sync(FULL, den, off);
  }
  if (lane < p.top_k) {
    p.ids[(size_t)t * p.top_k + lane] = my_e;
    p.w[(size_t)t * p.top_k + lane] = on ? p.scale * (u / den) : 0.f;
  }
}

// ---------------------------------------------------------------- grouping
// Stable counting sort of the pairs by expert.  Every warp owns one stretch of
// consecutive pairs and a histogram of its own; warps' histograms, summed in
// order, give each warp its first place in every expert's range, and a second
// pass over the stretch hands the places out in order.  No atomic decides an
// order, so the result is the same on every call.
constexpr int GP_WARPS = 32;

__global__ void __launch_bounds__(GP_WARPS * 32) group_kernel(const int32_t* __restrict__ ids, int P, int E,
                                                              int32_t* __restrict__ offsets,
                                                              int32_t* __restrict__ order, int32_t* __restrict__ pos) {
  extern __shared__ int hist[];  // [GP_WARPS][E], then [E + 1] totals
  int* first = hist + GP_WARPS * E;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < GP_WARPS * E; i += GP_WARPS * 32) hist[i] = 0;
  __syncthreads();
  const int per = ((P + GP_WARPS * 32 - 1) / (GP_WARPS * 32)) * 32;  // pairs of a warp
  const long long lo = (long long)warp * per;
  int* h = hist + warp * E;
  for (int i = 0; i < per; i += 32) {
    const long long at = lo + i + lane;
    const int id = at < P ? __ldg(ids + at) : -1;
    if (id >= 0 && id < E) atomicAdd(&h[id], 1);
  }
  __syncthreads();
  for (int e = tid; e < E; e += GP_WARPS * 32) {  // per expert: exclusive sums over the warps
    int s = 0;
    for (int w = 0; w < GP_WARPS; ++w) {
      const int c = hist[w * E + e];
      hist[w * E + e] = s;
      s += c;
    }
    first[e] = s;
  }
  __syncthreads();
  if (warp == 0) {  // exclusive sums over the experts
    int base = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const int c = e < E ? first[e] : 0;
      int incl = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(FULL, incl, off);
        if (lane >= off) incl += v;
      }
      if (e < E) {
        first[e] = base + incl - c;
        offsets[e] = base + incl - c;
      }
      base += __shfl_sync(FULL, incl, 31);
    }
    if (lane == 0) {
      first[E] = base;
      offsets[E] = base;
    }
  }
  __syncthreads();
  for (int i = 0; i < per; i += 32) {
    const long long at = lo + i + lane;
    const bool in = at < P;
    int id = in ? __ldg(ids + at) : -1;
    if (id < 0 || id >= E) id = -1;
    const uint32_t peers = __match_any_sync(FULL, id);
    int place = -1;
    if (id >= 0) place = first[id] + h[id] + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (id >= 0 && lane == __ffs(peers) - 1) h[id] += __popc(peers);
    __syncwarp();
    if (in) pos[at] = place;
    if (place >= 0) order[place] = (int)at;
  }
  for (int i = first[E] + tid; i < P; i += GP_WARPS * 32) order[i] = -1;
}

template <int EPL>
cudaError_t launch_route_epl(const RouteParams& p, bool bf16, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.T + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&cfg, route_kernel<EPL, true>, p)
              : cudaLaunchKernelEx(&cfg, route_kernel<EPL, false>, p);
}

}  // namespace

cudaError_t route_kernels_init() {
  return cudaFuncSetAttribute(group_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (GP_WARPS * ROUTE_MAX_E + ROUTE_MAX_E + 1) * 4);
}

cudaError_t launch_route(const RouteSpec& r, const void* logits, bool bf16, long long stride, int T, const float* bias,
                         int32_t* ids, float* w, cudaStream_t st) {
  RouteParams p;
  p.logits = logits;
  p.stride = stride;
  p.bias = bias;
  p.ids = ids;
  p.w = w;
  p.T = T;
  p.E = r.E;
  p.top_k = r.top_k;
  p.n_groups = r.n_groups;
  p.top_groups = r.top_groups;
  p.softmax = r.softmax;
  p.top2 = r.top2;
  p.renorm = r.renorm;
  p.scale = r.scale;
  if (r.E <= 64) return launch_route_epl<2>(p, bf16, st);
  if (r.E <= 128) return launch_route_epl<4>(p, bf16, st);
  if (r.E <= 256) return launch_route_epl<8>(p, bf16, st);
  if (r.E <= 512) return launch_route_epl<16>(p, bf16, st);
  return launch_route_epl<32>(p, bf16, st);
}

cudaError_t launch_group_pairs(const int32_t* ids, int P, int E, int32_t* offsets, int32_t* order, int32_t* pos,
                               cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(GP_WARPS * 32);
  cfg.dynamicSmemBytes = (size_t)(GP_WARPS * E + E + 1) * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, group_kernel, ids, P, E, offsets, order, pos);
}

}  // namespace flint
