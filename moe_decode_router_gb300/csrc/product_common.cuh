// What the bf16 and the 8-bit integer products share: their arguments, the
// gated activations, and how a thread block finds the expert of a row.
#pragma once

#include <cstdint>

#include "flint_common.cuh"
#include "flint_internal.h"

namespace flint {

// 16 bytes of weights: read once, so not kept in L1.
__device__ __forceinline__ uint4 ldg_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Both activations are g * sigmoid(v): v = g, or 2 sqrt(2 / pi) (g + 0.044715 g^3),
// which is g / 2 * (1 + tanh(v / 2)).  __expf and __fdividef are off by a few units of
// 2^-23 of the value (and of |v|); below v = -88 the sigmoid is 0.
constexpr float GELU_C = 1.5957691216057308f, GELU_C3 = 0.07135481282553226f;  // 2 sqrt(2 / pi), times 0.044715

__device__ __forceinline__ float sigmoid_fast(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

__device__ __forceinline__ float activation(float g, int act) {
  const float v = act == FFN_SILU ? g : g * fmaf(GELU_C3 * g, g, GELU_C);
  return g * sigmoid_fast(v);
}

// The activation and its derivative, p + g p (1 - p) dv/dg.  Beyond |g| = 30 the
// sigmoid of the gelu form is 0 or 1 and its polynomial is not needed (nor let overflow).
__device__ __forceinline__ void activation_slope(float g, int act, float& a, float& slope) {
  float v = g, dv = 1.f;
  if (act != FFN_SILU) {
    const float c = fminf(fmaxf(g, -30.f), 30.f);
    v = c * fmaf(GELU_C3 * c, c, GELU_C);
    dv = fmaf(3.f * GELU_C3 * c, c, GELU_C);
  }
  // 1 - p is formed as sigmoid(-v): the difference would lose its bits near 1
  const float e = __expf(-fabsf(v)), r = __fdividef(1.f, 1.f + e);
  const float p = v >= 0.f ? r : e * r, q = v >= 0.f ? e * r : r;
  a = g * p;
  slope = fmaf(a * q, dv, p);
  if (g != g) slope = a = g;
}

// The expert of row r and its rows, found by one whole warp from offsets [E + 1]:
// the last group that starts at or before r.
struct RowGroup {
  int e, lo, hi;
};
__device__ __forceinline__ RowGroup group_of_row(const int32_t* offsets, int E, int M, int r, int lane) {
  unsigned begun = 0, from = 0, to = (unsigned)M;
  for (int i = lane; i <= E; i += 32) {
    const int o = __ldg(offsets + i);
    if (o <= r) {
      ++begun;
      from = max(from, (unsigned)max(o, 0));
    } else {
      to = min(to, (unsigned)o);
    }
  }
  begun = __reduce_add_sync(0xffffffffu, begun);
  RowGroup g;
  g.e = (int)begun - 1;
  g.lo = (int)redux_max(from);
  g.hi = (int)redux_min(to);
  return g;
}

}  // namespace flint
