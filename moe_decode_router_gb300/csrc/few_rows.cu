// Products of few rows, bf16 or 8-bit integer, dense or grouped by expert, plain or
// gated: the weights are streamed once for up to 8 rows of one expert.
//   y[m][n] = sum over k of x[m][k] * w[e][n][k]          (integer: times sx[m] * sw[e][n])
//   gated:  h[m][i] = act(y[m][i]) * y[m][I + i]
//
// A warp takes 16 rows of the mma's M side: 16 weight rows, or 8 of the gate's and the
// same 8 of the other factor's, so that the thread that holds a gate's sum holds its
// partner's too.  Both operands are read straight from global memory into fragments:
// a sum does not depend on the order of k, so lane t of a row's four takes bytes
// 16 t .. 16 t + 15 of each 64 for either operand (8 bf16 or 16 integers: two mma).
// DEEP pieces of 128 bytes a row (2 KB of weights a warp each) are under way at a time.
// Every SPLIT-th piece of K is a warp's; SPLIT warps of a CTA share their rows and add
// their sums in the warps' order, so that a small product has enough warps.  The tensor cores cut a
// sum of bf16 products instead of rounding it (2^17 into one accumulator lost 7e-4 of it), so in shapes
// of 4 pieces each pass's products begin from zero and are added in fp32; a warp of a shape of 2 has no
// more than ALONE.  A dense
// product asks for its first weights before it waits for the kernel before it: into L2
// alone, where a write of that kernel would still reach them.
//
// Grid (M, weight rows / rows of a CTA): the CTA of row r works when r is the first of a
// run of 8 rows of its expert; a dense product has CTAs for every eighth row alone.
#include "product_common.cuh"

namespace flint {

namespace {

__device__ __forceinline__ void mma_k64(float (&d)[4], const uint4& a, const uint4& b, const uint4& x) {
  mma_bf16(d, a.x, b.x, a.y, b.y, x.x, x.y);
  mma_bf16(d, a.z, b.z, a.w, b.w, x.z, x.w);
}
__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_k64(int (&d)[4], const uint4& a, const uint4& b, const uint4& x) {
  mma_s8(d, a.x, b.x, a.y, b.y, x.x, x.y);
  mma_s8(d, a.z, b.z, a.w, b.w, x.z, x.w);
}

template <bool INT8>
struct Sum {
  using type = float;
};
template <>
struct Sum<true> {
  using type = int;
};

template <bool INT8, bool GATED, int SPLIT, int WARPS, int DEEP>
__global__ void __launch_bounds__(WARPS * 32, (DEEP > 2 ? 16 : 24) / WARPS) few_rows_kernel(const ProductArgs p) {
  using S = typename Sum<INT8>::type;
  constexpr int SIZE = INT8 ? 1 : 2;
  constexpr bool ROUND = !INT8 && DEEP > 2;
  __shared__ S red[SPLIT == 1 ? 1 : WARPS][128];
  __shared__ int range[3];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int outs = GATED ? p.N / 2 : p.N;          // outputs of a row
  constexpr int STEP = GATED ? 8 : 16;             // of them, a warp's
  const int tile = blockIdx.y * (WARPS / SPLIT) + warp / SPLIT, n0 = tile * STEP;
  const int g = lane >> 2, t = lane & 3;
  const size_t kbytes = (size_t)p.K * SIZE;
  const int pieces = (int)((kbytes + 127) / 128);
  if (p.offsets == nullptr && n0 < outs) {
    const uint8_t* w = static_cast<const uint8_t*>(p.w);
    for (int i = t; i < 2 * DEEP; i += 4) {  // lanes t of a row: its two halves of 16 and the pieces
      const int row = i & 1 ? (GATED ? outs + n0 + g : min(n0 + g + 8, p.N - 1)) : n0 + g;
      const int piece = warp % SPLIT + (i >> 1) * SPLIT;
      if (piece < pieces) prefetch_l2(w + (size_t)row * kbytes + (size_t)piece * 128);
    }
  }
  pdl_wait();
  pdl_trigger();
  const int r = p.offsets == nullptr ? blockIdx.x * 8 : blockIdx.x;
  int e = 0, r0 = 0, r1 = p.M;
  if (p.offsets != nullptr) {
    if (warp == 0) {
      const RowGroup g = group_of_row(p.offsets, p.E, p.M, r, lane);
      if (lane == 0) {
        range[0] = g.e;
        range[1] = g.lo;
        range[2] = g.hi;
      }
    }
    __syncthreads();
    e = range[0];
    if (e < 0 || e >= p.E) return;
    r0 = range[1];
    r1 = range[2];
    if (r < r0 || r >= r1) return;
  }
  if ((r - r0) & 7) return;
  const int n_rows = min(8, r1 - r);
  S acc[4] = {0, 0, 0, 0};
  if (n0 < outs) {  // outs is a multiple of 8
    const uint8_t* w = static_cast<const uint8_t*>(p.w) + (size_t)e * p.N * kbytes;
    const uint8_t* b0 = w + (size_t)(n0 + g) * kbytes;
    const uint8_t* b1 = w + (size_t)(GATED ? outs + n0 + g : min(n0 + g + 8, p.N - 1)) * kbytes;
    const uint8_t* a0 = static_cast<const uint8_t*>(p.x) + (size_t)(r + min(g, n_rows - 1)) * kbytes;
    constexpr int U = DEEP;
    for (int q0 = warp % SPLIT; q0 < pieces; q0 += U * SPLIT) {
      uint4 v[U][4], x[U][2];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const size_t k0 = (size_t)(q0 + i * SPLIT) * 128 + 16 * t, k1 = k0 + 64;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        const bool in0 = k0 < kbytes, in1 = k1 < kbytes;  // K is a multiple of 16
        v[i][0] = in0 ? ldg_once(b0 + k0) : zero;
        v[i][1] = in0 ? ldg_once(b1 + k0) : zero;
        v[i][2] = in1 ? ldg_once(b0 + k1) : zero;
        v[i][3] = in1 ? ldg_once(b1 + k1) : zero;
        x[i][0] = in0 ? __ldg(reinterpret_cast<const uint4*>(a0 + k0)) : zero;
        x[i][1] = in1 ? __ldg(reinterpret_cast<const uint4*>(a0 + k1)) : zero;
      }
      S part[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < U; ++i) {
        mma_k64(ROUND ? part : acc, v[i][0], v[i][1], x[i][0]);
        mma_k64(ROUND ? part : acc, v[i][2], v[i][3], x[i][1]);
      }
      if (ROUND)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += part[i];
    }
  }
  auto put = [&](void* base, size_t at, float v) {
    if (p.f32)
      static_cast<float*>(base)[at] = v;
    else
      static_cast<__nv_bfloat16*>(base)[at] = __float2bfloat16_rn(v);
  };
  // Sum `a` of output n of row `col`; with GATED `b`, its partner's.
  auto store = [&](int col, int n, S a, S b) {
    if (col >= n_rows || n >= outs) return;
    float u = (float)a, v = (float)b;
    if (INT8) {
      const float s = __ldg(p.sx + r + col);
      const float* sw = p.sw + (size_t)e * p.N + n;
      u *= s * __ldg(sw);
      if (GATED) v *= s * __ldg(sw + outs);
    }
    if (GATED) {
      if (p.keep != nullptr) {
        __nv_bfloat16* keep = static_cast<__nv_bfloat16*>(p.keep) + (size_t)(r + col) * p.N + n;
        keep[0] = __float2bfloat16_rn(u);
        keep[outs] = __float2bfloat16_rn(v);
      }
      u = activation(u, p.act) * v;
    }
    put(p.y, (size_t)(r + col) * outs + n, u);
  };
  if constexpr (SPLIT == 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      store(2 * t + i, n0 + g, acc[i], acc[2 + i]);
      if (!GATED) store(2 * t + i, n0 + g + 8, acc[2 + i], 0);
    }
  } else {
    // red[warp][column * 16 + mma row]
#pragma unroll
    for (int i = 0; i < 4; ++i) red[warp][(2 * t + (i & 1)) * 16 + g + (i >> 1) * 8] = acc[i];
    __syncthreads();
    for (int o = tid; o < 8 * STEP * (WARPS / SPLIT); o += WARPS * 32) {
      const int part = o / (8 * STEP), c = o % (8 * STEP), col = c / STEP, row = c % STEP, at = col * 16 + row;
      S a = 0, b = 0;
#pragma unroll
      for (int w = 0; w < SPLIT; ++w) {
        a += red[part * SPLIT + w][at];
        if (GATED) b += red[part * SPLIT + w][at + 8];
      }
      store(col, (blockIdx.y * (WARPS / SPLIT) + part) * STEP + row, a, b);
    }
  }
}

template <bool INT8, bool GATED, int SPLIT, int WARPS, int DEEP>
cudaError_t launch(const ProductArgs& p, cudaStream_t st) {
  constexpr int ROWS = WARPS / SPLIT * (GATED ? 8 : 16);
  const int outs = GATED ? p.N / 2 : p.N;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.offsets == nullptr ? (p.M + 7) / 8 : p.M), (unsigned)((outs + ROWS - 1) / ROWS));
  cfg.blockDim = dim3(WARPS * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_rows_kernel<INT8, GATED, SPLIT, WARPS, DEEP>, p);
}

// Warps that share K and pieces under way, measured (us; calls in a graph; the second digits are the next
// best).  By expert all figures are of 256 experts of 1024 x 2048 (floors: the weights of as many of them
// as a uniform draw reaches; from call to call L2 keeps some), other widths follow them; dense N x K:
//   up to 16 rows by expert   8 of 8, 2    bf16 6 rows 6.5 (4 of 4: 7.2)
//   up to 128                 4 of 4, 2    integers 48 rows 19.2 (8 of 8: 21.9), bf16 96 rows 54.7 (55.7)
//   more                      1 of 4, 4    integers 384 rows 67.0 (4 of 4: 70.1), bf16 123.0 (126.3), floors 60 and 125
//   dense, a warp's share of  8 of 8, 4    bf16 4 x 2048 x 8192 8.8 (2 pieces: 9.8), 1 x 2048 x 2048 3.3 (3.6)
//     K is 4 pieces and more
//   dense, less               8 of 8, 2    integers 8 x 8192 x 2048 5.5 (4 pieces: 7.5)
// Shapes of 2 pieces have no registers for another set of sums (48 rows took 30.8 us with it, 28.8
// without), so their warps have up to ALONE products; a longer contraction by expert takes 4.
constexpr int ALONE = 1024;
template <bool INT8, bool GATED>
cudaError_t launch_shape(const ProductArgs& p, cudaStream_t st) {
  if (p.offsets == nullptr)
    return (long long)p.K * (INT8 ? 1 : 2) >= 8 * 4 * 128 ? launch<INT8, GATED, 8, 8, 4>(p, st)
                                                           : launch<INT8, GATED, 8, 8, 2>(p, st);
  if (p.M <= 16)
    return !INT8 && p.K > 8 * ALONE ? launch<INT8, GATED, 8, 8, 4>(p, st) : launch<INT8, GATED, 8, 8, 2>(p, st);
  if (p.M <= 128) {
    if constexpr (!INT8)
      if (p.K > 4 * ALONE) return launch<INT8, GATED, 4, 4, 4>(p, st);
    return launch<INT8, GATED, 4, 4, 2>(p, st);
  }
  return launch<INT8, GATED, 1, 4, 4>(p, st);
}

}  // namespace

cudaError_t launch_few_rows(const ProductArgs& p, bool int8, cudaStream_t st) {
  if (int8) return p.act != FFN_NONE ? launch_shape<true, true>(p, st) : launch_shape<true, false>(p, st);
  return p.act != FFN_NONE ? launch_shape<false, true>(p, st) : launch_shape<false, false>(p, st);
}

}  // namespace flint
