// Row-wise operators around the FP8 expert products: quantisation of rows in
// blocks of 128 (with the gated activation in the same pass, and written to
// every place that the routing gives a row), and the weighted combine.
#include "flint_common.cuh"
#include "flint_internal.h"

namespace flint {

namespace {

__device__ __forceinline__ void bf16x8_to_f32(const uint4 r, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <bool BF16>
__device__ __forceinline__ void load8(const void* base, size_t at, float (&v)[8]) {
  if (BF16) {
    bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at)), v);
  } else {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = __ldg(s), b = __ldg(s + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Smallest block maximum that a scale is made for: 448 / 2^-96 stays finite.
constexpr float Q_FLOOR = 1.262177448353618888658765704e-29f;  // 2^-96
constexpr float E4M3_TOP = 448.f;

struct QuantParams {
  const void* x;
  long long stride;
  int rows, K;
  unsigned col_tiles;  // CTAs side by side
  int wide;            // log2 of a CTA's block columns
  const int32_t* pos;
  int top_k;
  int places;  // rows of q and of a scale line
  uint8_t* q;
  float* scales;
};

__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// The larger magnitude, NaN if either is.
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// 8 lanes per block of 128, 16 values each.  A CTA has 32 blocks: 2^wide
// neighbouring block columns of 32 / 2^wide rows, as wide as the row's blocks
// divide evenly, so that a row's bytes are read and written together.  The
// block's largest magnitude a (NaN if the block holds one) gives scale = a / 448
// and codes e4m3(x * (448 / a)), one rounding to nearest even.
//
// Bound by HBM.  8,192 x 2,048 bf16 to six places each 24.5 us, 5.6 TB/s (the
// scattered scales cost 3 us of it); 49,152 gated rows of 512 22.0 us, 5.8 TB/s.
template <bool BF16, bool SILU>
__global__ void __launch_bounds__(256) quantize_kernel(const QuantParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 7;
  const unsigned tile = blockIdx.x / p.col_tiles, u = threadIdx.x >> 3;
  const int b = (int)(((blockIdx.x - tile * p.col_tiles) << p.wide) + (u & ((1u << p.wide) - 1u)));
  const int row = (int)(tile * (32u >> p.wide) + (u >> p.wide));
  const int k = b * 128 + lane * 16;
  const bool in = row < p.rows && k < p.K;  // K is a multiple of 16
  constexpr int AT_ONCE = 8;
  int to[AT_ONCE];  // the first places, on their way while the row is
  const int32_t* pos = p.pos + (size_t)row * p.top_k;
  if (p.pos != nullptr) {
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) to[j] = in && j < p.top_k ? __ldg(pos + j) : -1;
  }
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.f;
  if (in) {
    const size_t at = (size_t)row * (size_t)p.stride + (size_t)k;
    float* lo = v;
    load8<BF16>(p.x, at, *reinterpret_cast<float(*)[8]>(lo));
    load8<BF16>(p.x, at + 8, *reinterpret_cast<float(*)[8]>(lo + 8));
    if (SILU) {
      float u[16];
      load8<BF16>(p.x, at + (size_t)p.K, *reinterpret_cast<float(*)[8]>(u));
      load8<BF16>(p.x, at + (size_t)p.K + 8, *reinterpret_cast<float(*)[8]>(u + 8));
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = v[i] * rcp_approx(1.f + __expf(-v[i])) * u[i];
    }
  }
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) a = max_abs(a, v[i]);
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) a = max_abs(a, __shfl_xor_sync(0xffffffffu, a, off));
  if (a < Q_FLOOR) a = Q_FLOOR;  // false for NaN
  const float scale = __fdiv_rn(a, E4M3_TOP), r = __fdiv_rn(E4M3_TOP, a);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = e4m3x2(v[4 * i] * r, v[4 * i + 1] * r) | (e4m3x2(v[4 * i + 2] * r, v[4 * i + 3] * r) << 16);
  if (!in) return;
  const uint4 code = make_uint4(c[0], c[1], c[2], c[3]);
  uint8_t* q = p.q + k;
  float* scales = p.scales + (size_t)b * p.places;
  auto put = [&](int place) {
    if (place < 0 || place >= p.places) return;
    *reinterpret_cast<uint4*>(q + (size_t)place * p.K) = code;
    if (lane == 0) scales[place] = scale;
  };
  if (p.pos == nullptr) {
    put(row);
    return;
  }
#pragma unroll
  for (int j = 0; j < AT_ONCE; ++j) put(to[j]);
  for (int j = AT_ONCE; j < p.top_k; ++j) put(__ldg(pos + j));
}

struct CombineParams {
  const void* rows;
  long long n_rows;
  const int32_t* pos;
  const float* w;
  const uint16_t* shared;
  uint16_t* y;
  int T, N, top_k;
};

// One thread per 8 outputs of a token; the sum runs over the choices in order,
// then the shared row, in fp32, and is rounded once to bf16.  Bound by HBM:
// AT_ONCE choices' rows are under way at a time.  8,192 tokens x 6 rows of 2,048
// with a shared row 43.3 us, 6.1 TB/s (47.4 us with one row at a time).
template <bool BF16>
__global__ void __launch_bounds__(128) combine_kernel(const CombineParams p) {
  constexpr int AT_ONCE = BF16 ? 8 : 4, WORDS = BF16 ? 1 : 2;
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x, n = (blockIdx.y * 128 + threadIdx.x) * 8;
  if (n >= p.N) return;
  const int32_t* pos = p.pos + (size_t)t * p.top_k;
  const float* w = p.w + (size_t)t * p.top_k;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 sh = zero;
  if (p.shared != nullptr) sh = __ldg(reinterpret_cast<const uint4*>(p.shared + (size_t)t * p.N + n));
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int j0 = 0; j0 < p.top_k; j0 += AT_ONCE) {
    uint4 raw[AT_ONCE][WORDS];
    float f[AT_ONCE];
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      const int r = j0 + j < p.top_k ? __ldg(pos + j0 + j) : -1;
      const bool on = r >= 0 && r < p.n_rows;
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.rows) +
                                                        ((size_t)(on ? r : 0) * p.N + n) * (BF16 ? 2 : 4));
      f[j] = on ? __ldg(w + j0 + j) : 0.f;
#pragma unroll
      for (int i = 0; i < WORDS; ++i) raw[j][i] = on ? __ldg(src + i) : zero;
    }
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      if (j0 + j >= p.top_k) break;
      float v[8];
      if (BF16) {
        bf16x8_to_f32(raw[j][0], v);
      } else {
        const uint32_t u[8] = {raw[j][0].x,         raw[j][0].y,         raw[j][0].z,         raw[j][0].w,
                               raw[j][WORDS - 1].x, raw[j][WORDS - 1].y, raw[j][WORDS - 1].z, raw[j][WORDS - 1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(f[j], v[i], acc[i]);
    }
  }
  float s[8];
  bf16x8_to_f32(sh, s);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(acc[2 * i] + s[2 * i], acc[2 * i + 1] + s[2 * i + 1]);
    o[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p.y + (size_t)t * p.N + n) = make_uint4(o[0], o[1], o[2], o[3]);
}

template <typename P>
cudaError_t launch_pdl(void (*kernel)(const P), const P& p, dim3 ctas, int threads, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = ctas;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_quantize_rows(const void* x, bool bf16, long long stride, int rows, int K, bool silu,
                                 const int32_t* pos, int top_k, long long places, void* q, float* scales,
                                 cudaStream_t st) {
  QuantParams p;
  p.x = x;
  p.stride = stride;
  p.rows = rows;
  p.K = K;
  p.pos = pos;
  p.top_k = top_k;
  p.places = (int)places;
  p.q = static_cast<uint8_t*>(q);
  p.scales = scales;
  // As many block columns as leave at most an eighth of the CTA's places unused.
  const int kb = (K + 127) / 128;
  p.wide = 5;
  while (p.wide > 0 && (((kb - 1) >> p.wide) + 1) * 8 << p.wide > kb * 9) --p.wide;
  p.col_tiles = (unsigned)(((kb - 1) >> p.wide) + 1);
  const unsigned row_tiles = ((unsigned)rows + (32u >> p.wide) - 1) / (32u >> p.wide);
  const dim3 ctas(row_tiles * p.col_tiles);
  if (bf16) return silu ? launch_pdl(quantize_kernel<true, true>, p, ctas, 256, st)
                        : launch_pdl(quantize_kernel<true, false>, p, ctas, 256, st);
  return silu ? launch_pdl(quantize_kernel<false, true>, p, ctas, 256, st)
              : launch_pdl(quantize_kernel<false, false>, p, ctas, 256, st);
}

cudaError_t launch_combine(const void* rows, bool bf16, long long n_rows, const int32_t* pos, const float* w, int T,
                           int top_k, int N, const void* shared, void* y, cudaStream_t st) {
  CombineParams p;
  p.rows = rows;
  p.n_rows = n_rows;
  p.pos = pos;
  p.w = w;
  p.shared = static_cast<const uint16_t*>(shared);
  p.y = static_cast<uint16_t*>(y);
  p.T = T;
  p.N = N;
  p.top_k = top_k;
  const dim3 ctas((unsigned)T, (unsigned)((N / 8 + 127) / 128));
  return bf16 ? launch_pdl(combine_kernel<true>, p, ctas, 128, st) : launch_pdl(combine_kernel<false>, p, ctas, 128, st);
}

}  // namespace flint
