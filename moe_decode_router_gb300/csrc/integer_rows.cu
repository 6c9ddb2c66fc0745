// Rows to 8-bit integers with one scale each, written to every place that the routing
// gives a row.
#include "product_common.cuh"

namespace flint {

namespace {

// Smallest row maximum that a scale is made for.
constexpr float ROW_FLOOR = 1.262177448353618888658765704e-29f;  // 2^-96

struct IntRowsArgs {
  const void* x;
  long long stride;
  int rows, K;
  const int32_t* pos;
  int top_k, places;
  uint8_t* q;
  float* scales;
};

// The larger magnitude, NaN if either is.
__device__ __forceinline__ float max_magnitude(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// 16 values of a row as they lie: 2 (bf16) or 4 (fp32) pieces of 16 bytes.
template <bool BF16>
struct Raw16 {
  uint4 v[BF16 ? 2 : 4];
  __device__ __forceinline__ void load(const void* base, size_t at) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + at * (BF16 ? 2 : 4));
#pragma unroll
    for (int i = 0; i < (BF16 ? 2 : 4); ++i) v[i] = __ldg(s + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (BF16 ? 2 : 4); ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float value(int i) const {
    const uint4& w = v[BF16 ? i >> 3 : i >> 2];
    const int c = BF16 ? (i >> 1) & 3 : i & 3;
    const uint32_t b = c == 0 ? w.x : c == 1 ? w.y : c == 2 ? w.z : w.w;
    if (!BF16) return __uint_as_float(b);
    return __uint_as_float(i & 1 ? b & 0xFFFF0000u : b << 16);
  }
  // The largest magnitude, NaN if there is one: of bf16 two at a time.
  __device__ __forceinline__ float top() const {
    if (BF16) {
      uint32_t a = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4& w = v[i >> 2];
        const uint32_t b = ((i & 3) == 0 ? w.x : (i & 3) == 1 ? w.y : (i & 3) == 2 ? w.z : w.w) & 0x7FFF7FFFu;
        asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
      }
      return max_magnitude(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
    }
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = max_magnitude(a, value(i));
    return a;
  }
};

__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// The whole numbers next to v / s of two values, ties to even, in the low bytes.  v * (1 / s) is off
// by 2^-16 of a step at most, so only next to a border (one bf16 value in 200 is a tie) does the
// exact remainder v - n * s, a multiple of the scale's last bit, decide.  The kernel is bound by its
// instructions: in pairs, 8,192 rows of
// 4,096 take 19 us, one by one they took 25.
struct Scale {
  float s, near;               // near: remainders above are next to a border
  uint64_t inv, minus, magic;  // pairs of 1 / s, -s and 1.5 * 2^23, whose unit is 1
};
__device__ __forceinline__ float settle(float m, float rest, float s) {
  const float twice = 2.f * fabsf(rest);
  return twice > s || (twice == s && (__float_as_uint(m) & 1u)) ? m + copysignf(1.f, rest) : m;
}
__device__ __forceinline__ void codes_of(float v0, float v1, const Scale& k, uint32_t& c0, uint32_t& c1) {
  constexpr float MAGIC = 12582912.f;
  const uint64_t v = f2pack(v0, v1), m = fma_pair(v, k.inv, k.magic), n = f2add(m, f2pack(-MAGIC, -MAGIC));
  float m0, m1, r0, r1;
  f2unpack(m, m0, m1);
  f2unpack(fma_pair(n, k.minus, v), r0, r1);
  if (fmaxf(fabsf(r0), fabsf(r1)) > k.near) {
    m0 = settle(m0, r0, k.s);
    m1 = settle(m1, r1, k.s);
  }
  c0 = __float_as_uint(m0);
  c1 = __float_as_uint(m1);
}

// a = max(largest magnitude of the row, 2^-96), scale = a * (1 / 127) (both in fp32), code =
// the whole number next to x / scale.  THREADS lanes of a CTA of 256 have a row: each 16 neighbouring
// values at a time, the first HELD x 16 of them kept in registers between the two passes
// (a longer row is read a second time).  Bound by HBM.
template <bool BF16, int THREADS, int HELD>
__global__ void __launch_bounds__(256, HELD == 1 ? 5 : HELD == 2 ? 4 : 2) integer_rows_kernel(const IntRowsArgs p) {
  __shared__ float tops[8];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % THREADS, warp = threadIdx.x >> 5;
  const int row = blockIdx.x * (256 / THREADS) + threadIdx.x / THREADS;
  const bool in = row < p.rows;
  const size_t base = (size_t)row * (size_t)p.stride;
  constexpr int AT_ONCE = HELD == 1 ? 8 : 0;
  int to[8];  // the first places, on their way while the row is
  const int32_t* pos = p.pos + (size_t)row * p.top_k;
#pragma unroll
  for (int j = 0; j < AT_ONCE; ++j) to[j] = in && p.pos != nullptr && j < p.top_k ? __ldg(pos + j) : -1;
  Raw16<BF16> held[HELD];
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int k = (i * THREADS + lane) * 16;
    if (in && k < p.K) held[i].load(p.x, base + k);  // K is a multiple of 16
    else held[i].zero();
  }
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < HELD; ++i) a = max_magnitude(a, held[i].top());
  if (in)
    for (int k = (HELD * THREADS + lane) * 16; k < p.K; k += THREADS * 16) {
      Raw16<BF16> v;
      v.load(p.x, base + k);
      a = max_magnitude(a, v.top());
    }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) a = max_magnitude(a, __shfl_xor_sync(0xffffffffu, a, off));
  if (THREADS > 32) {
    if ((threadIdx.x & 31) == 0) tops[warp] = a;
    __syncthreads();
    constexpr int WARPS = THREADS / 32;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) a = max_magnitude(a, tops[warp / WARPS * WARPS + i]);
  }
  if (!in) return;
  if (a < ROW_FLOOR) a = ROW_FLOOR;  // false for NaN
  const float scale = __fmul_rn(a, 1.f / 127.f), inv = __frcp_rn(scale);
  const Scale steps = {scale, 0.4999f * scale, f2pack(inv, inv), f2pack(-scale, -scale), f2pack(12582912.f, 12582912.f)};
  const bool fine = scale < INFINITY;  // false for NaN: the codes of such a row are 0
  auto put = [&](const Raw16<BF16>& v, int k) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t b0, b1, b2, b3;
      codes_of(v.value(4 * i), v.value(4 * i + 1), steps, b0, b1);
      codes_of(v.value(4 * i + 2), v.value(4 * i + 3), steps, b2, b3);
      c[i] = fine ? __byte_perm(__byte_perm(b0, b1, 0x0040), __byte_perm(b2, b3, 0x0040), 0x5410) : 0u;
    }
    const uint4 codes = make_uint4(c[0], c[1], c[2], c[3]);
    if (p.pos == nullptr) {
      *reinterpret_cast<uint4*>(p.q + (size_t)row * p.K + k) = codes;
      return;
    }
    auto store = [&](int place) {
      if (place >= 0 && place < p.places) *reinterpret_cast<uint4*>(p.q + (size_t)place * p.K + k) = codes;
    };
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) store(to[j]);
    for (int j = AT_ONCE; j < p.top_k; ++j) store(__ldg(pos + j));
  };
#pragma unroll
  for (int i = 0; i < HELD; ++i) {
    const int k = (i * THREADS + lane) * 16;
    if (k < p.K) put(held[i], k);
  }
  for (int k = (HELD * THREADS + lane) * 16; k < p.K; k += THREADS * 16) {
    Raw16<BF16> v;
    v.load(p.x, base + k);
    put(v, k);
  }
  if (p.pos == nullptr) {
    if (lane == 0) p.scales[row] = scale;
  } else if (lane < p.top_k) {
    const int place = __ldg(pos + lane);
    if (place >= 0 && place < p.places) p.scales[place] = scale;
  }
}

template <bool BF16, int THREADS, int HELD>
cudaError_t launch(const IntRowsArgs& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.rows + 256 / THREADS - 1) / (256 / THREADS)));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, integer_rows_kernel<BF16, THREADS, HELD>, p);
}

}  // namespace

cudaError_t launch_integer_rows(const void* x, bool bf16, long long stride, int rows, int K, const int32_t* pos,
                                int top_k, int places, void* q, float* scales, cudaStream_t st) {
  IntRowsArgs p;
  p.x = x;
  p.stride = stride;
  p.rows = rows;
  p.K = K;
  p.pos = pos;
  p.top_k = top_k;
  p.places = places;
  p.q = static_cast<uint8_t*>(q);
  p.scales = scales;
  // Threads on a row and pieces of 16 each of them keeps, measured (us, bf16; the second digits the next best).
  // fp32 rows, four registers a piece more, take the same: with two pieces they spill 32 bytes a thread,
  // and 8,192 rows of 4096 take 29 us (floor 25), 49,152 of 1408 62 (51), of 512 21 (18.5).
  //   K 512, 49,152 rows             32, 1   15.0 (32, 2: 16.3)
  //   K 1024, 8,192 rows to 2 places  32, 2    6.4 (64, 1: 7.3)
  //   K 1408, 49,152 rows            64, 2   48.8 (32, 4: 53.7)
  //   K 2048, 8,191 rows to 6 places 128, 1   22.7 (64, 2: 24.5); 300 rows 2.7 (3.6)
  //   K 4096, 8,192 rows            128, 2   19.2 (256, 1: 23.3)
  //   K 8192, 4,096 rows            256, 2   19.0 (256, 4: 34)
  if (K <= 512) return bf16 ? launch<true, 32, 1>(p, st) : launch<false, 32, 1>(p, st);
  if (K <= 1024) return bf16 ? launch<true, 32, 2>(p, st) : launch<false, 32, 2>(p, st);
  if (K <= 1792 && rows > 1024) return bf16 ? launch<true, 64, 2>(p, st) : launch<false, 64, 2>(p, st);
  if (K <= 2048) return bf16 ? launch<true, 128, 1>(p, st) : launch<false, 128, 1>(p, st);
  if (K <= 4096) return bf16 ? launch<true, 128, 2>(p, st) : launch<false, 128, 2>(p, st);
  if (K <= 8192) return bf16 ? launch<true, 256, 2>(p, st) : launch<false, 256, 2>(p, st);
  return bf16 ? launch<true, 256, 4>(p, st) : launch<false, 256, 4>(p, st);
}

}  // namespace flint
