// Matrix product of FP8 (E4M3) operands with block scales, dense or grouped by
// expert:
//   y[m][n] = sum over kb of sa[kb][m] * sb[e][n / 128][kb] *
//             sum over k in block kb of a[m][k] * b[e][n][k]
// Each 128-long partial sum is formed by the tensor cores in fp32, then scaled
// and added in fp32.
#include "flint_common.cuh"
#include "flint_internal.h"

namespace flint {

namespace {

struct GemmArgs {
  const uint8_t* a;
  const float* sa;
  const uint8_t* b;
  const float* sb;
  const int32_t* offsets;
  void* y;
  int M, N, K, E, kb, nb;
};

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---- few rows: a CTA streams 16 weight rows once for up to 8 activation rows
// of one expert.  Grid (M, ceil(N / 16)): the CTA of row r works when r is the
// first of a run of 8 rows of its expert.  The K blocks go round the 8 warps.
// Both operands are read straight from global memory into mma fragments: the
// product of a block does not depend on the order of k, so lane t of a row's
// four takes bytes 16t..16t+15 of each half block for either operand.
constexpr int SK_WARPS = 8;

template <bool F32>
__global__ void __launch_bounds__(SK_WARPS * 32) block_gemm_skinny_kernel(const GemmArgs p) {
  __shared__ float red[SK_WARPS][128];
  __shared__ int range[3];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = blockIdx.x;
  int e = 0, r0 = r, r1 = p.M;
  if (p.offsets != nullptr) {
    // expert of row r: the number of groups that end at or before it
    if (warp == 0) {
      int ended = 0;
      for (int i = lane; i < p.E; i += 32) ended += __ldg(p.offsets + i + 1) <= r ? 1 : 0;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) ended += __shfl_xor_sync(0xffffffffu, ended, off);
      if (lane == 0) {
        range[0] = ended;
        range[1] = ended < p.E ? __ldg(p.offsets + ended) : 0;
        range[2] = ended < p.E ? min(__ldg(p.offsets + ended + 1), p.M) : 0;
      }
    }
    __syncthreads();
    e = range[0];
    if (e >= p.E) return;
    r0 = range[1];
    r1 = range[2];
    if (r < r0 || r >= r1) return;
  } else {
    r0 = 0;
  }
  if ((r - r0) & 7) return;
  const int n_rows = min(8, r1 - r);
  const int n0 = blockIdx.y * 16;
  const int g = lane >> 2, t = lane & 3;
  const int na = n0 + g, nb = n0 + g + 8;
  const uint8_t* b0 = p.b + ((size_t)e * p.N + min(na, p.N - 1)) * p.K;
  const uint8_t* b1 = p.b + ((size_t)e * p.N + min(nb, p.N - 1)) * p.K;
  const uint8_t* a0 = p.a + (size_t)(r + min(g, n_rows - 1)) * p.K;
  const float* sb = p.sb + ((size_t)e * p.nb + n0 / 128) * p.kb;
  const int c0 = min(2 * t, n_rows - 1), c1 = min(2 * t + 1, n_rows - 1);
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int kb = warp; kb < p.kb; kb += SK_WARPS) {
    const int k0 = kb * 128 + 16 * t, k1 = k0 + 64;
    const bool in0 = k0 < p.K, in1 = k1 < p.K;  // K is a multiple of 16
    const uint4 wa0 = in0 ? __ldg(reinterpret_cast<const uint4*>(b0 + k0)) : zero;
    const uint4 wb0 = in0 ? __ldg(reinterpret_cast<const uint4*>(b1 + k0)) : zero;
    const uint4 xa0 = in0 ? __ldg(reinterpret_cast<const uint4*>(a0 + k0)) : zero;
    const uint4 wa1 = in1 ? __ldg(reinterpret_cast<const uint4*>(b0 + k1)) : zero;
    const uint4 wb1 = in1 ? __ldg(reinterpret_cast<const uint4*>(b1 + k1)) : zero;
    const uint4 xa1 = in1 ? __ldg(reinterpret_cast<const uint4*>(a0 + k1)) : zero;
    const float s = __ldg(sb + kb);
    const float s0 = s * __ldg(p.sa + (size_t)kb * p.M + r + c0), s1 = s * __ldg(p.sa + (size_t)kb * p.M + r + c1);
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    mma_e4m3(d, wa0.x, wb0.x, wa0.y, wb0.y, xa0.x, xa0.y);
    mma_e4m3(d, wa0.z, wb0.z, wa0.w, wb0.w, xa0.z, xa0.w);
    mma_e4m3(d, wa1.x, wb1.x, wa1.y, wb1.y, xa1.x, xa1.y);
    mma_e4m3(d, wa1.z, wb1.z, wa1.w, wb1.w, xa1.z, xa1.w);
    acc[0] = fmaf(s0, d[0], acc[0]);
    acc[1] = fmaf(s1, d[1], acc[1]);
    acc[2] = fmaf(s0, d[2], acc[2]);
    acc[3] = fmaf(s1, d[3], acc[3]);
  }
  // red[warp][column * 16 + weight row]
  red[warp][(2 * t) * 16 + g] = acc[0];
  red[warp][(2 * t + 1) * 16 + g] = acc[1];
  red[warp][(2 * t) * 16 + g + 8] = acc[2];
  red[warp][(2 * t + 1) * 16 + g + 8] = acc[3];
  __syncthreads();
  if (tid < 128) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < SK_WARPS; ++w) v += red[w][tid];
    const int col = tid >> 4, n = n0 + (tid & 15);
    if (col < n_rows && n < p.N) {
      const size_t at = (size_t)(r + col) * p.N + n;
      if (F32)
        static_cast<float*>(p.y)[at] = v;
      else
        static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
    }
  }
}

}  // namespace

cudaError_t block_gemm_kernels_init() { return cudaSuccess; }

cudaError_t launch_block_gemm(const void* a, const float* sa, int M, const void* b, const float* sb, int E,
                              const int32_t* offsets, int N, int K, void* y, bool f32, int sm_count, unsigned* err,
                              cudaStream_t st) {
  GemmArgs p;
  p.a = static_cast<const uint8_t*>(a);
  p.sa = sa;
  p.b = static_cast<const uint8_t*>(b);
  p.sb = sb;
  p.offsets = offsets;
  p.y = y;
  p.M = M;
  p.N = N;
  p.K = K;
  p.E = E;
  p.kb = (K + 127) / 128;
  p.nb = (N + 127) / 128;
  (void)sm_count;
  (void)err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)M, (unsigned)((N + 15) / 16));
  cfg.blockDim = dim3(SK_WARPS * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return f32 ? cudaLaunchKernelEx(&cfg, block_gemm_skinny_kernel<true>, p)
             : cudaLaunchKernelEx(&cfg, block_gemm_skinny_kernel<false>, p);
}

}  // namespace flint
