// Gradients of the bf16 products: of the gated sums (one pass over the rows), of the
// input and of the weights.
#include "product_common.cuh"

namespace flint {

namespace {

__device__ __forceinline__ void unpack8(const uint4 r, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

struct GateArgs {
  const uint16_t* dh;
  const uint16_t* gu;
  const int32_t* offsets;
  uint16_t* dgu;
  int M, I, E, act;
};

// dg = dh * u * act'(g), du = dh * act(g), formed in fp32 from the kept bf16 sums and
// rounded once to bf16, the type of the products that read them.  A thread takes 8
// outputs of a row; bound by HBM (5 values of 2 bytes an output).
__global__ void __launch_bounds__(256) gate_backward_kernel(const GateArgs p) {
  pdl_wait();
  pdl_trigger();
  const unsigned per_row = (unsigned)p.I / 8;
  const int live = p.offsets == nullptr ? p.M : min(max(__ldg(p.offsets + p.E), 0), p.M);
  const size_t at = (size_t)blockIdx.x * 256 + threadIdx.x;
  const size_t row = at / per_row;
  if (row >= (size_t)live) return;
  const int i = (int)(at - row * per_row) * 8;
  const uint16_t* gu = p.gu + row * 2 * p.I + i;
  const uint4 rd = ldg_once(p.dh + row * p.I + i), rg = ldg_once(gu), ru = ldg_once(gu + p.I);
  float d[8], g[8], u[8], dg[8], du[8];
  unpack8(rd, d);
  unpack8(rg, g);
  unpack8(ru, u);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float a, slope;
    activation_slope(g[j], p.act, a, slope);
    dg[j] = d[j] * u[j] * slope;
    du[j] = d[j] * a;
  }
  uint16_t* out = p.dgu + row * 2 * p.I + i;
  *reinterpret_cast<uint4*>(out) = make_uint4(bf16x2_bits(dg[0], dg[1]), bf16x2_bits(dg[2], dg[3]),
                                              bf16x2_bits(dg[4], dg[5]), bf16x2_bits(dg[6], dg[7]));
  *reinterpret_cast<uint4*>(out + p.I) = make_uint4(bf16x2_bits(du[0], du[1]), bf16x2_bits(du[2], du[3]),
                                                    bf16x2_bits(du[4], du[5]), bf16x2_bits(du[6], du[7]));
}

// Tiles of 64 x 64 outputs, 16 of the contracted dimension at a time, in fp32.
//   WEIGHTS false: dx[m][k] = sum over n of dy[m][n] * w[e][n][k]; grid (M, tiles of K):
//     the block of row r works when r is the first of a run of 64 rows of its expert
//   WEIGHTS true: dw[e][n][k] = sum over the expert's rows m of dy[m][n] * x[m][k]; grid
//     (tiles of K, tiles of N, E)
template <bool WEIGHTS>
__global__ void __launch_bounds__(256) simple_gradient_kernel(const GradArgs p) {
  __shared__ float sa[16][65], sb[16][65];
  __shared__ int range[3];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  const uint16_t* dy = static_cast<const uint16_t*>(p.dy);
  const uint16_t* other = static_cast<const uint16_t*>(p.other);
  auto value = [](uint16_t v) { return __uint_as_float((uint32_t)v << 16); };
  int e = 0, lo = 0, hi = p.M;
  if (WEIGHTS) {
    e = blockIdx.z;
    if (p.offsets != nullptr) {
      lo = min(max(__ldg(p.offsets + e), 0), p.M);
      hi = min(max(__ldg(p.offsets + e + 1), lo), p.M);
    }
  } else {
    const int r = p.offsets == nullptr ? blockIdx.x * 64 : blockIdx.x;
    if (p.offsets != nullptr) {
      if (tid < 32) {
        const RowGroup g = group_of_row(p.offsets, p.E, p.M, r, tid);
        if (tid == 0) {
          range[0] = g.e;
          range[1] = g.lo;
          range[2] = g.hi;
        }
      }
      __syncthreads();
      e = range[0];
      if (e < 0 || e >= p.E || r < range[1] || r >= range[2] || (r - range[1]) % 64) return;
      hi = range[2];
    }
    lo = r;
  }
  const int k0 = (WEIGHTS ? blockIdx.x : blockIdx.y) * 64, o0 = WEIGHTS ? blockIdx.y * 64 : lo;
  const int o_end = WEIGHTS ? p.N : hi, c_begin = WEIGHTS ? lo : 0, c_end = WEIGHTS ? hi : p.N;
  float acc[4][4] = {};
  for (int c0 = c_begin; c0 < c_end; c0 += 16) {
    for (int i = tid; i < 1024; i += 256) {
      int c, o;
      if (WEIGHTS) {
        o = i & 63;
        c = i >> 6;
      } else {
        c = i & 15;
        o = i >> 4;
      }
      const int cc = c0 + c, oo = o0 + o;
      float v = 0.f;
      if (cc < c_end && oo < o_end) v = value(WEIGHTS ? dy[(size_t)cc * p.N + oo] : dy[(size_t)oo * p.N + cc]);
      sa[c][o] = v;
      const int kc = i >> 6, kk = k0 + (i & 63), ck = c0 + kc;
      v = 0.f;
      if (ck < c_end && kk < p.K)
        v = value(other[(WEIGHTS ? (size_t)ck : (size_t)e * p.N + ck) * p.K + kk]);
      sb[kc][i & 63] = v;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = sa[c][(tid >> 4) + 16 * i];
        b[i] = sb[c][(tid & 15) + 16 * i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int o = o0 + (tid >> 4) + 16 * i, k = k0 + (tid & 15) + 16 * j;
      if (o >= o_end || k >= p.K) continue;
      const size_t at = ((size_t)(WEIGHTS ? e * (size_t)p.N : 0) + o) * p.K + k;
      if (p.f32)
        static_cast<float*>(p.out)[at] = acc[i][j];
      else
        static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(acc[i][j]);
    }
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

cudaError_t launch_gate_backward(const void* dh, const void* gu, const int32_t* offsets, int M, int I, int E, int act,
                                 void* dgu, cudaStream_t st) {
  GateArgs p;
  p.dh = static_cast<const uint16_t*>(dh);
  p.gu = static_cast<const uint16_t*>(gu);
  p.offsets = offsets;
  p.dgu = static_cast<uint16_t*>(dgu);
  p.M = M;
  p.I = I;
  p.E = E;
  p.act = act;
  const size_t pieces = (size_t)M * (I / 8);
  return launch_pdl(gate_backward_kernel, p, dim3((unsigned)((pieces + 255) / 256)), 256, st);
}

cudaError_t launch_input_gradient(const GradArgs& p, cudaStream_t st) {
  const unsigned rows = p.offsets == nullptr ? (unsigned)(p.M + 63) / 64 : (unsigned)p.M;
  return launch_pdl(simple_gradient_kernel<false>, p, dim3(rows, (unsigned)(p.K + 63) / 64), 256, st);
}
cudaError_t launch_weight_gradient(const GradArgs& p, cudaStream_t st) {
  return launch_pdl(simple_gradient_kernel<true>, p,
                    dim3((unsigned)(p.K + 63) / 64, (unsigned)(p.N + 63) / 64, (unsigned)p.E), 256, st);
}

}  // namespace flint
