// Gradients of the gated sums, in one pass over the rows.
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
  unsigned col_tiles;  // CTAs side by side
  int wide;            // log2 of a CTA's threads on a row
};

// dg = dh * u * act'(g), du = dh * act(g), formed in fp32 from the kept bf16 sums and
// rounded once to bf16, the type of the products that read them.  A thread takes 8
// outputs of a row; bound by HBM (5 values of 2 bytes an output).
__global__ void __launch_bounds__(256) gate_backward_kernel(const GateArgs p) {
  pdl_wait();
  pdl_trigger();
  const int live = p.offsets == nullptr ? p.M : min(max(__ldg(p.offsets + p.E), 0), p.M);
  const unsigned tile = blockIdx.x / p.col_tiles, at = blockIdx.x - tile * p.col_tiles;
  const size_t row = (size_t)tile * (256u >> p.wide) + (threadIdx.x >> p.wide);
  const int i = (int)((at << p.wide) + (threadIdx.x & ((1u << p.wide) - 1u))) * 8;
  if (row >= (size_t)live || i >= p.I) return;
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
  // as many threads on a row as leave at most an eighth of them without work
  const int per_row = I / 8;
  p.wide = 8;
  while (p.wide > 0 && (((per_row - 1) >> p.wide) + 1) * 8 << p.wide > per_row * 9) --p.wide;
  p.col_tiles = (unsigned)(((per_row - 1) >> p.wide) + 1);
  const unsigned row_tiles = (unsigned)(((long long)M + (256 >> p.wide) - 1) / (256 >> p.wide));
  return launch_pdl(gate_backward_kernel, p, dim3(row_tiles * p.col_tiles), 256, st);
}

}  // namespace flint
