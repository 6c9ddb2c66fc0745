// Matrix product of FP8 (E4M3) operands with block scales, dense or grouped by
// expert:
//   y[m][n] = sum over kb of sa[kb][m] * sb[e][n / 128][kb] *
//             sum over k in block kb of a[m][k] * b[e][n][k]
// Each 128-long partial sum is formed by the tensor cores in fp32, then scaled
// and added in fp32.
#include <cuda.h>

#include <type_traits>

#include "flint_common.cuh"
#include "flint_internal.h"
#include "tc05_e4m3.cuh"

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

// 16 bytes of weights: read once, so not kept in L1.
__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---- few rows: weights are streamed once for up to 8 activation rows of one
// expert.  Grid (M, N / rows of a CTA): the CTA of row r works when r is the
// first of a run of 8 rows of its expert.  With SPLIT 8 a dense product has CTAs
// for every eighth row alone (SPLIT 1 sees grouped rows only, where this choice
// alone cost 1.4 of 21 us).  A warp takes 16 weight rows and every SPLIT-th K block of
// them; SPLIT warps of a CTA share 16 rows, so that a small product has enough
// warps (SPLIT 8) and a large one few sums across warps (SPLIT 1).  Both operands
// are read straight from global memory into mma fragments: the product of a
// block does not depend on the order of k, so lane t of a row's four takes bytes
// 16t..16t+15 of each half block for either operand.  Two K blocks (4 KB of
// weights a warp) are under way at a time.

template <int SPLIT, int SK_WARPS, bool F32>
__global__ void __launch_bounds__(SK_WARPS * 32, 24 / SK_WARPS) block_gemm_skinny_kernel(const GemmArgs p) {
  __shared__ float red[SPLIT == 1 ? 1 : SK_WARPS][128];
  __shared__ int range[3];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = SPLIT > 1 && p.offsets == nullptr ? blockIdx.x * 8 : blockIdx.x;
  int e = 0, r0 = 0, r1 = p.M;
  if (p.offsets != nullptr) {
    // expert of row r: the last group that starts at or before it; its range: the
    // offsets on either side of r
    if (warp == 0) {
      unsigned begun = 0, from = 0, to = (unsigned)p.M;
      for (int i = lane; i <= p.E; i += 32) {
        const int o = __ldg(p.offsets + i);
        if (o <= r) {
          ++begun;
          from = max(from, (unsigned)max(o, 0));
        } else {
          to = min(to, (unsigned)o);
        }
      }
      begun = __reduce_add_sync(0xffffffffu, begun);
      from = redux_max(from);
      to = redux_min(to);
      if (lane == 0) {
        range[0] = (int)begun - 1;
        range[1] = (int)from;
        range[2] = (int)to;
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
  const int n0 = (blockIdx.y * (SK_WARPS / SPLIT) + warp / SPLIT) * 16;
  const int g = lane >> 2, t = lane & 3;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (n0 < p.N) {
    const int na = n0 + g, nb = n0 + g + 8;
    const uint8_t* b0 = p.b + ((size_t)e * p.N + na) * p.K;
    const uint8_t* b1 = p.b + ((size_t)e * p.N + min(nb, p.N - 1)) * p.K;  // N is a multiple of 8
    const uint8_t* a0 = p.a + (size_t)(r + min(g, n_rows - 1)) * p.K;
    const float* sb = p.sb + ((size_t)e * p.nb + n0 / 128) * p.kb;
    const int c0 = min(2 * t, n_rows - 1), c1 = min(2 * t + 1, n_rows - 1);
    constexpr int U = 2;
    for (int kb0 = warp % SPLIT; kb0 < p.kb; kb0 += U * SPLIT) {
      uint4 w[U][4], x[U][2];
      float s0[U], s1[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int kb = kb0 + i * SPLIT, k0 = kb * 128 + 16 * t, k1 = k0 + 64;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        const bool in0 = k0 < p.K, in1 = k1 < p.K;  // K is a multiple of 16
        w[i][0] = in0 ? ldg_stream(b0 + k0) : zero;
        w[i][1] = in0 ? ldg_stream(b1 + k0) : zero;
        w[i][2] = in1 ? ldg_stream(b0 + k1) : zero;
        w[i][3] = in1 ? ldg_stream(b1 + k1) : zero;
        x[i][0] = in0 ? __ldg(reinterpret_cast<const uint4*>(a0 + k0)) : zero;
        x[i][1] = in1 ? __ldg(reinterpret_cast<const uint4*>(a0 + k1)) : zero;
        s0[i] = s1[i] = 0.f;
        if (kb < p.kb) {
          const float s = __ldg(sb + kb);
          s0[i] = s * __ldg(p.sa + (size_t)kb * p.M + r + c0);
          s1[i] = s * __ldg(p.sa + (size_t)kb * p.M + r + c1);
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (kb0 + i * SPLIT >= p.kb) break;
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma_e4m3(d, w[i][0].x, w[i][1].x, w[i][0].y, w[i][1].y, x[i][0].x, x[i][0].y);
        mma_e4m3(d, w[i][0].z, w[i][1].z, w[i][0].w, w[i][1].w, x[i][0].z, x[i][0].w);
        mma_e4m3(d, w[i][2].x, w[i][3].x, w[i][2].y, w[i][3].y, x[i][1].x, x[i][1].y);
        mma_e4m3(d, w[i][2].z, w[i][3].z, w[i][2].w, w[i][3].w, x[i][1].z, x[i][1].w);
        acc[0] = fmaf(s0[i], d[0], acc[0]);
        acc[1] = fmaf(s1[i], d[1], acc[1]);
        acc[2] = fmaf(s0[i], d[2], acc[2]);
        acc[3] = fmaf(s1[i], d[3], acc[3]);
      }
    }
  }
  auto store = [&](int col, int n, float v) {
    if (col < n_rows && n < p.N) {
      const size_t at = (size_t)(r + col) * p.N + n;
      if (F32)
        static_cast<float*>(p.y)[at] = v;
      else
        static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
    }
  };
  if constexpr (SPLIT == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) store(2 * t + (i & 1), n0 + g + (i >> 1) * 8, acc[i]);
  } else {
    // red[warp][column * 16 + weight row]
#pragma unroll
    for (int i = 0; i < 4; ++i) red[warp][(2 * t + (i & 1)) * 16 + g + (i >> 1) * 8] = acc[i];
    __syncthreads();
    for (int o = tid; o < 128 * (SK_WARPS / SPLIT); o += SK_WARPS * 32) {
      const int tile = o >> 7, c = o & 127;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < SPLIT; ++w) v += red[tile * SPLIT + w][c];
      store(c >> 4, (blockIdx.y * (SK_WARPS / SPLIT) + tile) * 16 + (c & 15), v);
    }
  }
}

template <int SPLIT, int SK_WARPS, bool F32>
cudaError_t launch_skinny(const GemmArgs& p, cudaStream_t st) {
  constexpr int ROWS = SK_WARPS / SPLIT * 16;
  cudaLaunchConfig_t cfg = {};
  const bool eighths = SPLIT > 1 && p.offsets == nullptr;
  cfg.gridDim = dim3((unsigned)(eighths ? (p.M + 7) / 8 : p.M), (unsigned)((p.N + ROWS - 1) / ROWS));
  cfg.blockDim = dim3(SK_WARPS * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_gemm_skinny_kernel<SPLIT, SK_WARPS, F32>, p);
}

// ---- many rows: tcgen05.
//
// The block scales allow the tensor cores 128 of K at a time: every K block is
// a fresh accumulator in tensor memory, and eight promotion warps read it back
// and add it, scaled, into fp32 registers while the next blocks are multiplied.
// An accumulator is free again only after its MMAs, a barrier, the read and a
// barrier back, and a barrier costs some 100 cycles on either side: the hand-over
// stays inside one SM (with cta_group::2 it crosses SMs, which took 1.2 times as
// long), nothing else is waited for on the way (the scales come through a ring in
// shared memory), and the MMAs of the next block cover it.  Two arrangements of
// the same pipeline:
//
// TALL (long groups).  128 rows of a are the M side and 256 weight rows the N
// side.  A thread holds one row of a (its tensor-memory lane) and 128 outputs,
// all with one scale a K block, the product of the row's and the weight
// block's: per K block and SM 512 cycles of MMA, 256 of tensor-memory reads
// (32x32b; the 16-lane forms read at half that rate) and 256 of packed fma,
// which overlap.  Every CTA loads its own 48 KB a K block; sharing the weight tile
// between two CTAs gains little (8191 x 4096 x 4096 107 us either way, ragged
// experts 146 shared, 147 alone with weights from HBM) and ties their steps together.
//
// WIDE (short groups).  128 weight rows are the M side, always full, and up to
// 64 rows of a the N side in steps of 16, so that a group of few rows costs
// little more than its weights' bytes.  Scales differ by column: tensor memory
// is read in 16x256b form, where a thread holds 4 weight rows x pairs of
// neighbouring columns, so that a pair of column scales, read once from a ring
// in shared memory, serves 4 packed fma.  A K block takes a CTA some 0.33 us
// however few units there are, so where units leave SMs idle KS = 2 or 4 CTAs of
// a cluster share a unit's K blocks.  Each leaves its partial sums in its own
// stages, and after a cluster barrier adds its part of the unit's columns over
// all of them, in the CTAs' order: the result is the same on every call.
//
// Warps: 0-7 promotion and output, two column halves; 8 TMA producer; 9 MMA
// issuer; 10 loader of scales; 11 nothing but its registers.
constexpr int TC_THREADS = 384;
// Registers of TALL: the promotion warps hold 128 accumulators each and take
// what the other four warps give up.  Launched with 168 a thread.
constexpr int TC_REGS = 168, TC_REGS_LOW = 48, TC_REGS_HIGH = 224;
static_assert(TC_REGS_HIGH * 256 + TC_REGS_LOW * 128 <= TC_REGS * TC_THREADS, "register shares");

template <bool TALL>
struct TcCfg {
  static constexpr int ROWS = TALL ? 128 : 64;     // rows of a in a unit
  static constexpr int WROWS = TALL ? 256 : 128;   // weight rows in a unit
  static constexpr int ACC = TALL ? 256 : 64;      // columns of an accumulator
  static constexpr int NBUF = 512 / ACC;
  static constexpr int X_BYTES = TALL ? 128 * 128 : 64 * 128;  // rows of a in a stage
  static constexpr int W_BYTES = WROWS * 128;
  static constexpr int STAGE = X_BYTES + W_BYTES;
  static constexpr int STAGES = TALL ? 3 : 8;
  // Scale ring.  TALL: a slot has 4 K blocks, a scale for each of the CTA's 128
  // rows, then one for each half of the weight tile.  WIDE: one K block, a scale
  // for each column, then the weights'.
  static constexpr int SLOTS = TALL ? 2 : 4;
  static constexpr int SLOT_FLOATS = TALL ? 4 * 128 + 8 : ACC + 4;
  static constexpr int X_BOX = TALL ? 128 : 32;    // rows of a in one copy
  static constexpr int OUT_WARP = TALL ? 8192 : 32 * 80;  // output staging: 32 rows a warp
  static constexpr int OFF_OUT = STAGES * STAGE;
  static constexpr int OFF_SCALE = OFF_OUT + 8 * OUT_WARP;
  static constexpr int OFF_BARS = OFF_SCALE + SLOTS * SLOT_FLOATS * 4;
  static constexpr int OFF_GROUPS = OFF_BARS + 512;
  static constexpr int smem(int E) { return OFF_GROUPS + (3 * E + 1) * 4; }
  static_assert(OFF_GROUPS + (3 * ROUTE_MAX_E + 1) * 4 <= 232448, "shared memory");
  static_assert(X_BYTES % 1024 == 0 && W_BYTES % 1024 == 0, "swizzle atoms");
};

struct TcArgs {
  const float* sa;
  const float* sb;
  const int32_t* offsets;
  void* y;
  unsigned* err;
  int M, N, E, kb, nb, n_tiles;  // n_tiles: weight tiles
  unsigned n_tiles_recip;        // ceil(2^32 / n_tiles)
};

struct TcUnit {
  int e, wt, row0, cnt, n;  // n: columns of the MMAs
};

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint32_t bf16_pair(uint64_t v) {
  float lo, hi;
  f2unpack(v, lo, hi);
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Output of WIDE: `groups` (up to 4, known when unrolled) groups of 8 columns of a
// warp's half, the first the `first`-th; acc as the promotion warps hold them, from 0.
template <bool F32>
__device__ __forceinline__ void wide_output(const TcArgs& p, const TcUnit& t, const uint64_t (&acc)[2][8], int first,
                                            int groups, uint8_t* out, int quad, int half, int lane) {
  const int g = lane >> 2, q = lane & 3, nh = t.n >> 1;
  const int n0 = t.wt * 128 + quad * 32;  // first weight row of the warp
  if (F32) {
    float* y = static_cast<float*>(p.y);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int cl = (first + (i >> 1)) * 8 + 2 * q, col = half * nh + cl;
      if ((i >> 1) >= groups) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v0, v1;
        f2unpack(acc[h][i], v0, v1);
        const int n = n0 + 16 * h + (i & 1) * 8 + g;
        if (n < p.N && cl < nh) {
          if (col < t.cnt) y[(size_t)(t.row0 + col) * p.N + n] = v0;
          if (col + 1 < t.cnt) y[(size_t)(t.row0 + col + 1) * p.N + n] = v1;
        }
      }
    }
  } else {
    // 8 x 8 transposes on the way into shared memory; four lanes store 32 columns of a row of y
    uint16_t* y = static_cast<uint16_t*>(p.y);
    const uint32_t st = smem_u32(out) + (lane & 7) * 80 + (lane >> 3) * 16;  // row lane % 8 of matrix lane / 8
    const uint4* ld = reinterpret_cast<const uint4*>(out + (lane >> 2) * 80 + (lane & 3) * 16);
    const int n = n0 + (lane & 3) * 8;
#pragma unroll
    for (int k = 0; k < 4; ++k)  // weight rows 0-7, 8-15, 16-23, 24-31 of the warp x 8 rows of y
      if (k < groups)
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(st + k * 640),
                     "r"(bf16_pair(acc[0][2 * k])), "r"(bf16_pair(acc[0][2 * k + 1])), "r"(bf16_pair(acc[1][2 * k])),
                     "r"(bf16_pair(acc[1][2 * k + 1]))
                     : "memory");
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int cl = (first + k) * 8 + (lane >> 2), col = half * nh + cl;
      if (k < groups && cl < nh && col < t.cnt && n < p.N)
        *reinterpret_cast<uint4*>(y + (size_t)(t.row0 + col) * p.N + n) = ld[40 * k];
    }
    __syncwarp();
  }
}

template <bool TALL, bool F32, int KS>
__global__ void __launch_bounds__(TC_THREADS, 1)
    block_gemm_tc_kernel(const TcArgs p, const __grid_constant__ CUtensorMap map_w,
                         const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_y) {
  using C = TcCfg<TALL>;
  static_assert(KS == 1 || !TALL, "K is split for WIDE alone");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::OFF_BARS);  // [STAGES] operands landed
  uint64_t* empty = full + C::STAGES;                              // [STAGES] stage consumed
  uint64_t* tfull = empty + C::STAGES;                             // [NBUF] accumulator complete
  uint64_t* tempty = tfull + C::NBUF;                              // [NBUF] accumulator read
  uint64_t* sfull = tempty + C::NBUF;                              // [SLOTS] scales landed
  uint64_t* sempty = sfull + C::SLOTS;                             // [SLOTS] scales read
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sempty + C::SLOTS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  static_assert((2 * C::STAGES + 2 * C::NBUF + 2 * C::SLOTS) * 8 + 8 <= 512, "barriers");
  int* g_units = reinterpret_cast<int*>(sm + C::OFF_GROUPS);  // [E + 1] units before each group
  int* g_lo = g_units + p.E + 1;                              // [E] first row
  int* g_cnt = g_lo + p.E;                                    // [E] rows

  if (warp == 8) {
    tc05::tmem_alloc(tslot, 512);
    tc05::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::NBUF; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 8);
    }
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(&sfull[i], 32);
      mbar_init(&sempty[i], 8);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_trigger();
  // groups: rows, and units before each
  if (p.offsets != nullptr)
    for (int e = tid; e <= p.E; e += TC_THREADS) g_units[e] = __ldg(p.offsets + e);  // all on their way at once
  __syncthreads();
  if (warp == 8) {
    int base = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int lo = 0, cnt = 0;
      if (e < p.E) {
        lo = p.offsets ? min(max(g_units[e], 0), p.M) : 0;
        cnt = p.offsets ? min(max(g_units[e + 1], lo), p.M) - lo : p.M;
        g_lo[e] = lo;
        g_cnt[e] = cnt;
      }
      __syncwarp();  // the offsets of these groups make room for their units; the next group's first is read below
      int t = (cnt + C::ROWS - 1) / C::ROWS * p.n_tiles;
      if (base > 1 << 29) t = 0;  // offsets that descend could count rows over and over: stay inside int
      int incl = t;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
      }
      if (e < p.E) g_units[e] = base + incl - t;
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) g_units[p.E] = base;
  }
  tc05::fence_before_sync();
  __syncthreads();
  tc05::fence_after_sync();
  const uint32_t tmem = *tslot;
  const int n_units = g_units[p.E];
  // with K split one unit alone, whatever the offsets say
  const int u0 = blockIdx.x / KS, ustep = KS > 1 ? 1 << 30 : gridDim.x;
  // this CTA's K blocks
  const int split = KS > 1 ? (int)tc05::cluster_rank() : 0, share = (p.kb + KS - 1) / KS;
  const int kb_from = KS > 1 ? min(split * share, p.kb) : 0, kb_to = KS > 1 ? min(kb_from + share, p.kb) : p.kb;

  auto unit_of = [&](int u) -> TcUnit {
    // The group is the last whose first unit is at or before u: the whole warp
    // looks, at every 32nd group and then at 32 neighbours (a binary search of
    // 256 groups takes 1,000 cycles).
    TcUnit t;
    int from = 0;
    if (p.E > 32) from = 32 * (__popc(__ballot_sync(0xffffffffu, 32 * lane < p.E && g_units[32 * lane] <= u)) - 1);
    const int e = from + lane;
    const int lo = from + __popc(__ballot_sync(0xffffffffu, e < p.E && g_units[e] <= u)) - 1;
    t.e = lo;
    const int cnt = g_cnt[lo], v = u - g_units[lo];
    int tile = v;  // v / n_tiles
    if (p.n_tiles > 1) {
      tile = (int)__umulhi((unsigned)v, p.n_tiles_recip);  // too large by one at most
      if (tile * p.n_tiles > v) --tile;
    }
    t.wt = v - tile * p.n_tiles;
    if (TALL) {
      // Two row tiles of a group go side by side, so that both ask for a weight tile at
      // about the same time: ragged experts 142.2 -> 141.4 us against one after the other.
      const int first = tile & ~1;
      if ((first + 1) * C::ROWS < cnt) {
        const int r = v - first * p.n_tiles;
        t.wt = r >> 1;
        tile = first + (r & 1);
      }
    }
    t.row0 = g_lo[lo] + tile * C::ROWS;
    t.cnt = min(C::ROWS, cnt - tile * C::ROWS);
    t.n = TALL ? min(256, (p.N - t.wt * 256 + 15) & ~15) : (t.cnt + 15) & ~15;
    return t;
  };
  // Bounded wait.  Lanes of a warp that wait together agree on the result: the
  // awaited phase cannot move on without a later arrival of this same warp.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (mbar_wait(bar, parity)) return true;
    atomicOr(p.err, ERR_WAIT_FULL);
    *abort_flag = 1;
    return false;
  };

  if (warp >= 8) {
    if (TALL) tc05::regs_down<TC_REGS_LOW>();
    if (warp == 8) {
      // ---------------- producer
      uint32_t s = 0, ph = 0, issued = 0;  // of lane 0, which copies
      bool ok = true;
      for (int u = u0; u < n_units && ok; u += ustep) {
        const TcUnit t = unit_of(u);
        const int boxes = TALL ? 1 : (t.n + 31) >> 5;
        const uint32_t bytes = C::W_BYTES + boxes * C::X_BOX * 128;
        for (int kb = kb_from; kb < kb_to && lane == 0; ++kb) {
          if (!wait(&empty[s], ph ^ 1)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], bytes);
          const uint32_t w = smem_u32(sm) + s * C::STAGE, x = w + C::W_BYTES;
          if (TALL) {
            tma_3d(w, &map_w, kb * 128, t.wt * 256, t.e, &full[s]);
            tma_3d(w + 16384, &map_w, kb * 128, t.wt * 256 + 128, t.e, &full[s]);
            tma_2d(x, &map_x, kb * 128, t.row0, &full[s]);
          } else {
            tma_3d(w, &map_w, kb * 128, t.wt * 128, t.e, &full[s]);
            for (int i = 0; i < boxes; ++i) tma_2d(x + i * 4096, &map_x, kb * 128, t.row0 + 32 * i, &full[s]);
          }
          ++issued;
          if (++s == C::STAGES) {
            s = 0;
            ph ^= 1;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (lane == 0) {
        // Every stage's last phase: normally its release by all MMAs, after
        // which nothing is under way to this CTA; after a wait that ran out,
        // the arrival of the copies.
        const uint32_t n = issued < (uint32_t)C::STAGES ? issued : (uint32_t)C::STAGES;
        for (uint32_t q = issued - n; q < issued; ++q) {
          if (ok) ok = wait(&empty[q % C::STAGES], (q / C::STAGES) & 1);
          else (void)mbar_wait(&full[q % C::STAGES], (q / C::STAGES) & 1);
        }
      }
    } else if (warp == 9) {
      // ---------------- MMA issuer.  The whole warp runs the loop, so that the
      // descriptors are warp-uniform values: 40 cycles an MMA, 70 from one lane's
      // loop.
      uint32_t g = 0;  // K blocks so far
      bool ok = true;
      const uint64_t dw0 = tc05::sw128_desc(smem_u32(sm)), dx0 = tc05::sw128_desc(smem_u32(sm) + C::W_BYTES);
      for (int u = u0; u < n_units && ok; u += ustep) {
        const TcUnit t = unit_of(u);
        const uint32_t idesc = tc05::idesc_e4m3(128, t.n);
        for (int kb = kb_from; kb < kb_to; ++kb, ++g) {
          const uint32_t s = g % C::STAGES, ph = (g / C::STAGES) & 1;
          const uint32_t b = g % C::NBUF, bph = ((g / C::NBUF) & 1) ^ 1;
          // every lane looks and waits, and all go on or none
          const bool ready = mbar_test(&full[s], ph) & mbar_test(&tempty[b], bph);
          if (!__all_sync(0xffffffffu, ready)) {
            ok = wait(&full[s], ph) && wait(&tempty[b], bph);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          tc05::fence_after_sync();
          const uint64_t dw = dw0 + (uint64_t)(s * (C::STAGE >> 4)), dx = dx0 + (uint64_t)(s * (C::STAGE >> 4));
          const uint32_t d = tmem + b * C::ACC;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (TALL) tc05::mma_e4m3(d, dx + 2 * k, dw + 2 * k, idesc, k > 0 ? 1u : 0u);
            else tc05::mma_e4m3(d, dw + 2 * k, dx + 2 * k, idesc, k > 0 ? 1u : 0u);
          }
          tc05::commit(&tfull[b]);
          tc05::commit(&empty[s]);
        }
      }
      if (!ok) {  // what has been issued retires before tensor memory goes
        const long long t0 = clock64();
        while (clock64() - t0 < 2000000) {
        }
      }
    } else if (warp == 10) {
      // ---------------- scales
      uint32_t s = 0, ph = 0;
      float* ring = reinterpret_cast<float*>(sm + C::OFF_SCALE);
      bool ok = true;
      auto copy4 = [](float* dst, const float* src) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
      };
      auto filled = [&]() {  // arrives when this lane's copies have landed
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sfull[s])) : "memory");
        if (++s == C::SLOTS) {
          s = 0;
          ph ^= 1;
        }
      };
      for (int u = u0; u < n_units && ok; u += ustep) {
        const TcUnit t = unit_of(u);
        if (TALL) {
          const float* sb = p.sb + ((size_t)t.e * p.nb + min(t.wt * 2 + (lane & 1), p.nb - 1)) * p.kb;
          const int last = t.cnt - 1;
          for (int kb = 0; kb < p.kb; kb += 4) {
            if (!wait(&sempty[s], ph ^ 1)) {
              ok = false;
              break;
            }
            float* slot = ring + s * C::SLOT_FLOATS;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (kb + j < p.kb) {
                const float* sa = p.sa + (size_t)(kb + j) * p.M + t.row0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  copy4(slot + j * 128 + i * 32 + lane, sa + min(i * 32 + lane, last));
                if (lane < 2) copy4(slot + 512 + j * 2 + lane, sb + kb + j);
              }
            }
            filled();
          }
          continue;
        }
        const int nh = t.n >> 1;
        const float* sb = p.sb + ((size_t)t.e * p.nb + t.wt) * p.kb;
        for (int kb = kb_from; kb < kb_to; ++kb) {
          if (!wait(&sempty[s], ph ^ 1)) {
            ok = false;
            break;
          }
          float* slot = ring + s * C::SLOT_FLOATS;
          const float* sa = p.sa + (size_t)kb * p.M + t.row0;
#pragma unroll
          for (int i = 0; i < C::ACC / 32; ++i) {
            const int c = lane + 32 * i;
            if (c < t.n) {
              // thread q of a promotion quad reads its pairs of the 4 neighbouring 8-column groups together
              const int h = c >= nh ? 1 : 0, cc = c - h * nh;
              const int at = h * (C::ACC / 2) + ((cc & 7) >> 1) * 8 + (cc >> 3) * 2 + (cc & 1);
              copy4(slot + at, sa + min(c, t.cnt - 1));
            }
          }
          if (lane == 0) copy4(slot + C::ACC, sb + kb);
          filled();
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    if (TALL) tc05::regs_up<TC_REGS_HIGH>();
    // ---------------- promotion: acc += scale * block, then the output
    const int quad = warp & 3, half = warp >> 2;
    uint8_t* out = sm + C::OFF_OUT + warp * C::OUT_WARP;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    uint32_t v = 0;  // accumulators so far
    uint32_t s = 0, sph = 0;
    const float* ring = reinterpret_cast<const float*>(sm + C::OFF_SCALE);
    bool ok = true;
    // The accumulator is in registers: back to the MMAs.
    auto give_back = [&](uint32_t b) {
      tc05::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[b]);
    };
    if constexpr (TALL) {
      for (int u = u0; u < n_units && ok; u += ustep) {
        const TcUnit t = unit_of(u);
        const int row = quad * 32;                   // first of the warp's 32 rows in the tile
        const int live = t.n > 128 * half ? min(32, t.cnt - row) : 0;  // its rows of a, <= 0: none
        uint64_t acc[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) acc[i] = 0ull;
        auto promote = [&](const float* sa, const float* sb) -> bool {  // one K block
          const float sc = sa[quad * 32 + lane] * sb[half];
          const uint32_t b = v % C::NBUF, bph = (v / C::NBUF) & 1;
          ++v;
          if (!wait(&tfull[b], bph)) return false;
          tc05::fence_after_sync();
          if (live > 0) {
            const uint32_t ta = lanes + b * C::ACC + half * 128;
            uint32_t r[2][16];
            tc05::ld_32x32b_x16(ta, r[0]);
            const uint64_t s2 = f2pack(sc, sc);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              tc05::wait_ld16(r[c & 1]);
              if (c < 7) tc05::ld_32x32b_x16(ta + 16 * (c + 1), r[(c + 1) & 1]);
              else give_back(b);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                acc[8 * c + i] = fma2(pack2(r[c & 1][2 * i], r[c & 1][2 * i + 1]), s2, acc[8 * c + i]);
            }
          } else {
            give_back(b);
          }
          return true;
        };
        for (int kb = 0; kb < p.kb && ok; kb += 4) {
          ok = wait(&sfull[s], sph);
          const float* slot = ring + s * C::SLOT_FLOATS;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (ok && kb + j < p.kb) ok = promote(slot + 128 * j, slot + 512 + 2 * j);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sempty[s]);  // every lane has used its scales
          if (++s == C::SLOTS) {
            s = 0;
            sph ^= 1;
          }
        }
        if (!ok) break;
        // Output: 128-byte pieces of 32 rows in the 128-byte swizzle, copied out by
        // TMA while the next unit is multiplied.  Where a row behind the group's
        // last belongs to another group, the warp stores its rows itself.
        constexpr int SIZE = F32 ? 4 : 2, COLS = 128 / SIZE;  // columns of a piece
        const int n0 = t.wt * 256 + half * 128, row0 = t.row0 + row;
        const bool box = live == 32 || t.row0 + t.cnt == p.M;  // TMA leaves out what lies outside y
#pragma unroll
        for (int r = 0; r < (F32 ? 2 : 1); ++r) {  // two pieces a round: 8 KB
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint64_t* src = acc + (2 * r + c) * (COLS / 2) + j * (F32 ? 2 : 4);
              uint4 v;
              if (F32) {
                const ulonglong2 q = make_ulonglong2(src[0], src[1]);
                v = *reinterpret_cast<const uint4*>(&q);
              } else {
                v = make_uint4(bf16_pair(src[0]), bf16_pair(src[1]), bf16_pair(src[2]), bf16_pair(src[3]));
              }
              *reinterpret_cast<uint4*>(out + c * 4096 + lane * 128 + ((j ^ (lane & 7)) << 4)) = v;
            }
          tc05::fence_proxy_async_smem();
          __syncwarp();
          const int nr = n0 + r * 2 * COLS;  // first column of the round
          if (box) {
            if (lane == 0 && live > 0) {
#pragma unroll
              for (int c = 0; c < 2; ++c)
                if (nr + c * COLS < p.N)
                  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                                   &map_y),
                               "r"(nr + c * COLS), "r"(row0), "r"(smem_u32(out + c * 4096))
                               : "memory");
            }
          } else {
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {  // two rows at a time, 16 lanes each
              const int rr = 2 * i + (lane >> 4), c = (lane >> 3) & 1, j = lane & 7;
              const int n = nr + c * COLS + j * (16 / SIZE);
              if (rr < live && n < p.N)
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.y) + ((size_t)(row0 + rr) * p.N + n) * SIZE) =
                    *reinterpret_cast<const uint4*>(out + c * 4096 + rr * 128 + ((j ^ (rr & 7)) << 4));
            }
          }
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
      }
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    } else {
      const int q = lane & 3;
      for (int u = u0; u < n_units && ok; u += ustep) {
        const TcUnit t = unit_of(u);
        const int nh = t.n >> 1;
        uint64_t acc[2][8];  // [lane half][4 groups x (row g, row g + 8)]
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[0][i] = acc[1][i] = 0ull;
        for (int kb = kb_from; kb < kb_to; ++kb) {
          const uint32_t b = v % C::NBUF, bph = (v / C::NBUF) & 1;
          ++v;
          if (!wait(&sfull[s], sph) || !wait(&tfull[b], bph)) {
            ok = false;
            break;
          }
          tc05::fence_after_sync();
          const float* slot = ring + s * C::SLOT_FLOATS;
          const uint32_t ta = lanes + b * C::ACC + (uint32_t)(half * nh);
          uint32_t r[32];
          tc05::ld_16x256b_x4(ta, r);
          tc05::ld_16x256b_x4(ta + (16u << 16), r + 16);
          const float wsc = slot[C::ACC];
          const uint64_t w2 = f2pack(wsc, wsc);
          const float4* sc = reinterpret_cast<const float4*>(slot + half * (C::ACC / 2) + q * 8);
          const float4 s0 = sc[0], s1 = sc[1];
          const uint64_t s2[4] = {f2mul(f2pack(s0.x, s0.y), w2), f2mul(f2pack(s0.z, s0.w), w2),
                                  f2mul(f2pack(s1.x, s1.y), w2), f2mul(f2pack(s1.z, s1.w), w2)};
          tc05::wait_ld32(r);
          give_back(b);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              acc[h][i] = fma2(pack2(r[16 * h + 2 * i], r[16 * h + 2 * i + 1]), s2[i >> 1], acc[h][i]);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sempty[s]);  // every lane has used its scales
          if (++s == C::SLOTS) {
            s = 0;
            sph ^= 1;
          }
        }
        if (!ok) break;
        if constexpr (KS > 1) {
          // The stages are free: every block of this CTA has landed and been multiplied.
          uint64_t* part = reinterpret_cast<uint64_t*>(sm) + tid;
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) part[(4 * k + j) * 256] = acc[j >> 1][2 * k + (j & 1)];
        } else {
          wide_output<F32>(p, t, acc, 0, 4, out, quad, half, lane);
        }
      }
    }
  }
  if constexpr (KS > 1) {
    // The partial sums, in the order of the CTAs; each CTA puts out 4 / KS of every
    // warp's four groups of 8 columns.
    __syncwarp();
    tc05::cluster_sync();
    if (warp < 8 && u0 < n_units) {
      const TcUnit t = unit_of(u0);
      constexpr int G = 4 / KS;
      uint64_t v[KS][4 * G], acc[2][8];
#pragma unroll
      for (int r = 0; r < KS; ++r) {
        uint32_t at;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(sm) + (split * 4 * G * 256 + tid) * 8), "r"(r));
#pragma unroll
        for (int j = 0; j < 4 * G; ++j)
          asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v[r][j]) : "r"(at + j * 2048) : "memory");
      }
      const uint64_t one = f2pack(1.f, 1.f);
#pragma unroll
      for (int r = 1; r < KS; ++r)
#pragma unroll
        for (int j = 0; j < 4 * G; ++j) v[0][j] = fma2(v[r][j], one, v[0][j]);
#pragma unroll
      for (int j = 0; j < 4 * G; ++j) acc[(j >> 1) & 1][2 * (j >> 2) + (j & 1)] = v[0][j];
      wide_output<F32>(p, t, acc, split * G, G, sm + C::OFF_OUT + warp * C::OUT_WARP, warp & 3, warp >> 2, lane);
    }
    tc05::cluster_sync();  // the other CTAs have read this one's
  }
  __syncwarp();
  tc05::fence_before_sync();
  __syncthreads();
  if (warp == 8) {
    tc05::fence_after_sync();
    tc05::tmem_dealloc(tmem, 512);
  }
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled g_encode = nullptr;  // set once, under the library's lock

// A map of rows of `cols` elements of `size` bytes, of one matrix (mats 0) or
// `mats` of them; boxes of 128 bytes x `box` rows in the 128-byte swizzle, zeros
// outside.
bool row_map(CUtensorMap* m, const void* base, int size, uint64_t cols, uint64_t rows, uint64_t mats, uint32_t box) {
  const cuuint64_t dims[3] = {cols, rows, mats}, strides[2] = {cols * size, cols * size * rows};
  const cuuint32_t boxes[3] = {128u / (uint32_t)size, box, 1}, steps[3] = {1, 1, 1};
  const CUtensorMapDataType type = size == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : size == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  return g_encode(m, type, mats ? 3 : 2, const_cast<void*>(base), dims, strides, boxes, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool TALL, bool F32, int KS = 1>
cudaError_t launch_tc(const GemmArgs& p, int sm_count, unsigned* err, cudaStream_t st) {
  using C = TcCfg<TALL>;
  TcArgs t;
  t.sa = p.sa;
  t.sb = p.sb;
  t.offsets = p.offsets;
  t.y = p.y;
  t.err = err;
  t.M = p.M;
  t.N = p.N;
  t.E = p.E;
  t.kb = p.kb;
  t.nb = p.nb;
  t.n_tiles = (p.N + C::WROWS - 1) / C::WROWS;
  t.n_tiles_recip = 0xFFFFFFFFu / (unsigned)t.n_tiles + 1u;
  CUtensorMap mw, mx, my;
  const int size = F32 ? 4 : 2;
  if (!row_map(&mw, p.b, 1, p.K, p.N, p.E, 128) || !row_map(&mx, p.a, 1, p.K, p.M, 0, C::X_BOX) ||
      !row_map(&my, p.y, size, p.N, p.M, 0, 32))
    return cudaErrorInvalidValue;
  const long long groups = p.M < p.E ? p.M : p.E;  // that can have rows
  const long long tiles = p.offsets == nullptr ? (p.M + C::ROWS - 1LL) / C::ROWS : (long long)p.M / C::ROWS + groups;
  const long long most = tiles * t.n_tiles;  // units, at most
  // With K split a cluster takes one unit and no more (its operands' memory holds the partial sums).
  const long long clusters = KS > 1 ? most : sm_count;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(KS * (most < clusters ? most : clusters)));
  cfg.blockDim = dim3(TC_THREADS);
  cfg.dynamicSmemBytes = C::smem(p.E);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = KS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, block_gemm_tc_kernel<TALL, F32, KS>, t, mw, mx, my);
}

}  // namespace

cudaError_t block_gemm_kernels_init() {
  if (g_encode == nullptr) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || fn == nullptr) return cudaErrorNotSupported;
    g_encode = reinterpret_cast<EncodeTiled>(fn);
  }
  const void* k[] = {reinterpret_cast<const void*>(block_gemm_tc_kernel<true, false, 1>),
                     reinterpret_cast<const void*>(block_gemm_tc_kernel<true, true, 1>),
                     reinterpret_cast<const void*>(block_gemm_tc_kernel<false, false, 1>),
                     reinterpret_cast<const void*>(block_gemm_tc_kernel<false, true, 1>),
                     reinterpret_cast<const void*>(block_gemm_tc_kernel<false, false, 2>),
                     reinterpret_cast<const void*>(block_gemm_tc_kernel<false, true, 2>),
                     reinterpret_cast<const void*>(block_gemm_tc_kernel<false, false, 4>),
                     reinterpret_cast<const void*>(block_gemm_tc_kernel<false, true, 4>)};
  for (int i = 0; i < 8; ++i) {
    const int bytes = i < 2 ? TcCfg<true>::smem(ROUTE_MAX_E) : TcCfg<false>::smem(ROUTE_MAX_E);
    cudaError_t e = cudaFuncSetAttribute(k[i], cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, k[i])) != cudaSuccess) return e;
    if (i < 2 && fa.numRegs < TC_REGS) return cudaErrorInvalidConfiguration;  // the shares would never be met
  }
  return cudaSuccess;
}

// Which kernel a product takes, measured (us, calls in a graph) on 256 experts of
// 1024 x 2048, R rows in all, and on one matrix of 4096 x 2048:
//   up to 8 grouped rows        few-row SPLIT 8  R 8: 6.2, WIDE 9.4
//   up to 8 dense rows, 28 M
//   weights                     few-row SPLIT 8  8 of 6144 x 4096: 6.2, WIDE in 2 9.0; but 8192 x 8192: 14.6, 13.4
//   more dense rows, passes of
//   8 x N up to 14,336, x K up
//   to 21 M                     few-row SPLIT 8  16 rows: 5.2, WIDE in 4 5.8; 40 of 2048 x 2048 5.8, 5.8; 192 of
//                                                512 x 512 3.5, 4.1; but 32 rows: 7.9, 5.8; 80 of 2048 x 1024 6.1, 5.2
//   33 to 128 rows, at most one
//   an expert on average        few-row SPLIT 1  R 48: 17.3, WIDE 19.1; R 128: 36.6, 34.5; but R 32: 16.5, 14.3
//   a seventh of the SMs spare
//   with 4 CTAs a unit, K from
//   8 blocks                    WIDE in 4        32 rows: 5.8, in 2 6.9, whole 7.6; 64 of 2048 x 8192: 10.3, 15.2, 24.6
//   2 CTAs a unit, 12 blocks    WIDE in 2        100 of 4096 x 4096: 10.4, whole 14.0
//   one wave of WIDE's units,
//   or 36 rows an expert        WIDE             24 rows each: 85.7, TALL 87.8; 256 dense: 9.0, 10.5
//   else                        TALL             48 rows each: 91.5, WIDE 102.7; 512 dense: 10.7, 14.9
enum GemmKernel { GEMM_FEW_SPLIT, GEMM_FEW, GEMM_WIDE_IN_4, GEMM_WIDE_IN_2, GEMM_WIDE, GEMM_TALL };
static GemmKernel choose_block_gemm(int M, int N, int K, int E, bool grouped, int sm_count) {
  constexpr int WIDE_ROWS = TcCfg<false>::ROWS, WIDE_W = TcCfg<false>::WROWS;
  const int kb = (K + 127) / 128;
  const long long groups = M < E ? M : E;  // that can have rows
  const long long wide_tiles = grouped ? M / WIDE_ROWS + groups : (M + WIDE_ROWS - 1) / WIDE_ROWS;
  const long long wide_units = wide_tiles * ((N + WIDE_W - 1) / WIDE_W);
  const long long passes = (M + 7) / 8;
  bool few;
  if (grouped) few = M <= 8;
  else if (passes == 1) few = (long long)N * K <= 28 << 20;
  else few = passes * N <= 14336 && passes * N * K <= 21 << 20;
  if (few) return GEMM_FEW_SPLIT;
  if (M > 32 && M <= 128 && M <= E) return GEMM_FEW;
  if (kb >= 8 && 4 * wide_units <= 7 * sm_count / 8) return GEMM_WIDE_IN_4;
  if (kb >= 12 && 2 * wide_units <= sm_count) return GEMM_WIDE_IN_2;
  if (M <= 36LL * E || wide_units <= sm_count) return GEMM_WIDE;
  return GEMM_TALL;
}

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
  switch (choose_block_gemm(M, N, K, E, offsets != nullptr, sm_count)) {
    case GEMM_FEW_SPLIT: return f32 ? launch_skinny<8, 8, true>(p, st) : launch_skinny<8, 8, false>(p, st);
    case GEMM_FEW: return f32 ? launch_skinny<1, 4, true>(p, st) : launch_skinny<1, 4, false>(p, st);
    case GEMM_WIDE_IN_4:
      return f32 ? launch_tc<false, true, 4>(p, sm_count, err, st) : launch_tc<false, false, 4>(p, sm_count, err, st);
    case GEMM_WIDE_IN_2:
      return f32 ? launch_tc<false, true, 2>(p, sm_count, err, st) : launch_tc<false, false, 2>(p, sm_count, err, st);
    case GEMM_WIDE:
      return f32 ? launch_tc<false, true>(p, sm_count, err, st) : launch_tc<false, false>(p, sm_count, err, st);
    case GEMM_TALL:
      return f32 ? launch_tc<true, true>(p, sm_count, err, st) : launch_tc<true, false>(p, sm_count, err, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace flint

// For the tests: which kernel a product takes on a GPU of so many SMs.
extern "C" int flint_block_gemm_kernel(int M, int N, int K, int n_experts, int grouped, int sm_count) {
  return flint::choose_block_gemm(M, N, K, n_experts, grouped != 0, sm_count);
}
