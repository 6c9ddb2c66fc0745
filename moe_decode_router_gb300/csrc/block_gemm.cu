// Matrix product of FP8 (E4M3) operands with block scales, dense or grouped by
// expert:
//   y[m][n] = sum over kb of sa[kb][m] * sb[e][n / 128][kb] *
//             sum over k in block kb of a[m][k] * b[e][n][k]
// Each 128-long partial sum is formed by the tensor cores in fp32, then scaled
// and added in fp32.
#include <cuda.h>

#include "flint_common.cuh"
#include "flint_internal.h"
#include "tc05.cuh"

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

// ---- many rows: tcgen05 over pairs of CTAs.
//
// The weights are the M side (256 weight rows per pair, 128 per CTA, always
// full) and the activation rows the N side, which takes any multiple of 32 up
// to NT: a ragged group of an expert wastes at most 31 columns.  The block
// scales allow the tensor cores 128 of K at a time: every K block is a fresh
// accumulator in tensor memory (NBUF of them in a ring), and eight warps per
// CTA read it back and add it, scaled, into fp32 registers while the next
// block is multiplied.
//
// Per SM and K block at NT = 256: 512 cycles of MMA, against 128 KB of tensor
// memory read and 16,384 packed fma for the promotion, about 256 cycles each,
// that overlap with it; 32 KB of operands from L2 (64 B per cycle).
//
// Tensor memory is read in 16x256b form: a thread holds 4 weight rows x pairs
// of neighbouring columns, so a pair of column scales, read once from shared
// memory, serves 4 packed fma.
//
// Warps: 0 TMA producer, 1 MMA issuer (even CTA), 2 scale loader, 3 tensor
// memory; 4-7 and 8-11 promotion and output, one column half each.
constexpr int TC_THREADS = 384;
constexpr int TC_A_BYTES = 128 * 128;
// Registers at NT = 256: the promotion warps hold 128 accumulators each and
// take what the other four warps give up.  Launched with 168 a thread.
constexpr int TC_REGS = 168, TC_REGS_LOW = 56, TC_REGS_HIGH = 216;
static_assert(TC_REGS_HIGH * 256 + TC_REGS_LOW * 128 <= TC_REGS * TC_THREADS, "register shares");

template <int NT>
struct TcCfg {
  static constexpr int NBUF = 512 / NT;
  static constexpr int B_BYTES = NT / 2 * 128;
  static constexpr int STAGE = TC_A_BYTES + B_BYTES;
  static constexpr int STAGES = NT == 256 ? 6 : 9;
  static constexpr int SLOTS = 4;                // scale ring
  static constexpr int SLOT_FLOATS = NT + 4;     // column scales, then the weight scale
  static constexpr int OUT_WARP = 16 * 80;       // 16 rows of y x 32 columns, 80-byte pitch
  static constexpr int OFF_OUT = STAGES * STAGE;
  static constexpr int OFF_SCALE = OFF_OUT + 8 * OUT_WARP;
  static constexpr int OFF_BARS = OFF_SCALE + SLOTS * SLOT_FLOATS * 4;
  static constexpr int OFF_GROUPS = OFF_BARS + 512;
  static constexpr int smem(int E) { return OFF_GROUPS + (3 * E + 1) * 4; }
  static_assert(OFF_GROUPS + (3 * 1024 + 1) * 4 <= 232448, "shared memory");
};

struct TcArgs {
  const float* sa;
  const float* sb;
  const int32_t* offsets;
  void* y;
  unsigned* err;
  int M, N, E, kb, nb, n_tiles;  // n_tiles: weight tiles of 256 rows
};

struct TcUnit {
  int e, wt, row0, cnt, n;  // n: columns of the MMA
};

__device__ __forceinline__ void tma_pair_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_pair_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
      "%3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
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

template <int NT, bool F32>
__global__ void __launch_bounds__(TC_THREADS, 1)
    block_gemm_tc_kernel(const TcArgs p, const __grid_constant__ CUtensorMap map_w,
                         const __grid_constant__ CUtensorMap map_x) {
  using C = TcCfg<NT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = tc05::cluster_rank();
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::OFF_BARS);  // [STAGES] both CTAs' operands landed (even CTA's)
  uint64_t* empty = full + C::STAGES;                              // [STAGES] stage consumed
  uint64_t* tfull = empty + C::STAGES;                             // [NBUF] accumulator complete
  uint64_t* tempty = tfull + C::NBUF;                              // [NBUF] accumulator read, 16 warps (even CTA's)
  uint64_t* sfull = tempty + C::NBUF;                              // [SLOTS] scales landed
  uint64_t* sempty = sfull + C::SLOTS;                             // [SLOTS] scales read, 8 warps
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sempty + C::SLOTS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  static_assert((2 * C::STAGES + 2 * C::NBUF + 2 * C::SLOTS) * 8 + 8 <= 512, "barriers");
  int* g_tiles = reinterpret_cast<int*>(sm + C::OFF_GROUPS);  // [E + 1] column tiles before each group
  int* g_lo = g_tiles + p.E + 1;                              // [E] first row
  int* g_cnt = g_lo + p.E;                                    // [E] rows

  if (warp == 3) {
    tc05::tmem_alloc_pair(tslot, 512);
    tc05::tmem_relinquish_pair();
  }
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::NBUF; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 16);
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
  if (warp == 2) {  // groups: rows, and column tiles before each
    int base = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int lo = 0, cnt = 0;
      if (e < p.E) {
        lo = p.offsets ? min(max(__ldg(p.offsets + e), 0), p.M) : 0;
        cnt = p.offsets ? min(max(__ldg(p.offsets + e + 1), lo), p.M) - lo : p.M;
        g_lo[e] = lo;
        g_cnt[e] = cnt;
      }
      const int t = (cnt + NT - 1) / NT;
      int incl = t;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
      }
      if (e < p.E) g_tiles[e] = base + incl - t;
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) g_tiles[p.E] = base;
  }
  tc05::fence_before_sync();
  __syncthreads();
  tc05::cluster_sync();  // both CTAs' barriers are ready
  tc05::fence_after_sync();
  const uint32_t tmem = *tslot;
  const int n_units = g_tiles[p.E] * p.n_tiles;
  const int u0 = blockIdx.x >> 1, ustep = gridDim.x >> 1;

  auto unit_of = [&](int u) -> TcUnit {
    TcUnit t;
    const int tile = u / p.n_tiles;
    t.wt = u - tile * p.n_tiles;
    int lo = 0, hi = p.E;  // largest e with g_tiles[e] <= tile: the group that holds the tile
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (g_tiles[mid] <= tile) lo = mid;
      else hi = mid;
    }
    t.e = lo;
    const int tiles = g_tiles[lo + 1] - g_tiles[lo], cnt = g_cnt[lo];
    const int size = ((cnt + tiles - 1) / tiles + 31) & ~31;  // a group's tiles are of one size, to 32 rows
    const int at = (tile - g_tiles[lo]) * size;
    t.row0 = g_lo[lo] + at;
    t.cnt = max(0, min(size, cnt - at));
    t.n = max(32, (t.cnt + 31) & ~31);
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

  if (warp < 4) {
    if (NT == 256) tc05::regs_down<TC_REGS_LOW>();
    if (warp == 0) {
      // ---------------- producer: this CTA's 128 weight rows and its half of the columns
      if (lane == 0) {
        uint32_t s = 0, ph = 0, issued = 0;
        bool ok = true;
        const uint32_t base = smem_u32(sm), full0 = tc05::map_rank(smem_u32(full), 0);
        for (int u = u0; u < n_units && ok; u += ustep) {
          const TcUnit t = unit_of(u);
          const int nh = t.n >> 1, boxes = (nh + 31) >> 5;
          const int wrow = t.wt * 256 + (int)rank * 128, xrow = t.row0 + (int)rank * nh;
          const uint32_t bytes = 2u * (TC_A_BYTES + boxes * 4096);
          for (int kb = 0; kb < p.kb; ++kb) {
            if (!wait(&empty[s], ph ^ 1)) {
              ok = false;
              break;
            }
            if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
            const uint32_t dst = base + s * C::STAGE, bar = full0 + s * 8;
            tma_pair_3d(dst, &map_w, kb * 128, wrow, t.e, bar);
            for (int i = 0; i < boxes; ++i) tma_pair_2d(dst + TC_A_BYTES + i * 4096, &map_x, kb * 128, xrow + 32 * i, bar);
            ++issued;
            if (++s == C::STAGES) {
              s = 0;
              ph ^= 1;
            }
          }
        }
        // Every stage's last phase: normally its release by the MMAs (nothing of
        // the peer is then under way to this CTA); after a wait that ran out, the
        // arrival of the copies.
        const uint32_t n = issued < (uint32_t)C::STAGES ? issued : (uint32_t)C::STAGES;
        for (uint32_t q = issued - n; q < issued; ++q) {
          if (ok) {
            ok = wait(&empty[q % C::STAGES], (q / C::STAGES) & 1);
          } else if (rank == 0) {
            (void)mbar_wait(&full[q % C::STAGES], (q / C::STAGES) & 1);
          }
        }
        if (!ok && rank != 0) {  // the peer's barriers cannot be waited on: 1 ms covers any copy
          const long long t0 = clock64();
          while (clock64() - t0 < 2000000) {
          }
        }
      }
    } else if (warp == 1) {
      // ---------------- MMA issuer
      if (rank == 0 && lane == 0) {
        uint32_t s = 0, ph = 0, b = 0, bph = 0, steps = 0;
        bool ok = true;
        const uint64_t da0 = tc05::sw128_desc(smem_u32(sm)), db0 = tc05::sw128_desc(smem_u32(sm) + TC_A_BYTES);
        for (int u = u0; u < n_units && ok; u += ustep) {
          const TcUnit t = unit_of(u);
          const uint32_t idesc = tc05::idesc_e4m3(256, t.n);
          for (int kb = 0; kb < p.kb; ++kb) {
            if (!wait(&tempty[b], bph ^ 1) || !wait(&full[s], ph)) {
              ok = false;
              break;
            }
            tc05::fence_after_sync();
            const uint64_t da = da0 + (uint64_t)(s * (C::STAGE >> 4)), db = db0 + (uint64_t)(s * (C::STAGE >> 4));
            const uint32_t d = tmem + b * NT;
#pragma unroll
            for (int k = 0; k < 4; ++k) tc05::mma_e4m3_pair(d, da + 2 * k, db + 2 * k, idesc, k > 0 ? 1u : 0u);
            tc05::commit_pair(&empty[s]);
            tc05::commit_pair(&tfull[b]);
            ++steps;
            if (++s == C::STAGES) {
              s = 0;
              ph ^= 1;
            }
            if (++b == C::NBUF) {
              b = 0;
              bph ^= 1;
            }
          }
        }
        if (steps > 0) {  // the last MMAs have retired
          const uint32_t q = steps - 1;
          (void)mbar_wait(&empty[q % C::STAGES], (q / C::STAGES) & 1);
        }
      }
    } else if (warp == 2) {
      // ---------------- scales of each K block: one per column, and the weights' one
      uint32_t s = 0, ph = 0;
      float* ring = reinterpret_cast<float*>(sm + C::OFF_SCALE);
      bool ok = true;
      for (int u = u0; u < n_units && ok; u += ustep) {
        const TcUnit t = unit_of(u);
        const int nh = t.n >> 1;
        const int wblock = min(t.wt * 2 + (int)rank, p.nb - 1);
        const float* sb = p.sb + ((size_t)t.e * p.nb + wblock) * p.kb;
        for (int kb = 0; kb < p.kb; ++kb) {
          if (!wait(&sempty[s], ph ^ 1)) {
            ok = false;
            break;
          }
          float* slot = ring + s * C::SLOT_FLOATS;
          const float* sa = p.sa + (size_t)kb * p.M + t.row0;
#pragma unroll
          for (int i = 0; i < NT / 32; ++i) {
            const int c = lane + 32 * i;
            if (c < t.n) {
              // thread q of a promotion quad reads its pairs of 4 neighbouring 8-column groups together
              const int h = c >= nh ? 1 : 0, cc = c - h * nh;
              const int at = h * (NT / 2) + (cc & ~31) + ((cc & 7) >> 1) * 8 + ((cc >> 3) & 3) * 2 + (cc & 1);
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(slot + at)),
                           "l"(sa + min(c, t.cnt - 1))
                           : "memory");
            }
          }
          if (lane == 0)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(slot + NT)), "l"(sb + kb) : "memory");
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sfull[s])) : "memory");
          if (++s == C::SLOTS) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    if (NT == 256) tc05::regs_up<TC_REGS_HIGH>();
    // ---------------- promotion: acc += scale * block, then the output
    const int quad = warp & 3, half = warp >= 8 ? 1 : 0;
    const int g = lane >> 2, q = lane & 3;
    constexpr int CH = NT / 64;  // 32-column chunks of a half
    uint32_t b = 0, bph = 0, s = 0, sph = 0;
    const float* ring = reinterpret_cast<const float*>(sm + C::OFF_SCALE);
    uint8_t* out = sm + C::OFF_OUT + (warp - 4) * C::OUT_WARP;
    const uint32_t tempty0 = tc05::map_rank(smem_u32(tempty), 0);
    bool ok = true;
    for (int u = u0; u < n_units && ok; u += ustep) {
      const TcUnit t = unit_of(u);
      const int nh = t.n >> 1;
      uint64_t acc[CH][2][8];  // [chunk][lane half][4 groups x (row g, row g + 8)]
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[c][0][i] = acc[c][1][i] = 0ull;
      for (int kb = 0; kb < p.kb; ++kb) {
        if (!wait(&sfull[s], sph) || !wait(&tfull[b], bph)) {
          ok = false;
          break;
        }
        tc05::fence_after_sync();
        const float* slot = ring + s * C::SLOT_FLOATS;
        const float wsc = slot[NT];
        const uint64_t w2 = f2pack(wsc, wsc);
        const uint32_t ta = tmem + ((uint32_t)(quad * 32) << 16) + b * NT + (uint32_t)(half * nh);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if (32 * c < nh) {
            uint32_t r[32];
            tc05::ld_16x256b_x4(ta + 32 * c, r);
            tc05::ld_16x256b_x4(ta + (16u << 16) + 32 * c, r + 16);
            const float4* sc = reinterpret_cast<const float4*>(slot + half * (NT / 2) + 32 * c + q * 8);
            const float4 s0 = sc[0], s1 = sc[1];
            const uint64_t s2[4] = {f2mul(f2pack(s0.x, s0.y), w2), f2mul(f2pack(s0.z, s0.w), w2),
                                    f2mul(f2pack(s1.x, s1.y), w2), f2mul(f2pack(s1.z, s1.w), w2)};
            tc05::wait_ld32(r);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 8; ++i)
                acc[c][h][i] = fma2(pack2(r[16 * h + 2 * i], r[16 * h + 2 * i + 1]), s2[i >> 1], acc[c][h][i]);
          }
        }
        tc05::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          tc05::mbar_arrive_cluster(tempty0 + b * 8);
          mbar_arrive(&sempty[s]);
        }
        if (++b == C::NBUF) {
          b = 0;
          bph ^= 1;
        }
        if (++s == C::SLOTS) {
          s = 0;
          sph ^= 1;
        }
      }
      if (!ok) break;
      const int n0 = t.wt * 256 + (int)rank * 128 + quad * 32;  // first weight row of the warp
      if (F32) {
        float* y = static_cast<float*>(p.y);
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int cl = 32 * c + (i >> 1) * 8 + 2 * q, col = half * nh + cl;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float v0, v1;
              f2unpack(acc[c][h][i], v0, v1);
              const int n = n0 + 16 * h + (i & 1) * 8 + g;
              if (n < p.N && cl < nh) {
                if (col < t.cnt) y[(size_t)(t.row0 + col) * p.N + n] = v0;
                if (col + 1 < t.cnt) y[(size_t)(t.row0 + col + 1) * p.N + n] = v1;
              }
            }
          }
      } else {
        uint16_t* y = static_cast<uint16_t*>(p.y);
        const uint32_t st = smem_u32(out) + (lane & 7) * 80 + (lane >> 3) * 16;  // row lane % 8 of matrix lane / 8
        const uint4* ld = reinterpret_cast<const uint4*>(out + (lane >> 2) * 80 + (lane & 3) * 16);
        const int n = n0 + (lane & 3) * 8;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if (32 * c >= nh) break;
#pragma unroll
          for (int gp = 0; gp < 4; gp += 2) {  // 16 rows of y at a time
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t m[4];  // weight rows 0-7, 8-15, 16-23, 24-31 of the warp
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float v0, v1;
                f2unpack(acc[c][i >> 1][2 * (gp + k) + (i & 1)], v0, v1);
                const __nv_bfloat162 hv = __floats2bfloat162_rn(v0, v1);
                m[i] = *reinterpret_cast<const uint32_t*>(&hv);
              }
              asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(st + k * 640),
                           "r"(m[0]), "r"(m[1]), "r"(m[2]), "r"(m[3])
                           : "memory");
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int cl = 32 * c + (gp + k) * 8 + (lane >> 2), col = half * nh + cl;
              const uint4 v = ld[k * 40];
              if (cl < nh && col < t.cnt && n < p.N)
                *reinterpret_cast<uint4*>(y + (size_t)(t.row0 + col) * p.N + n) = v;
            }
            __syncwarp();
          }
        }
      }
    }
  }
  __syncwarp();
  tc05::fence_before_sync();
  __syncthreads();
  tc05::cluster_sync();  // no arrival or copy is under way to either CTA any more
  if (warp == 3) {
    tc05::fence_after_sync();
    tc05::tmem_dealloc_pair(tmem, 512);
  }
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled g_encode = nullptr;  // set once, under the library's lock

// A map of byte rows of length K, boxes of 128 bytes x `box` rows in the
// 128-byte swizzle, zeros outside.
bool row_map(CUtensorMap* m, const void* base, int rank, uint64_t K, uint64_t rows, uint64_t mats, uint32_t box) {
  const cuuint64_t dims[3] = {K, rows, mats}, strides[2] = {K, K * rows};
  const cuuint32_t boxes[3] = {128, box, 1}, steps[3] = {1, 1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, boxes,
                  steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, bool F32>
cudaError_t launch_tc(const GemmArgs& p, int sm_count, unsigned* err, cudaStream_t st) {
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
  t.n_tiles = (p.N + 255) / 256;
  CUtensorMap mw, mx;
  if (!row_map(&mw, p.b, 3, p.K, p.N, p.E, 128) || !row_map(&mx, p.a, 2, p.K, p.M, 1, 32)) return cudaErrorInvalidValue;
  const long long most = ((long long)(p.M + NT - 1) / NT + p.E) * t.n_tiles;  // units, at most
  const int pairs = sm_count / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)(most < pairs ? most : pairs));
  cfg.blockDim = dim3(TC_THREADS);
  cfg.dynamicSmemBytes = TcCfg<NT>::smem(p.E);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, block_gemm_tc_kernel<NT, F32>, t, mw, mx);
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
  const void* k[4] = {reinterpret_cast<const void*>(block_gemm_tc_kernel<256, false>),
                      reinterpret_cast<const void*>(block_gemm_tc_kernel<256, true>),
                      reinterpret_cast<const void*>(block_gemm_tc_kernel<64, false>),
                      reinterpret_cast<const void*>(block_gemm_tc_kernel<64, true>)};
  for (int i = 0; i < 4; ++i) {
    const int bytes = i < 2 ? TcCfg<256>::smem(ROUTE_MAX_E) : TcCfg<64>::smem(ROUTE_MAX_E);
    cudaError_t e = cudaFuncSetAttribute(k[i], cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, k[i])) != cudaSuccess) return e;
    if (i < 2 && fa.numRegs < TC_REGS) return cudaErrorInvalidConfiguration;  // the shares would never be met
  }
  return cudaSuccess;
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
  if (M > (offsets != nullptr ? 64 : 8)) {
    if ((long long)M <= 64LL * E) return f32 ? launch_tc<64, true>(p, sm_count, err, st) : launch_tc<64, false>(p, sm_count, err, st);
    return f32 ? launch_tc<256, true>(p, sm_count, err, st) : launch_tc<256, false>(p, sm_count, err, st);
  }
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
