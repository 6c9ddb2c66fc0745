// Products on the tensor cores (tcgen05 over pairs of CTAs), dense or grouped by expert:
// linear and gated products in bf16 and their gradients, and 8-bit integer products.
//
// Three products in one kernel (both gradients in one launch, the weights' behind).  The M
// side of the MMA is the dimension that lies contiguous in the output (i), always 256 of it a
// unit; the N side (o), up to 256 in steps of 32, is what is ragged:
//   forward  y[m][n]     i = n: weights by rows       o = m: rows of x       sum over k
//   input    dx[m][k]    i = k: weights by columns    o = m: rows of dy      sum over n
//   weights  dw[e][n][k] i = k: columns of x          o = n: columns of dy   sum over the rows m of e
// An operand whose M or N dimension is contiguous in memory is taken as it lies (the
// descriptors' other major order), so nothing is transposed on the way in; on the way out
// the accumulator (lanes i, columns o) is turned by stmatrix into rows of the output.
//
// A gated unit has 8 strips of 16 gate rows and the 16 rows of the other factor that
// belong to them, so that a warp's 32 lanes hold both and the thread that reads a gate's
// sum reads its partner's.
//
// Each CTA loads its 128 rows of A and half of B, 64 of the contracted dimension at a time
// (128 bytes, 128-byte swizzle): 32 KB a stage and CTA against 512 cycles of MMA, 64 bytes
// a cycle and SM; a CTA by itself would load 96.  A stage is two copies, as large as they may be: with
// boxes of 32 rows of B (five copies a stage) 8192 x 8192 x 8192 took 693 us, with 128 574.  The accumulator is double-buffered in
// tensor memory, so that a unit's output overlaps the next one's products.
//
// The weights' gradient contracts over an expert's rows, which end anywhere: whole steps of 16 rows are
// multiplied, and in the last a warp of each CTA overwrites the rows behind the end (another
// expert's, perhaps infinite) with zeros before the stage is handed on.
//
// 8-bit integers.  This GPU's tensor cores take none at a rate worth using, but a code is
// exact in fp16, a product of two in fp32, and a sum of 896 products stays below 2^24 - 2^21
// (up to 2^24 fp32 holds every whole number).  Codes land in a ring of their own (128 of K a
// stage); eight warps turn them into fp16 (code + 1152 is put together from the bits,
// 1152 taken off), the weights' into tensor memory and the others into shared memory, whose
// bandwidth would be the bound with both: 96 KB for 64 of K, 768 cycles against 512 of MMA.
// Every 896 of K the accumulator (one alone, beside the weights: no MMA runs meanwhile) is added to
// sums in registers: in fp32 while they are at most 2^21, and once one of a warp's has passed that in
// 32-bit integers, whose conversions (16 lanes a cycle) are most of the time of the hand-over: 8191 x
// 4096 x 4096 takes 173 us, 194 with integers from the start (replays of a graph on a cool board; in a
// row of calls 190).  Registers are short where 128 sums a thread are held: the integer kernels spill 24
// to 92 bytes a thread, the fp32 ones up to 24.
//
// fp32 outputs of bf16 operands are promoted the same way every 512 of the contracted dimension: the
// tensor cores cut a sum instead of rounding it, which adds up (n products of one sign lose some n 2^-27
// of their sum: 2^17 a quarter of bf16's rounding, 2^22 2.3 %).  A weights' gradient of more than 2^17
// rows is promoted whatever its type.
//
// Where a dense product has units for few pairs alone, KS = 2 or 4 pairs of a cluster share a
// unit's contraction.  Each leaves its sums in its stages, and after a cluster barrier adds its
// part of the unit's columns over all of them, in the pairs' order: the result is the same on
// every call.
//
// Warps: output (the first 8 or 16, a quarter of the lanes and a part of the columns each); then the
// TMA producer; the MMA issuer (of the even CTA); rows behind the end; tensor memory;
// integers: four and four that turn codes to fp16.
#include <initializer_list>

#include "product_common.cuh"
#include "tc05_pair.cuh"

namespace flint {

namespace {

enum { FORWARD, BACKWARD };
enum { BF16, F32, BF16_ADDED };  // outputs (of gradients dw); the last two of bf16 operands are promoted

constexpr int A_BYTES = 128 * 128, B_BYTES = 128 * 128, STAGE = A_BYTES + B_BYTES;
constexpr int RING = 6;            // stages of operands
constexpr int CODES = 3;           // integers: stages of codes, 128 of K each, then
constexpr int TURNED = 3;          //   stages of one operand in fp16, and as many in tensor memory behind the sums
static_assert(CODES * STAGE + TURNED * 2 * B_BYTES <= RING * STAGE && 256 + TURNED * 64 <= 512, "rings");
constexpr int OUT_BYTES = 8 * 32 * 80;  // output staging: rows of 64 bytes, 80 apart, 32 a warp (16 of 16 warps)
constexpr int OFF_OUT = RING * STAGE;
constexpr int OFF_BARS = OFF_OUT + OUT_BYTES;
constexpr int SEG_F32 = 8, SEG_INT = 7;  // steps (of 64; integers: of 128) between promotions
constexpr int ALONE = 1 << 17;           // products that a bf16 output's accumulator takes without; N and K are no more

constexpr int OFF_GROUPS = OFF_BARS + 256;
constexpr int pair_smem(int E) { return OFF_GROUPS + (3 * E + 1) * 4; }
static_assert(pair_smem(ROUTE_MAX_E) <= 232448, "shared memory");
static_assert((3 * RING + CODES + 5) * 8 + 12 <= 256, "barriers");

// Warps and registers.  A kernel that adds up its accumulators has 8 output warps, which hold
// 128 sums a thread and take registers that the others give up (a block is launched with LAUNCH
// a thread); the others have 16, as a tile's way out is a chain of short steps: the weights'
// gradient of 256 experts (49,152 rows, 1024 x 2048) took 284 us with 8.
template <bool PROMOTE, bool INT8>
struct Shape {
  static constexpr int OUT_WARPS = PROMOTE ? 8 : 16, PARTS = OUT_WARPS / 4;  // parts of the columns
  static constexpr int CHUNK = PROMOTE ? 32 : 16;                            // columns on their way at a time
  static constexpr int THREADS = PROMOTE && !INT8 ? 384 : 640;
  static constexpr int LAUNCH = INT8 ? 96 : 168, HIGH = INT8 ? 168 : 224, LOW = 48;
  static_assert(!PROMOTE || HIGH * 256 + LOW * (THREADS - 256) <= LAUNCH * THREADS, "register shares");
};

struct PairArgs {
  const int32_t* offsets;
  void* y;          // forward: y; backward: dx, or null
  void* dw;         // backward: or null
  uint16_t* keep;   // gated: the sums, or null
  const float* sx;  // integers: scales
  const float* sw;
  unsigned* err;
  int M, E;
  int I;          // width of the outputs (i)
  int O;          // backward: N, rows of an expert's dw
  int steps;      // forward, input: steps of 64 of the contracted dimension (integers: of 128)
  int a_tiles;    // units side by side in i
  int tile;       // forward, input: o's of a unit, at most (a multiple of 32); grouped: 256
  int row_tiles;  // dense: units side by side in o
  int units;      // dense: of the forward product or dx
  int rows;       // dense: rows, and from bit 26 a tile's rows / 32
  int tile_w;     // weights: o's of a unit, at most
  int o_tiles;    // weights: units side by side in o, 0: not wanted
  unsigned per_band, per_expert;  // reciprocals of BAND * a_tiles and of o_tiles * a_tiles
  int act;
  bool pieces_k, pieces_n;  // K, N are multiples of 64: two pieces of 64 make one copy
};

// Tiles of o that go side by side, with all of i: what runs at a time shares both operands.
constexpr int BAND = 8;
// x / n for n up to BAND: (x + 1/2) / n is 1/16 at least from a whole number, and off by less than 2^-20 of itself.
__device__ __forceinline__ int small_quotient(int x, int n) { return (int)__fdividef((float)x + 0.5f, (float)n); }
static_assert(BAND <= 8 && BAND * ((1 << 17) / 256) < 1 << 14, "a band's units");
// x / n from n's reciprocal, 2^32 / n rounded up (0 for n = 1): too large by one at most.
__device__ __forceinline__ int quotient(int x, unsigned recip, int n) {
  if (n == 1) return x;
  const int q = (int)__umulhi((unsigned)x, recip);
  return q * n > x ? q - 1 : q;
}
unsigned reciprocal(int n) { return 0xFFFFFFFFu / (unsigned)n + 1u; }

// Boxes of operands in shared memory: rows of 128 bytes.
struct Maps {
  CUtensorMap a;     // forward: 128 rows of weights; input: 64 columns of 64 rows of weights (or 2 x 64 columns)
  CUtensorMap b[4];  // 16, 32, 64 or 128 rows of x (dy)
  CUtensorMap aw;    // weights: 64 columns of 64 rows of x (or 2 x 64)
  CUtensorMap bw;    // weights: 64 columns of 64 rows of dy
  CUtensorMap bw1;   // weights: the same as pieces of 64 columns
  CUtensorMap bw2;   // weights: 2 x 64
};

struct Unit {
  int e, at, o0, cnt, n;  // tile of i; first o and how many; columns of the MMAs
  bool weights;
  int c0, clen;           // weights: the expert's rows
};

// fp32 adds whole numbers exactly up to 2^24: a segment's sum to one of ROOM at most.
constexpr float ROOM = (float)((1 << 24) - SEG_INT * 128 * (1 << 14));
static_assert(SEG_INT * 128 * (1 << 14) < 1 << 24, "exact sums");
// Sums of a promoting kernel.
template <bool INT8>
struct Held {
  using type = float;
};
template <>
struct Held<true> {
  using type = int;
};

// 16 codes to 16 fp16 values: code + 1152 is 0x6400 with the code, its sign bit turned, in the low byte.
__device__ __forceinline__ void codes_to_f16(const uint4 c, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u, c.z ^ 0x80808080u, c.w ^ 0x80808080u};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __byte_perm(w[i >> 1], 0x64646464u, i & 1 ? 0x4342 : 0x4140);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&u), __float2half2_rn(1152.f));
    o[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

template <int MODE, bool GATED, int OUT, bool INT8, int KS>
__global__ void __launch_bounds__(Shape<OUT != BF16 || INT8, INT8>::THREADS, 1)
    pair_gemm_kernel(const PairArgs p, const __grid_constant__ Maps maps) {
  constexpr int STAGES = INT8 ? TURNED : RING, BUFS = INT8 ? 1 : 2;
  constexpr bool PROMOTE = OUT != BF16 || INT8;
  using W = Shape<PROMOTE, INT8>;
  constexpr int THREADS = W::THREADS, PRODUCER = W::OUT_WARPS, ISSUER = PRODUCER + 1, ZEROS = PRODUCER + 2,
                KEEPER = PRODUCER + 3;
  static_assert(!INT8 || MODE == FORWARD, "integers have no gradient");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // of the cluster's pairs this one's contraction; of the pair this CTA's half
  const uint32_t rank = tc05::cluster_rank() & 1u, lead = tc05::cluster_rank() & ~1u;
  const int split = KS > 1 ? (int)(tc05::cluster_rank() >> 1) : 0;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + OFF_BARS);  // [STAGES] both CTAs' operands landed (even CTA's)
  uint64_t* empty = full + STAGES;                              // [STAGES] stage consumed
  uint64_t* landed = empty + STAGES;                            // [STAGES] weights: a last stage of this CTA landed;
                                                                // [CODES] integers: codes of this CTA landed
  uint64_t* taken = landed + RING;                              // [CODES] integers: codes turned
  uint64_t* tfull = taken + CODES;                              // [2] accumulator complete
  uint64_t* tempty = tfull + 2;                                 // [2] accumulator read, by both CTAs' output warps (even CTA's)
  uint64_t* taken_mem = tempty + 2;                             // tensor memory taken, by both CTAs
  uint32_t* tslot = reinterpret_cast<uint32_t*>(taken_mem + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  volatile uint32_t* begun = tslot + 2;  // gradients: the unit that this CTA's producer has begun, + 1
  int* g_units = reinterpret_cast<int*>(sm + OFF_GROUPS);  // [E + 1] units before each group
  int* g_lo = g_units + p.E + 1;                           // [E] first row
  int* g_cnt = g_lo + p.E;                                 // [E] rows, and from bit 26 a tile's rows / 32

  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], INT8 ? 16 : MODE == BACKWARD ? 2 : 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < RING; ++i) mbar_init(&landed[i], 1);
    for (int i = 0; i < CODES; ++i) mbar_init(&taken[i], 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 2 * W::OUT_WARPS);
    }
    mbar_init(taken_mem, 2);
    *abort_flag = 0;
    *begun = 0;
    fence_mbar_init();
  }
  if (tid == 32) {  // the copies' descriptors, on their way while the grid before this one ends
    tc05::prefetch_map(&maps.a);
    for (int i = 0; i < 4; ++i) tc05::prefetch_map(&maps.b[i]);
    if (MODE == BACKWARD) {
      tc05::prefetch_map(&maps.aw);
      tc05::prefetch_map(&maps.bw);
      tc05::prefetch_map(&maps.bw1);
      tc05::prefetch_map(&maps.bw2);
    }
  }
  // The groups' units, by one warp.
  auto count_units = [&] {
    int base = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + lane;
      int lo = 0, cnt = 0;
      if (e < p.E) {
        lo = min(max(g_units[e], 0), p.M);
        cnt = min(max(g_units[e + 1], lo), p.M) - lo;
        // a group's tiles are of one size, to 32 rows
        const int tiles = (cnt + p.tile - 1) / p.tile;
        g_lo[e] = lo;
        g_cnt[e] = cnt | (cnt > 0 ? ((cnt + tiles - 1) / tiles + 31) >> 5 : 0) << 26;
      }
      __syncwarp();  // the offsets of these groups make room for their units; the next group's first is read below
      int t = MODE == BACKWARD && p.y == nullptr ? 0 : (cnt + p.tile - 1) / p.tile;
      t *= p.a_tiles;
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
  };
  if (p.offsets == nullptr && tid == 64) {
    g_units[0] = 0;
    g_units[1] = p.units;
    g_lo[0] = 0;
    g_cnt[0] = p.rows;
  }
  __syncthreads();
  tc05::cluster_sync();  // both CTAs' barriers are ready
  // A dense product's first copies are worked out before the wait.
  const bool early = p.offsets == nullptr && warp == PRODUCER;
  auto follow = [] {
    pdl_wait();
    pdl_trigger();
  };
  if (!early) follow();
  if (p.offsets != nullptr) {
    for (int e = tid; e <= p.E; e += THREADS) g_units[e] = __ldg(p.offsets + e);  // all on their way at once
    __syncthreads();
    if (warp == PRODUCER) count_units();
    __syncthreads();
  }
  const int n_rows_units = g_units[p.E];  // forward, input; behind them the weights'
  const int n_units = n_rows_units + (MODE == BACKWARD ? p.E * p.o_tiles * p.a_tiles : 0);
  // with the contraction shared one unit alone (its operands' memory takes the sums)
  const int u0 = blockIdx.x / (2 * KS), ustep = KS > 1 ? 1 << 30 : gridDim.x >> 1;

  // Few divisions: every role looks its units up, and a weights' unit may be three steps long.
  auto unit_of = [&](int u) -> Unit {
    Unit t;
    int v, tiles;
    t.weights = MODE == BACKWARD && u >= n_rows_units;
    t.e = 0;
    if (t.weights) {
      const int per = p.o_tiles * p.a_tiles;
      t.e = quotient(u - n_rows_units, p.per_expert, per);
      v = u - n_rows_units - t.e * per;
      tiles = p.o_tiles;
    } else {
      // The group is the last whose first unit is at or before u: the whole warp looks, at
      // every 32nd group and then at 32 neighbours.
      if (p.E > 1) {
        int from = 0;
        if (p.E > 32) from = 32 * (__popc(__ballot_sync(0xffffffffu, 32 * lane < p.E && g_units[32 * lane] <= u)) - 1);
        const int e = from + lane;
        t.e = from + __popc(__ballot_sync(0xffffffffu, e < p.E && g_units[e] <= u)) - 1;
      }
      v = u - g_units[t.e];
    }
    const int g = g_cnt[t.e], rows = g & ((1 << 26) - 1);
    if (!t.weights) tiles = p.offsets != nullptr ? (rows + 255) >> 8 : p.row_tiles;
    const int per = BAND * p.a_tiles, band = quotient(v, p.per_band, per), rest = v - band * per;
    const int high = min(BAND, tiles - band * BAND);
    t.at = small_quotient(rest, high);
    const int tile = band * BAND + rest - t.at * high;
    if (t.weights) {
      t.o0 = tile * p.tile_w;
      t.cnt = min(p.tile_w, p.O - t.o0);
      t.c0 = g_lo[t.e];
      t.clen = rows;
    } else {
      const int size = g >> 26 << 5;
      t.o0 = g_lo[t.e] + tile * size;
      t.cnt = max(0, min(size, rows - tile * size));
      t.c0 = t.clen = 0;
    }
    t.n = max(32, (t.cnt + 31) & ~31);
    return t;
  };
  // this pair's steps of a unit
  struct Steps {
    int from, to, all;
  };
  auto steps_of = [&](const Unit& t) {
    Steps s;
    s.all = t.weights ? (t.clen + 63) >> 6 : p.steps;
    const int share = (s.all + KS - 1) / KS;
    s.from = KS > 1 ? min(split * share, s.all) : 0;
    s.to = KS > 1 ? min(s.from + share, s.all) : s.all;
    return s;
  };
  // Bounded wait.  Lanes of a warp that wait together agree on the result: the awaited
  // phase cannot move on without a later arrival of this same warp.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (mbar_wait(bar, parity)) return true;
    atomicOr(p.err, ERR_WAIT_FULL);
    *abort_flag = 1;
    return false;
  };
  // the smallest box of B that holds so many rows: 16 << box_of
  auto box_of = [](int rows) { return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : 3; };
  // Tensor memory, when a warp of either CTA has taken it: the copies start meanwhile.
  auto tensor_memory = [&](bool& ok) -> uint32_t {
    ok = __all_sync(0xffffffffu, wait(taken_mem, 0));
    tc05::fence_after_sync();
    return *reinterpret_cast<volatile uint32_t*>(tslot);
  };
  const uint32_t base = smem_u32(sm), full0 = tc05::map_rank(smem_u32(full), lead);
  if (warp >= W::OUT_WARPS) {
    if (PROMOTE) tc05::regs_down<W::LOW>();
    if (INT8 && warp == PRODUCER) {
      // ---------------- producer of codes: stages of 128 of K
      uint32_t r = 0, ph = 0, issued = 0;
      bool ok = true;
      for (int u = u0; u < n_units && ok; u += ustep) {
        const Unit t = unit_of(u);
        const int nh = t.n >> 1, oh = t.o0 + (int)rank * nh, sel = box_of(nh);
        const uint32_t bytes = A_BYTES + (2048u << sel);
        const Steps steps = steps_of(t);
        if (early && u == u0) follow();
        for (int k = steps.from; k < steps.to && lane == 0; ++k) {
          if (!wait(&taken[r], ph ^ 1)) {
            ok = false;
            break;
          }
          const uint32_t a = base + r * STAGE, b = a + A_BYTES, bar = smem_u32(&landed[r]);
          mbar_arrive_expect_tx(&landed[r], bytes);
          if (GATED) tc05::tma_pair_5d(a, &maps.a, k * 128, 0, 0, t.at * 8 + (int)rank * 4, t.e, bar);
          else tc05::tma_pair_3d(a, &maps.a, k * 128, t.at * 256 + (int)rank * 128, t.e, bar);
          tc05::tma_pair_2d(b, &maps.b[sel], k * 128, oh, bar);
          ++issued;
          if (++r == CODES) {
            r = 0;
            ph ^= 1;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (lane == 0) {
        const uint32_t n = min(issued, (uint32_t)CODES);
        for (uint32_t q = issued - n; q < issued && ok; ++q) ok = wait(&taken[q % CODES], (q / CODES) & 1);
        if (!ok) {  // 1 ms covers any copy
          const long long t0 = clock64();
          while (clock64() - t0 < 2000000) {
          }
        }
      }
    } else if (INT8 && warp >= 12) {
      // ---------------- codes to fp16, 128 of K at a time: take(stage of codes, stage, unit) turns this
      // warp's part of them, done() makes what it wrote visible to the MMAs.
      auto turn = [&](auto&& take, auto&& done) {
        uint32_t s = 0, ph = 0, r = 0, rph = 0, turned = 0;
        bool ok = true;
        for (int u = u0; u < n_units && ok; u += ustep) {
          const Unit t = unit_of(u);
          const Steps steps = steps_of(t);
          for (int k = steps.from; k < steps.to; ++k) {
            // every lane looks, and all go on or none
            if (!__all_sync(0xffffffffu, mbar_test(&landed[r], rph) & mbar_test(&empty[s], ph ^ 1)))
              ok = __all_sync(0xffffffffu, wait(&landed[r], rph)) && __all_sync(0xffffffffu, wait(&empty[s], ph ^ 1));
            if (!ok) break;
            take(r, s, t);
            __syncwarp();
            if (lane == 0) mbar_arrive(&taken[r]);  // the codes are in registers or beyond
            done();
            __syncwarp();
            if (lane == 0) tc05::arrive_cluster(full0 + s * 8);
            if (++s == STAGES) {
              s = 0;
              ph ^= 1;
            }
            if (++r == CODES) {
              r = 0;
              rph ^= 1;
            }
            ++turned;
          }
        }
        // The last releases of the stages have arrived: no arrival is under way to this CTA when it ends.
        for (uint32_t q = turned - min(turned, (uint32_t)STAGES); q < turned && ok; ++q)
          ok = __all_sync(0xffffffffu, wait(&empty[q % STAGES], (q / STAGES) & 1));
      };
      if (warp < 16) {
        // The weights: a lane has a row, that of its lane of tensor memory (the swizzle puts 8
        // neighbouring rows' pieces in different places).
        const int arow = (warp & 3) * 32 + lane;
        bool had;
        const uint32_t to = tensor_memory(had) + 256 + ((uint32_t)((warp & 3) * 32) << 16);
        if (had) turn(
            [&](uint32_t r, uint32_t s, const Unit&) {
              tc05::fence_after_sync();
              const uint8_t* at = sm + r * STAGE + arow * 128;
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                uint4 c[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) c[h] = *reinterpret_cast<const uint4*>(at + (((4 * g + h) ^ (arow & 7)) << 4));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  uint4 v[4];
                  codes_to_f16(c[2 * h], v[0], v[1]);
                  codes_to_f16(c[2 * h + 1], v[2], v[3]);
                  tc05::st_32x32b_x16(to + s * 64 + (2 * g + h) * 16, v);
                }
              }
            },
            [&] {
              tc05::wait_st();
              tc05::fence_before_sync();
            });
      } else {
        // The other operand: a warp takes 8 rows (a swizzle atom) at once, a lane 16 codes of a row;
        // the 8 lanes that shared memory serves together have two rows r and r ^ 5, whose
        // swizzled places differ on the way in (bit 2) and on the way out (bit 0).
        const int q = lane & 3, row = (lane >> 3) ^ (lane & 4 ? 5 : 0), first = warp - 16;
        const int in = A_BYTES + row * 128 + first * 1024, near = (q ^ row) << 4;  // the second 64 of K: near ^ 64
        const int out = CODES * STAGE + row * 128 + first * 1024, lo = ((2 * q) ^ row) << 4;  // the upper half: lo ^ 16
        turn(
            [&](uint32_t r, uint32_t s, const Unit& t) {
              const int atoms = t.n >> 4;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint8_t* at = sm + r * STAGE + in + (near ^ (h * 64));
                uint8_t* to = sm + (2 * s + h) * B_BYTES + out;
                uint4 c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (first + 4 * i < atoms) c[i] = *reinterpret_cast<const uint4*>(at + i * 4096);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (first + 4 * i < atoms) {
                    uint4 v0, v1;
                    codes_to_f16(c[i], v0, v1);
                    *reinterpret_cast<uint4*>(to + i * 4096 + lo) = v0;
                    *reinterpret_cast<uint4*>(to + i * 4096 + (lo ^ 16)) = v1;
                  }
              }
            },
            [&] { tc05::fence_proxy_async_smem(); });
      }
    } else if (warp == PRODUCER) {
      // ---------------- producer: this CTA's 128 of i and its half of the columns
      uint32_t s = 0, ph = 0, issued = 0;  // of lane 0, which copies
      bool ok = true;
      for (int u = u0; u < n_units && ok; u += ustep) {
        const Unit t = unit_of(u);
        const int nh = t.n >> 1;
        const Steps steps = steps_of(t);
        const int i0 = t.at * 256 + (int)rank * 128, oh = t.o0 + (int)rank * nh;
        const int sel = box_of(nh), boxes = (nh + 63) >> 6;
        const bool both = p.pieces_n && nh == 128, one = p.pieces_n && nh == 64;  // weights: pieces of 64 columns of B
        const uint32_t bytes = A_BYTES + (t.weights ? (uint32_t)boxes * 8192u : 2048u << sel);
        if (MODE == BACKWARD && lane == 0) *begun = (uint32_t)u + 1;
        if (early && u == u0) follow();
        for (int k = steps.from; k < steps.to && lane == 0; ++k) {
          if (!wait(&empty[s], ph ^ 1)) {
            ok = false;
            break;
          }
          uint32_t bar = full0 + s * 8;
          const uint32_t a = base + s * STAGE, b = a + A_BYTES;
          if (MODE == FORWARD) {
            if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * bytes);
          } else if (t.weights && k == steps.all - 1 && (t.clen & 15)) {
            mbar_arrive_expect_tx(&landed[s], bytes);  // handed on by the warp that zeroes what lies behind the end
            bar = smem_u32(&landed[s]);
          } else {
            tc05::arrive_expect_cluster(bar, bytes);
          }
          if (MODE == FORWARD) {
            if (GATED) tc05::tma_pair_5d(a, &maps.a, k * 64, 0, 0, t.at * 8 + (int)rank * 4, t.e, bar);
            else tc05::tma_pair_3d(a, &maps.a, k * 64, i0, t.e, bar);
            tc05::tma_pair_2d(b, &maps.b[sel], k * 64, oh, bar);
          } else if (!t.weights) {
            if (p.pieces_k) {
              tc05::tma_pair_4d(a, &maps.a, 0, k * 64, i0 >> 6, t.e, bar);
            } else {
              tc05::tma_pair_3d(a, &maps.a, i0, k * 64, t.e, bar);
              tc05::tma_pair_3d(a + 8192, &maps.a, i0 + 64, k * 64, t.e, bar);
            }
            tc05::tma_pair_2d(b, &maps.b[sel], k * 64, oh, bar);
          } else {
            const int c = t.c0 + k * 64;
            if (p.pieces_k) {
              tc05::tma_pair_3d(a, &maps.aw, 0, c, i0 >> 6, bar);
            } else {
              tc05::tma_pair_2d(a, &maps.aw, i0, c, bar);
              tc05::tma_pair_2d(a + 8192, &maps.aw, i0 + 64, c, bar);
            }
            if (both || one) tc05::tma_pair_3d(b, both ? &maps.bw2 : &maps.bw1, 0, c, oh >> 6, bar);
            else
              for (int i = 0; i < boxes; ++i) tc05::tma_pair_2d(b + i * 8192, &maps.bw, oh + i * 64, c, bar);
          }
          ++issued;
          if (++s == STAGES) {
            s = 0;
            ph ^= 1;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (lane == 0) {
        // Every stage's last phase: normally its release by the MMAs (nothing of the peer
        // is then under way to this CTA); after a wait that ran out, time for the copies.
        const uint32_t n = issued < (uint32_t)STAGES ? issued : (uint32_t)STAGES;
        for (uint32_t q = issued - n; q < issued && ok; ++q) ok = wait(&empty[q % STAGES], (q / STAGES) & 1);
        if (!ok) {  // 1 ms covers any copy
          const long long t0 = clock64();
          while (clock64() - t0 < 2000000) {
          }
        }
      }
    } else if (warp == ISSUER) {
      // ---------------- MMA issuer.  The whole warp runs the loop, so that the descriptors
      // are warp-uniform values.
      if (rank == 0) {
        uint32_t s = 0, ph = 0, v = 0;
        bool ok;
        const uint32_t tmem = tensor_memory(ok);
        constexpr bool A_ROWS = MODE == BACKWARD;
        constexpr int SEG = INT8 ? SEG_INT : SEG_F32;
        constexpr uint32_t TFULL = (2 * STAGES + RING + CODES) * 8;
        const uint32_t bars[2] = {full0, tc05::map_rank(smem_u32(full), lead | 1u)};  // of either CTA
        const uint64_t da0 = A_ROWS ? tc05::sw128_rows_desc(base, 8192) : tc05::sw128_desc(base);
        const uint64_t db_k = tc05::sw128_desc(base + A_BYTES), db_w = tc05::sw128_rows_desc(base + A_BYTES, 8192);
        const uint64_t db8 = tc05::sw128_desc(base + CODES * STAGE);
        constexpr int DA = A_ROWS ? 128 : 2;  // 16 of the contracted dimension
        for (int u = u0; u < n_units && ok; u += ustep) {
          const Unit t = unit_of(u);
          const Steps steps = steps_of(t);
          const uint32_t idesc = tc05::idesc_f16(256, t.n, INT8 ? 0 : 1) | (A_ROWS ? tc05::A_ROWS_CONTIGUOUS : 0u) |
                                 (t.weights ? tc05::B_ROWS_CONTIGUOUS : 0u);
          const uint64_t db0 = t.weights ? db_w : db_k;
          const uint32_t DB = t.weights ? 128 : 2;
          for (int k = steps.from; k < steps.to; ++k) {
            const int at = k - steps.from;
            const bool fresh = PROMOTE ? at % SEG == 0 : at == 0;
            const bool last = k == steps.to - 1 || (PROMOTE && at % SEG == SEG - 1);
            const uint32_t b = v % BUFS, d = tmem + b * 256;
            // every lane waits, and all go on or none
            ok = !fresh || __all_sync(0xffffffffu, wait(&tempty[b], ((v / BUFS) & 1) ^ 1));
            if (ok && !__all_sync(0xffffffffu, mbar_test(&full[s], ph))) ok = __all_sync(0xffffffffu, wait(&full[s], ph));
            if (!ok) break;
            tc05::fence_after_sync();
            const uint64_t da = da0 + s * (STAGE >> 4), db = db0 + s * (STAGE >> 4);
            const int parts = t.weights && k == steps.all - 1 ? (((t.clen - 1) & 63) >> 4) + 1 : 4;
            const uint32_t more = fresh ? 0u : 1u, free0 = bars[0] + STAGES * 8 + s * 8, free1 = bars[1] + STAGES * 8 + s * 8;
            if (INT8) {
              tc05::mma_pair_ts(d, tmem + 256 + s * 64, db8 + 2 * s * (B_BYTES >> 4), idesc, more);
              tc05::mma_pair_ts(d, tmem + 256 + s * 64 + 32, db8 + (2 * s + 1) * (B_BYTES >> 4), idesc, 1);
              tc05::commit_pair(free0);
              tc05::commit_pair(free1);
            } else if (parts == 4) {
              tc05::mma_pair_step<DA>(d, da, db, DB, idesc, more, free0, free1);
            } else {
              for (int j = 0; j < parts; ++j) tc05::mma_pair(d, da + j * DA, db + j * DB, idesc, j > 0 ? 1u : more);
              tc05::commit_pair(free0);
              tc05::commit_pair(free1);
            }
            if (last) {
              for (int c = 0; c < 2; ++c) tc05::commit_pair(bars[c] + TFULL + b * 8);
              ++v;
            }
            if (++s == STAGES) {
              s = 0;
              ph ^= 1;
            }
          }
        }
        // The last accumulators are given back: no arrival is under way to this CTA when it ends.
        for (uint32_t j = v - min(v, (uint32_t)BUFS); j < v && ok; ++j)
          ok = __all_sync(0xffffffffu, wait(&tempty[j % BUFS], (j / BUFS) & 1));
        if (!ok) {  // what has been issued retires before tensor memory goes
          const long long t0 = clock64();
          while (clock64() - t0 < 2000000) {
          }
        }
      }
    } else if (warp == ZEROS) {
      // ---------------- weights: zeros for the rows of a last step that are not the expert's
      if (MODE == BACKWARD) {
        uint32_t g = 0, parity = 0;  // steps so far; of `landed`, a bit a stage
        bool ok = true;
        // The units before the one that is waited for (all of dx's among them) may take longer than a
        // wait's limit: it begins anew while the producer gets on to further units, one of which takes
        // less (2^24 rows some 0.15e9 cycles of 2e9).
        auto wait_behind = [&](uint64_t* bar, uint32_t phase) -> bool {
          uint32_t seen = *begun;
          while (!mbar_wait(bar, phase)) {
            const uint32_t now = *begun;
            if (*abort_flag) return false;
            if (now == seen) return wait(bar, phase);
            seen = now;
          }
          return true;
        };
        for (int u = u0; u < n_units && ok; u += ustep) {
          const Unit t = unit_of(u);
          const Steps steps = steps_of(t);
          g += steps.to - steps.from;
          if (!(t.clen & 15) || steps.from == steps.to || steps.to < steps.all) continue;  // clen: 0 of what are not weights
          const uint32_t s = (g - 1) % STAGES;
          ok = __all_sync(0xffffffffu, wait_behind(&landed[s], (parity >> s) & 1));
          if (!ok) break;
          parity ^= 1u << s;
          // a row of every piece of both operands: 8 lanes each
          const int from = t.clen & 63, to = (from + 15) & ~15, pieces = 2 + ((t.n / 2 + 63) >> 6);
          uint8_t* at = sm + s * STAGE + (lane >> 3) * 8192 + (lane & 7) * 16;
          if (lane < pieces * 8)
            for (int row = from; row < to; ++row) *reinterpret_cast<uint4*>(at + row * 128) = make_uint4(0, 0, 0, 0);
          tc05::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc05::arrive_cluster(full0 + s * 8);
        }
      }
    }
    if (warp == KEEPER) {
      // ---------------- tensor memory: taken when the grid before this one is gone and (below) given
      // back before either CTA of a pair ends, as taking it may wait without a limit for another's.
      tc05::alloc_pair(tslot, 512);
      tc05::relinquish_pair();
      tc05::fence_before_sync();
      __syncwarp();
      if (lane == 0)
        for (uint32_t c = 0; c < 2; ++c) tc05::arrive_cluster(tc05::map_rank(smem_u32(taken_mem), lead | c));
    }
    if constexpr (KS > 1) {  // the output warps' barrier
      __syncwarp();
      tc05::cluster_sync();
    }
  } else {
    if (PROMOTE) tc05::regs_up<W::HIGH>();
    // ---------------- output
    const int quad = warp & 3, part = warp >> 2;
    uint8_t* out = sm + OFF_OUT + warp * (OUT_BYTES / W::OUT_WARPS);
    bool ok;
    const uint32_t lanes = tensor_memory(ok) + ((uint32_t)(quad * 32) << 16);
    const uint32_t tempty0 = tc05::map_rank(smem_u32(tempty), lead);
    const int g = lane >> 2, q = lane & 3;
    uint32_t v = 0;
    // The accumulator is in registers (or in shared memory): back to the MMAs.
    auto give_back = [&](uint32_t b) {
      tc05::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc05::arrive_cluster(tempty0 + b * 8);
    };
    using S = typename Held<INT8>::type;
    constexpr int CW = W::CHUNK, GROUPS = CW / 8;  // columns of a chunk, and groups of 8
    // Puts out chunk c of the warp's part of unit t: its sums x, as tensor memory is read.  With the
    // contraction shared every KS-th group is this pair's.
    auto put_out = [&](const Unit& t, int c, const float* x) {
      const int np = t.n / W::PARTS, first = part * np, live = min(np, t.cnt - first);
      // first i of the warp's lanes (gated: of its 16 pairs), and the row of the output that o 0 of the unit is
      const int i0 = GATED ? (t.at * 8 + (int)rank * 4 + quad) * 16 : t.at * 256 + (int)rank * 128 + quad * 32;
      const size_t row0 = t.weights ? (size_t)t.e * p.O + t.o0 : (size_t)t.o0, row = row0 + first + CW * c;
      void* to = t.weights ? p.dw : p.y;
      const int left = live - CW * c;  // columns of the chunk that are outputs
      auto mine = [&](int col) { return KS == 1 || (c * GROUPS + (col >> 3)) % KS == split; };
      float r[CW];
      if constexpr (INT8) {
        float sw[4];  // scales of lanes g, g + 8, g + 16, g + 24
        const float* w = p.sw + (size_t)t.e * p.I * (GATED ? 2 : 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = i0 + g + 8 * (GATED ? i & 1 : i);
          sw[i] = __ldg(w + min(n, p.I - 1) + (GATED && i >= 2 ? p.I : 0));
        }
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) {
          float sx[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) sx[j] = __ldg(p.sx + min(row + 8 * k + 2 * q + j, (size_t)p.M - 1));
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int at = (j >> 2) * (CW / 2) + 4 * k + (j & 3);
            r[at] = x[at] * (sx[j & 1] * sw[(j >> 2) * 2 + ((j >> 1) & 1)]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < CW; ++i) r[i] = x[i];
      }
      auto f = [&](int h, int k, int j) { return r[CW / 2 * h + 4 * k + j]; };
      if (GATED && OUT == F32) {
        float* y = static_cast<float*>(p.y);
#pragma unroll
        for (int k = 0; k < GROUPS; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int col = 8 * k + 2 * q + (j & 1), i = i0 + (j >> 1) * 8 + g;
            if (mine(col) && col < left && i < p.I) y[(row + col) * p.I + i] = activation(f(0, k, j), p.act) * f(1, k, j);
          }
      } else if (GATED) {
        // 16 i's x the chunk's columns, through shared memory: rows of 32 bytes
        auto put = [&](uint16_t* to, size_t width, auto&& pair) {
          const uint32_t st = smem_u32(out) + ((lane >> 4) * 8 + (lane & 7)) * 48 + ((lane >> 3) & 1) * 16;
#pragma unroll
          for (int k = 0; k < GROUPS; k += 2)
            asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                             st + k * 8 * 48),
                         "r"(pair(k, 0)), "r"(pair(k, 2)), "r"(pair(k + 1, 0)), "r"(pair(k + 1, 2))
                         : "memory");
          __syncwarp();
#pragma unroll
          for (int k = 0; k < GROUPS / 2; ++k) {
            const int col = 16 * k + (lane >> 1);
            if (mine(col) && col < left && i0 < p.I)
              *reinterpret_cast<uint4*>(to + (row + col) * width + i0 + (lane & 1) * 8) =
                  *reinterpret_cast<const uint4*>(out + col * 48 + (lane & 1) * 16);
          }
          __syncwarp();
        };
        if (p.keep != nullptr) {
          put(p.keep, (size_t)2 * p.I, [&](int k, int j) { return bf16x2_bits(f(0, k, j), f(0, k, j + 1)); });
          put(p.keep + p.I, (size_t)2 * p.I, [&](int k, int j) { return bf16x2_bits(f(1, k, j), f(1, k, j + 1)); });
        }
        put(static_cast<uint16_t*>(p.y), (size_t)p.I, [&](int k, int j) {
          return bf16x2_bits(activation(f(0, k, j), p.act) * f(1, k, j),
                             activation(f(0, k, j + 1), p.act) * f(1, k, j + 1));
        });
      } else if (OUT == F32 && (MODE == FORWARD || t.weights)) {
        float* y = static_cast<float*>(to);
#pragma unroll
        for (int k = 0; k < GROUPS; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int col = 8 * k + 2 * q + (j & 1), i = i0 + 16 * h + (j >> 1) * 8 + g;
              if (mine(col) && col < left && i < p.I) y[(row + col) * p.I + i] = f(h, k, j);
            }
      } else {
        uint16_t* y = static_cast<uint16_t*>(to);
        const uint32_t st = smem_u32(out) + (lane & 7) * 80 + (lane >> 3) * 16;  // row lane % 8 of matrix lane / 8
#pragma unroll
        for (int k = 0; k < GROUPS; ++k)
          asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(st + k * 640),
                       "r"(bf16x2_bits(f(0, k, 0), f(0, k, 1))), "r"(bf16x2_bits(f(0, k, 2), f(0, k, 3))),
                       "r"(bf16x2_bits(f(1, k, 0), f(1, k, 1))), "r"(bf16x2_bits(f(1, k, 2), f(1, k, 3)))
                       : "memory");
        __syncwarp();
        const int i = i0 + (lane & 3) * 8;
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) {
          const int col = 8 * k + (lane >> 2);
          if (mine(col) && col < left && i < p.I) {  // the width is a multiple of 8
            uint4* dst = reinterpret_cast<uint4*>(y + (row + col) * p.I + i);
            const uint4 x = *reinterpret_cast<const uint4*>(out + col * 80 + (lane & 3) * 16);
            if (t.weights) __stcs(dst, x);  // read again by no kernel soon: operands stay in L2
            else *dst = x;
          }
        }
        __syncwarp();
      }
    };
    // Partial sums of a shared contraction: of register i of chunk c.
    S* parts = reinterpret_cast<S*>(sm) + tid;
    auto part_at = [&](int c, int i) { return (c * CW + i) * (W::OUT_WARPS * 32); };
    for (int u = u0; u < n_units && ok; u += ustep) {
      const Unit t = unit_of(u);
      const int np = t.n / W::PARTS, first = part * np;
      const Steps steps = steps_of(t);
      const int live = min(np, t.cnt - first);  // columns of this part that are outputs
      uint32_t b = 0;
      if constexpr (PROMOTE) {
        float held[4][32];  // integers: as `whole` says, their bits
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) held[c][i] = 0.f;
        constexpr int SEG = INT8 ? SEG_INT : SEG_F32;
        bool whole = false;
        // Adds the accumulator, 16 columns at a time; with registers to spare (not of integers) the next
        // ones are on their way meanwhile (4095 rows of 2048 x 1408, both gradients: 36.9 us, 37.9 without).
        auto add = [&](auto&& sum) {
          constexpr int AHEAD = INT8 ? 0 : 1;
          uint32_t r[1 + AHEAD][16];
          auto fetch = [&](int c) {
            const uint32_t ta = lanes + b * 256 + (uint32_t)(first + 16 * c);
            tc05::ld_16x256b_x2(ta, r[c & AHEAD]);
            tc05::ld_16x256b_x2(ta + (16u << 16), r[c & AHEAD] + 8);
          };
          if (AHEAD && live > 0) fetch(0);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (16 * c >= live) break;
            if (!AHEAD) fetch(c);
            tc05::wait_ld16(r[c & AHEAD]);
            if (AHEAD && c < 7 && 16 * (c + 1) < live) fetch(c + 1);
#pragma unroll
            for (int i = 0; i < 16; i += 2)
              sum(held[c >> 1] + (i >> 3) * 16 + (c & 1) * 8 + (i & 7), __uint_as_float(r[c & AHEAD][i]),
                  __uint_as_float(r[c & AHEAD][i + 1]));
          }
        };
        for (int k = steps.from; k < steps.to; k += SEG) {
          b = v % BUFS;
          ok = __all_sync(0xffffffffu, wait(&tfull[b], (v / BUFS) & 1));
          if (!ok) break;
          ++v;
          tc05::fence_after_sync();
          if (INT8 && whole) {
            add([](float* h, float x0, float x1) {
              h[0] = __int_as_float(__float_as_int(h[0]) + __float2int_rn(x0));
              h[1] = __int_as_float(__float_as_int(h[1]) + __float2int_rn(x1));
            });
          } else if (INT8) {
            add([](float* h, float x0, float x1) { f2unpack(f2add(f2pack(h[0], h[1]), f2pack(x0, x1)), h[0], h[1]); });
          } else {
            add([](float* h, float x0, float x1) {
              h[0] += x0;
              h[1] += x1;
            });
          }
          give_back(b);
          if (INT8 && !whole) {
            // While the MMAs go on: may the next segment be added in fp32?
            const bool end = k + SEG >= steps.to;
            float top = 0.f;
            if (!end)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (32 * c < live)
#pragma unroll
                  for (int i = 0; i < 32; ++i) top = fmaxf(top, fabsf(held[c][i]));
            whole = __any_sync(0xffffffffu, top > ROOM) || (KS > 1 && end);  // several pairs' sums may be large
            if (whole)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (32 * c < live)
#pragma unroll
                  for (int i = 0; i < 32; ++i) held[c][i] = __int_as_float(__float2int_rn(held[c][i]));
          }
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (32 * c >= live) break;
          if constexpr (KS == 1) {
            if (INT8 && whole)
#pragma unroll
              for (int i = 0; i < 32; ++i) held[c][i] = (float)__float_as_int(held[c][i]);
            put_out(t, c, held[c]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) parts[part_at(c, i)] = reinterpret_cast<const S&>(held[c][i]);
          }
        }
      } else {
        const bool any = steps.from < steps.to;
        if (any) {
          b = v % BUFS;
          ok = __all_sync(0xffffffffu, wait(&tfull[b], (v / BUFS) & 1));
          if (!ok) break;
          ++v;
          tc05::fence_after_sync();
        }
        // Chunk c of the accumulator, on its way to registers while the one before is put out.
        uint32_t next[16];
        auto fetch = [&](int c) {
          if (any && CW * c < live) {
            const uint32_t ta = lanes + b * 256 + (uint32_t)(first + CW * c);
            tc05::ld_16x256b_x2(ta, next);
            tc05::ld_16x256b_x2(ta + (16u << 16), next + 8);
          }
        };
        fetch(0);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (CW * c >= live) break;
          S x[CW];
          if (any) tc05::wait_ld16(next);
#pragma unroll
          for (int i = 0; i < CW; ++i) x[i] = any ? __uint_as_float(next[i & 15]) : 0.f;
          fetch(c + 1);
          if (any && CW * (c + 1) >= live) give_back(b);
          if constexpr (KS == 1) {
            put_out(t, c, x);
          } else {
#pragma unroll
            for (int i = 0; i < CW; ++i) parts[part_at(c, i)] = x[i];
          }
        }
        if (any && live <= 0) give_back(b);
      }
    }
    if constexpr (KS > 1) {
      __syncwarp();
      tc05::cluster_sync();  // every pair's sums are there
      if (u0 < n_units) {
        const Unit t = unit_of(u0);
        const int live = min(t.n / W::PARTS, t.cnt - part * (t.n / W::PARTS));
        uint32_t seen = 0;
#pragma unroll 1
        for (int c = 0; CW * c < live; ++c) {
          S x[CW];
#pragma unroll
          for (int i = 0; i < CW; ++i) x[i] = 0;
#pragma unroll
          for (int k = 0; k < GROUPS; ++k) {
            if ((c * GROUPS + k) % KS != split) continue;
#pragma unroll
            for (int j = 0; j < KS; ++j) {
              const uint32_t from = tc05::map_rank(smem_u32(parts), 2 * j + rank);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int at = (i >> 2) * (CW / 2) + 4 * k + (i & 3);
                uint32_t word;
                asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(word) : "r"(from + (uint32_t)part_at(c, at) * 4u) : "memory");
                x[at] += *reinterpret_cast<const S*>(&word);
                seen |= word;
              }
            }
          }
          float sums[CW];
#pragma unroll
          for (int i = 0; i < CW; ++i) sums[i] = (float)x[i];
          put_out(t, c, sums);
        }
        // The end barriers publish nothing, so they do not order these reads before the other pairs' end:
        // the vote does, which needs every word, those of columns that are no outputs too.  (What it
        // writes is read by no one any more.  A release would wait for the outputs: 64 rows of 2048 x
        // 2048 took 7.5 us with one, and 7.0 without.)
        if (__all_sync(0xffffffffu, seen == 0xFFFFFFFFu)) *abort_flag = 1;
      }
    }
  }
  // Nothing is under way to either CTA any more: every arrival and copy has been waited for, and the
  // other pairs' sums are in registers.  So the barriers publish nothing (a release would wait for
  // the outputs to land): this CTA's memory is read by no other any more; tensor memory is given back.
  __syncwarp();
  tc05::fence_before_sync();
  tc05::cluster_meet();
  if (warp == KEEPER) {
    tc05::fence_after_sync();
    tc05::dealloc_pair(*tslot, 512);
  }
  __syncwarp();
  tc05::cluster_meet();
}

EncodeTiled g_encode = nullptr;  // set once, under the caller's lock

// A map of bf16 elements (size 2) or bytes in the 128-byte swizzle, zeros outside.  dims
// from the innermost, strides in elements from the second dimension on.
bool encode(CUtensorMap* m, int size, const void* base, std::initializer_list<uint64_t> dims,
            std::initializer_list<uint64_t> strides, std::initializer_list<uint32_t> box) {
  cuuint64_t d[5], s[4];
  cuuint32_t b[5], one[5] = {1, 1, 1, 1, 1};
  int n = 0;
  for (uint64_t v : dims) d[n++] = v;
  n = 0;
  for (uint64_t v : strides) s[n++] = v * size;
  n = 0;
  for (uint32_t v : box) b[n++] = v;
  return g_encode(m, size == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)n, const_cast<void*>(base), d, s, b, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, bool GATED, int OUT, bool INT8, int KS>
cudaError_t launch_split(const PairArgs& p, const Maps& maps, long long most, int sm_count, cudaStream_t st) {
  const long long pairs = KS > 1 ? most : sm_count / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * KS * (unsigned)(most < pairs ? most : pairs));
  cfg.blockDim = dim3(Shape<OUT != BF16 || INT8, INT8>::THREADS);
  cfg.dynamicSmemBytes = pair_smem(p.E);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2 * KS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, pair_gemm_kernel<MODE, GATED, OUT, INT8, KS>, p, maps);
}
template <int MODE, bool GATED, int OUT, bool INT8 = false>
cudaError_t launch(const PairArgs& p, const Maps& maps, int ks, long long most, int sm_count, cudaStream_t st) {
  if (ks == 4) return launch_split<MODE, GATED, OUT, INT8, 4>(p, maps, most, sm_count, st);
  if (ks == 2) return launch_split<MODE, GATED, OUT, INT8, 2>(p, maps, most, sm_count, st);
  return launch_split<MODE, GATED, OUT, INT8, 1>(p, maps, most, sm_count, st);
}

// Tiles of rows that a grouped (or dense) product may have, at most.
long long row_tiles(int M, int E, bool grouped, int tile) {
  if (!grouped) return (M + tile - 1LL) / tile;
  return (long long)M / tile + (M < E ? M : E);
}

// What a step of 64 of the contracted dimension takes, measured (ns, 64 units of 256 x n on 76 pairs):
//   n          256  192  128   64   32
//   forward    287  234  201  201  199     below 160 columns the way of a stage through the ring
//   input      289  250  241  241  239
//   weights    285    -  304  304    -
//   integers   356  308  285    -  269
// A unit takes its steps, or its way out; a launch 3 us (integers 3.5) and the last unit's way out besides.
enum Kind { K_FORWARD, K_INPUT, K_WEIGHTS, K_INTEGERS };
long long unit_ns(long long steps, int n, Kind kind) {
  constexpr int LEAST[] = {200, 240, 285, 269};
  const int by_columns = kind == K_INTEGERS ? 190 + n * 2 / 3 : 75 + n * 5 / 6;
  const long long loop = steps * (by_columns > LEAST[kind] ? by_columns : LEAST[kind]), out = 5 * n;
  return loop > out ? loop : out;
}
long long launch_ns(int n, bool int8 = false) { return int8 ? 3500 + 10 * n : 3000 + 8 * n; }

// Clusters of KS pairs that run at a time: a pair has two neighbouring SMs, and a cluster lies in
// one of the GPU's parts of 18 to 20 SMs.
long long clusters_of(int ks, int pairs) { return ks == 4 ? pairs / 5 : ks == 2 ? pairs * 2 / 5 : pairs; }
// What joining a shared contraction takes (integers: 32 rows of 2048 x 8192 1.7 us, 256 rows 4.2).
long long join_ns(int ks, int n = 0) { return ks > 1 ? (n ? 1300 + 11 * n : 2000) : 0; }

struct Plan {
  int tile, tile_w, ks;
  long long ns;
};

// Tile of a dense product's rows, and pairs that share its contraction, so that the units fill the
// pairs of SMs evenly.
Plan plan_forward(int M, long long a_tiles, long long steps, bool int8, int pairs, int most_ks) {
  Plan best = {256, 256, 1, -1};
  for (int ks = 1; ks <= most_ks; ks *= 2)
    for (int tile = 256; tile >= 32; tile -= 32) {
      const long long units = (M + tile - 1LL) / tile * a_tiles, room = clusters_of(ks, pairs);
      if (ks > 1 && (units > room || steps < 4 * ks)) continue;
      const int n = M < tile ? (M + 31) & ~31 : tile;
      const long long c = (units + room - 1) / room * unit_ns((steps + ks - 1) / ks, n, int8 ? K_INTEGERS : K_FORWARD) +
                          launch_ns(n, int8) + join_ns(ks, int8 ? n : 0);
      if (best.ns < 0 || c < best.ns) best = {tile, 256, ks, c};
    }
  return best;
}

// The same for both gradients in one launch (or one alone): units of dx first, then of dw, dealt out in turn.
Plan plan_backward(int M, int N, long long a_tiles, bool dx, bool dw, int pairs, int most_ks) {
  const long long dx_steps = (N + 63) / 64, dw_steps = (M + 63) / 64;
  Plan best = {256, 256, 1, -1};
  for (int ks = 1; ks <= most_ks; ks *= 2)
    for (int tile = 256; tile >= (dx ? 64 : 256); tile -= 32)
      for (int tile_w = 256; tile_w >= (dw ? 128 : 256); tile_w -= 128) {  // whole pieces of 64 columns
        const long long a = dx ? (M + tile - 1LL) / tile * a_tiles : 0, b = dw ? (N + tile_w - 1LL) / tile_w * a_tiles : 0;
        const long long room = clusters_of(ks, pairs);
        if (ks > 1 && (a + b > room || (dx ? dx_steps : 0) + (dw ? dw_steps : 0) < 8 * ks)) continue;
        const int n = M < tile ? (M + 31) & ~31 : tile;
        const long long ca = unit_ns((dx_steps + ks - 1) / ks, n, K_INPUT);
        const long long cb = unit_ns((dw_steps + ks - 1) / ks, tile_w, K_WEIGHTS);
        const long long edge = a % room, end = (a + b) % room;  // pairs below an edge have one unit more
        long long most = 0;
        for (long long q : {0LL, edge, end}) {
          if (q >= room) continue;
          const long long na = a / room + (q < edge), all = (a + b) / room + (q < end);
          const long long c = na * ca + (all - na) * cb;
          if (c > most) most = c;
        }
        most += launch_ns(dw ? tile_w : n) + join_ns(ks);
        if (best.ns < 0 || most < best.ns) best = {tile, tile_w, ks, most};
      }
  return best;
}

bool encode_rows(Maps& m, int size, const void* x, uint64_t rows, uint64_t K) {
  for (uint32_t i = 0; i < 4; ++i)
    if (!encode(&m.b[i], size, x, {K, rows}, {K}, {128u / size, 16u << i})) return false;
  return true;
}

}  // namespace

cudaError_t pair_gemm_kernels_init(int* most_ks) {
  if (g_encode == nullptr) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    if (q != cudaDriverEntryPointSuccess || fn == nullptr) return cudaErrorNotSupported;
    g_encode = reinterpret_cast<EncodeTiled>(fn);
  }
#define PAIR_KERNELS(ks)                                                                               \
  {reinterpret_cast<const void*>(pair_gemm_kernel<FORWARD, true, BF16, false, ks>), 0},                \
      {reinterpret_cast<const void*>(pair_gemm_kernel<FORWARD, false, BF16, false, ks>), 0},           \
      {reinterpret_cast<const void*>(pair_gemm_kernel<BACKWARD, false, BF16, false, ks>), 0},          \
      {reinterpret_cast<const void*>(pair_gemm_kernel<FORWARD, false, F32, false, ks>), LAUNCH},       \
      {reinterpret_cast<const void*>(pair_gemm_kernel<BACKWARD, false, F32, false, ks>), LAUNCH},      \
      {reinterpret_cast<const void*>(pair_gemm_kernel<BACKWARD, false, BF16_ADDED, false, ks>), LAUNCH}, \
      {reinterpret_cast<const void*>(pair_gemm_kernel<FORWARD, false, BF16, true, ks>), LAUNCH_INT},   \
      {reinterpret_cast<const void*>(pair_gemm_kernel<FORWARD, false, F32, true, ks>), LAUNCH_INT},    \
      {reinterpret_cast<const void*>(pair_gemm_kernel<FORWARD, true, BF16, true, ks>), LAUNCH_INT},    \
      {reinterpret_cast<const void*>(pair_gemm_kernel<FORWARD, true, F32, true, ks>), LAUNCH_INT}
  constexpr int LAUNCH = Shape<true, false>::LAUNCH, LAUNCH_INT = Shape<true, true>::LAUNCH;
  const struct {
    const void* f;
    int regs;  // that its shares are counted from
  } k[] = {PAIR_KERNELS(1), PAIR_KERNELS(2), PAIR_KERNELS(4)};
#undef PAIR_KERNELS
  for (const auto& x : k) {
    cudaError_t e = cudaFuncSetAttribute(x.f, cudaFuncAttributeMaxDynamicSharedMemorySize, pair_smem(ROUTE_MAX_E));
    if (e != cudaSuccess) return e;
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, x.f)) != cudaSuccess) return e;
    if (fa.numRegs < x.regs) return cudaErrorInvalidConfiguration;  // the shares would never be met
  }
  // Pairs of a cluster that share a contraction, as many as the device places.
  *most_ks = 1;
  for (int ks = 2; ks <= 4; ks *= 2) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2 * ks;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * ks);
    cfg.blockDim = dim3(Shape<true, true>::THREADS);
    cfg.dynamicSmemBytes = pair_smem(ROUTE_MAX_E);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int fit = 0;
    const cudaError_t e = ks == 2 ? cudaOccupancyMaxActiveClusters(&fit, pair_gemm_kernel<FORWARD, true, F32, true, 2>, &cfg)
                                  : cudaOccupancyMaxActiveClusters(&fit, pair_gemm_kernel<FORWARD, true, F32, true, 4>, &cfg);
    if (e != cudaSuccess) (void)cudaGetLastError();
    if (e != cudaSuccess || fit < 1) break;
    *most_ks = ks;
  }
  return cudaSuccess;
}

namespace {

// A dense product's tiles of rows, all of one size, to 32.
void dense_rows(PairArgs& p) {
  p.row_tiles = (p.M + p.tile - 1) / p.tile;
  p.units = p.y != nullptr ? p.row_tiles * p.a_tiles : 0;
  p.rows = p.M | ((p.M + p.row_tiles - 1) / p.row_tiles + 31) >> 5 << 26;
}

}  // namespace

cudaError_t launch_pair_forward(const ProductArgs& a, bool int8, const PairDevice& dev, cudaStream_t st) {
  const bool gated = a.act != FFN_NONE;
  const uint64_t M = a.M, N = a.N, K = a.K, E = a.E;
  PairArgs p = {};
  p.offsets = a.offsets;
  p.y = a.y;
  p.keep = static_cast<uint16_t*>(a.keep);
  p.sx = a.sx;
  p.sw = a.sw;
  p.err = dev.err;
  p.M = a.M;
  p.E = a.E;
  p.I = gated ? a.N / 2 : a.N;
  p.steps = int8 ? (a.K + 127) / 128 : (a.K + 63) / 64;
  p.a_tiles = (a.N + 255) / 256;
  const Plan plan = a.offsets == nullptr ? plan_forward(a.M, p.a_tiles, (a.K + 63) / 64, int8, dev.sms / 2, dev.most_ks)
                                         : Plan{256, 256, 1, 0};
  p.tile = plan.tile;
  p.act = a.act;
  dense_rows(p);
  p.per_band = reciprocal(BAND * p.a_tiles);
  Maps m;
  const int size = int8 ? 1 : 2;
  const uint32_t inner = 128 / size;
  const bool ok =
      gated ? encode(&m.a, size, a.w, {K, 16, 2, N / 32, E}, {K, N / 2 * K, 16 * K, N * K}, {inner, 16, 2, 4, 1})
            : encode(&m.a, size, a.w, {K, N, E}, {K, N * K}, {inner, 128, 1});
  if (!ok || !encode_rows(m, size, a.x, M, K)) return cudaErrorInvalidValue;
  m.aw = m.bw = m.bw1 = m.bw2 = m.a;
  const long long most = row_tiles(a.M, a.E, a.offsets != nullptr, p.tile) * p.a_tiles;
  if (int8) {
    if (gated) return a.f32 ? launch<FORWARD, true, F32, true>(p, m, plan.ks, most, dev.sms, st)
                            : launch<FORWARD, true, BF16, true>(p, m, plan.ks, most, dev.sms, st);
    return a.f32 ? launch<FORWARD, false, F32, true>(p, m, plan.ks, most, dev.sms, st)
                 : launch<FORWARD, false, BF16, true>(p, m, plan.ks, most, dev.sms, st);
  }
  if (gated) return launch<FORWARD, true, BF16>(p, m, plan.ks, most, dev.sms, st);
  return a.f32 ? launch<FORWARD, false, F32>(p, m, plan.ks, most, dev.sms, st)
               : launch<FORWARD, false, BF16>(p, m, plan.ks, most, dev.sms, st);
}

namespace {

cudaError_t launch_backward(const GradArgs& a, const Plan& plan, const PairDevice& dev, cudaStream_t st) {
  const uint64_t M = a.M, N = a.N, K = a.K, E = a.E;
  PairArgs p = {};
  p.offsets = a.offsets;
  p.y = a.dx;
  p.dw = a.dw;
  p.err = dev.err;
  p.M = a.M;
  p.E = a.E;
  p.I = a.K;
  p.O = a.N;
  p.steps = (a.N + 63) / 64;
  p.a_tiles = (a.K + 255) / 256;
  p.pieces_k = a.K % 64 == 0;
  p.pieces_n = a.N % 64 == 0;
  p.tile = plan.tile;
  p.tile_w = plan.tile_w;
  if (a.dw != nullptr) p.o_tiles = (a.N + p.tile_w - 1) / p.tile_w;
  dense_rows(p);
  p.per_band = reciprocal(BAND * p.a_tiles);
  p.per_expert = reciprocal(a.dw != nullptr ? p.o_tiles * p.a_tiles : 1);
  Maps m;
  bool ok = encode_rows(m, 2, a.dy, M, N);
  ok = ok && (p.pieces_k ? encode(&m.a, 2, a.w, {64, N, K / 64, E}, {K, 64, N * K}, {64, 64, 2, 1})
                         : encode(&m.a, 2, a.w, {K, N, E}, {K, N * K}, {64, 64, 1}));
  ok = ok && (p.pieces_k ? encode(&m.aw, 2, a.x, {64, M, K / 64}, {K, 64}, {64, 64, 2})
                         : encode(&m.aw, 2, a.x, {K, M}, {K}, {64, 64}));
  ok = ok && encode(&m.bw, 2, a.dy, {N, M}, {N}, {64, 64});
  m.bw1 = m.bw2 = m.bw;
  if (p.pieces_n)
    ok = ok && encode(&m.bw1, 2, a.dy, {64, M, N / 64}, {N, 64}, {64, 64, 1}) &&
         encode(&m.bw2, 2, a.dy, {64, M, N / 64}, {N, 64}, {64, 64, 2});
  if (!ok) return cudaErrorInvalidValue;
  long long most = (long long)a.E * p.o_tiles * p.a_tiles;
  if (a.dx != nullptr) most += row_tiles(a.M, a.E, a.offsets != nullptr, p.tile) * p.a_tiles;
  // (an expert may have all of the rows)
  if (a.f32) return launch<BACKWARD, false, F32>(p, m, plan.ks, most, dev.sms, st);
  return a.dw != nullptr && a.M > ALONE ? launch<BACKWARD, false, BF16_ADDED>(p, m, plan.ks, most, dev.sms, st)
                                        : launch<BACKWARD, false, BF16>(p, m, plan.ks, most, dev.sms, st);
}

}  // namespace

cudaError_t launch_pair_backward(const GradArgs& a, const PairDevice& dev, cudaStream_t st) {
  const int a_tiles = (a.K + 255) / 256, pairs = dev.sms / 2;
  const bool dx = a.dx != nullptr, dw = a.dw != nullptr;
  if (a.offsets != nullptr) return launch_backward(a, Plan{256, 256, 1, 0}, dev, st);
  const Plan plan = plan_backward(a.M, a.N, a_tiles, dx, dw, pairs, dev.most_ks);
  if (dx && dw) {
    // Long units of one and short ones of the other fill a launch badly: 16 rows of 8192 x 2048 take 41
    // us in one and 25 in two, each with its own share of the contraction a cluster.
    const Plan one = plan_backward(a.M, a.N, a_tiles, true, false, pairs, dev.most_ks);
    const Plan two = plan_backward(a.M, a.N, a_tiles, false, true, pairs, dev.most_ks);
    if (one.ns + two.ns < plan.ns) {
      GradArgs g = a;
      g.dw = nullptr;
      const cudaError_t e = launch_backward(g, one, dev, st);
      if (e != cudaSuccess) return e;
      g.dw = a.dw;
      g.dx = nullptr;
      return launch_backward(g, two, dev, st);
    }
  }
  return launch_backward(a, plan, dev, st);
}

// Whether the few-row kernel takes a product.  By expert: up to 8 rows an expert on average (1,536 rows
// of 256 experts 162 us, pairs 168; integers 107 and 131).  The host knows no expert's rows: where many
// fall to one, its weights are read again for every 8 of them, from L2, which takes longer than the
// pairs would and less than the same rows spread over all experts.  Dense: its passes of 8 rows over the weights,
// from L2 at 10.5 TB/s (integers 6.8), against the pairs' plan:
//   rows of N x K      few, pairs (us)
//   32 of 2048 x 2048   6.3,  6.8    but 48:  8.4,  6.4    integers  64:  7.0,  8.2 but 128: 12.7, 10.1
//   16 of 8192 x 2048   9.9,  9.8    but 24: 13.8,  9.9    integers  24:  9.8, 11.7 but  40: 14.7, 12.3
//   16 of 4096 x 4096  10.5, 10.9    but 24: 14.2, 11.0    integers  32: 12.8, 13.4 but  40: 15.5, 13.5
bool few_rows_take(const ProductArgs& a, bool int8, const PairDevice& dev) {
  if (a.offsets != nullptr) return a.M <= 8LL * a.E;
  if (a.M <= 8) return true;
  if (a.M > 256) return false;
  const long long bytes = (long long)a.N * a.K * (int8 ? 1 : 2), passes = (a.M + 7) / 8;
  return 3000 + passes * bytes / (int8 ? 6800 : 10500) <=
         plan_forward(a.M, (a.N + 255) / 256, (a.K + 63) / 64, int8, dev.sms / 2, dev.most_ks > 0 ? dev.most_ks : 1).ns;
}

}  // namespace flint

// For the tests: what a dense product (what 0: forward, 1: integers, 2: dx, 3: dw, 4: both) takes on a GPU
// of so many SMs: 0 the few-row kernel, else the pairs' KS * 1000000 + tile * 1000 + tile of dw.
extern "C" int flint_linear_plan(int what, int M, int N, int K, int sm_count) {
  using namespace flint;
  Plan plan;
  if (what < 2) {
    ProductArgs a = {};
    a.M = M;
    a.N = N;
    a.K = K;
    a.E = 1;
    if (few_rows_take(a, what == 1, PairDevice{sm_count, 4, nullptr})) return 0;
    plan = plan_forward(M, (N + 255) / 256, (K + 63) / 64, what == 1, sm_count / 2, 4);
  } else {
    plan = plan_backward(M, N, (K + 255) / 256, what != 3, what != 2, sm_count / 2, 4);
  }
  return plan.ks * 1000000 + plan.tile * 1000 + plan.tile_w;
}
