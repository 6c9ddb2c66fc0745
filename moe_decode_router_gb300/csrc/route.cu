// Routing to experts from given logits, and grouping of the chosen pairs by
// expert, for any number of experts (the sublayer calls have both built in for
// their one shape).
//
// Routing, one warp per token.  With s = sigmoid(logit) or softmax over the
// row, an expert is chosen by its key: the logit itself without a bias (both
// scores grow with it, so the order is exact), s + bias with one.  Ties go to
// the lower index.  A selection is a whole number and has no "almost": scores
// are first formed in fp32, and where two neighbours in the order, or a kept
// and a dropped group, are closer than the fp32 error bound, the warp puts those
// candidates in order in fp64 (about one row in 250 with 256 experts and a
// bias), or the whole row where that needs more than the candidates.
//
// Bound by dependent steps: a pick is one redux of the lanes' best keys, one of the
// indices that have it, and the next best in the lane that owned it (every lane
// keeps two at hand), one pick after another; and by a last wave that is mostly
// empty (2,048 blocks are 2.25 waves).  Some 1,000 instructions a row with groups
// and bias use 55 % of the issue slots while the SMs are busy, 39 % in all.  A lane's
// experts are neighbours: the row comes in 16-byte loads, and a group of whole
// lanes is scored by shuffles among them.  8,191 rows of 256 fp32 with 8 groups,
// bias and 8 picks: 276 us with every score in fp64, 15.4 us with the experts
// dealt out one by one, 13.1 us this way (the bytes alone: 1.3 us); 8,192 rows
// of 256 bf16, softmax, no groups: 8.1 us.
#include <type_traits>

#include "flint_common.cuh"
#include "flint_internal.h"

namespace flint {

namespace {

constexpr unsigned FULL = 0xffffffffu;

// Order-preserving key of a float, never 0 for a value above -inf; -0 and +0
// share a key.
__device__ __forceinline__ uint32_t ord_key(float f) {
  const uint32_t b = __float_as_uint(__fadd_rn(f, 0.0f));
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}

// A lane holds EPL neighbouring experts: lane * EPL + i.
struct RouteParams {
  const void* logits;
  long long stride;  // elements between rows
  const float* bias;
  int32_t* ids;
  float* w;
  int T, E, top_k, n_groups, top_groups;
  int softmax, top2, renorm;
  uint32_t recip;  // ceil(2^20 / experts of a group): e * recip >> 20 is expert e's group for e < 1024
  int group_lanes;  // lanes of a group where that is a power of two, else 0
  bool wide_loads;  // rows start on 16-byte boundaries
  float scale;
};

// The two largest of the values that the lanes hold as (a, b), a >= b, -inf
// where there is none; every lane gets the result.
template <typename F>
__device__ __forceinline__ void warp_top2(F& a, F& b) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const F oa = __shfl_xor_sync(FULL, a, off), ob = __shfl_xor_sync(FULL, b, off);
    if (oa > a) {
      b = a > ob ? a : ob;
      a = oa;
    } else {
      b = b > oa ? b : oa;
    }
  }
}

// Score of every group: lane g of the result holds group g's, -inf for a group
// without candidates and for lanes without a group.
template <typename F, int EPL>
__device__ __forceinline__ F group_scores(const F (&v)[EPL], int lane, int E, int G, bool top2) {
  const int size = E / G;
  F mine = -(F)INFINITY;
  for (int g = 0; g < G; ++g) {
    F a = -(F)INFINITY, b = -(F)INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane * EPL + i;
      if (e >= g * size && e < (g + 1) * size) {
        if (v[i] > a) {
          b = a;
          a = v[i];
        } else if (v[i] > b) {
          b = v[i];
        }
      }
    }
    warp_top2(a, b);
    const F s = (top2 && b > -(F)INFINITY) ? a + b : a;
    if (lane == g) mine = s;
  }
  return mine;
}

// Bit g of the result: group g is among the `top` best (ties to the lower
// group).  `unsure` is set when a kept and a dropped score are within `tol` of
// each other.
template <typename F>
__device__ __forceinline__ uint32_t keep_groups(F score, int lane, int G, int top, F tol, bool& unsure) {
  int rank = 0;
  for (int g = 0; g < G; ++g) {
    const F o = __shfl_sync(FULL, score, g);
    if (o > score || (o == score && g < lane)) ++rank;
  }
  const bool kept = lane < G && rank < top;
  const uint32_t mask = __ballot_sync(FULL, kept);
  // weakest kept score and strongest dropped one
  F lo = kept ? score : (F)INFINITY, hi = (lane < G && !kept) ? score : -(F)INFINITY;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const F l = __shfl_xor_sync(FULL, lo, off), h = __shfl_xor_sync(FULL, hi, off);
    lo = l < lo ? l : lo;
    hi = h > hi ? h : hi;
  }
  unsure = hi > -(F)INFINITY && !(lo - hi > tol);
  return mask;
}

template <typename F, int EPL>
__device__ __forceinline__ void softmax_scores(const float (&x)[EPL], F (&s)[EPL]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; ++i) m = x[i] > m ? x[i] : m;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, off));
  F z = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    s[i] = x[i] > -INFINITY ? (x[i] == m ? (F)1 : exp((F)x[i] - (F)m)) : (F)0;
    z += s[i];
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(FULL, z, off);
#pragma unroll
  for (int i = 0; i < EPL; ++i) s[i] = z > 0 ? s[i] / z : (F)0;
}

template <typename F, int EPL>
__device__ __forceinline__ void all_scores(const RouteParams& p, const float (&x)[EPL], F (&s)[EPL]) {
  if (p.softmax) {
    softmax_scores<F, EPL>(x, s);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] = x[i] > -INFINITY ? (F)1 / ((F)1 + exp(-(F)x[i])) : (F)0;
  }
}

// Keys (choice) and values (groups) of the row in type F; -inf: not a candidate.
template <typename F, int EPL>
__device__ __forceinline__ void keys_of(const RouteParams& p, const float (&x)[EPL], const F (&s)[EPL], int lane,
                                        F (&key)[EPL]) {
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    F k = -(F)INFINITY;
    if (x[i] > -INFINITY) {
      k = (p.bias != nullptr && e < p.E) ? s[i] + (F)__ldg(p.bias + e) : (F)x[i];
      if (!(k > -(F)INFINITY)) k = -(F)INFINITY;
    }
    key[i] = k;
  }
}

// Takes the groups that are out away from the keys.
template <typename F, int EPL>
__device__ __forceinline__ void drop_groups(F (&key)[EPL], int lane, int size, uint32_t kept) {
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int g = (lane * EPL + i) / size;
    if (g >= 32 || !((kept >> g) & 1u)) key[i] = -(F)INFINITY;
  }
}

// The `n` best keys in order: lane k ends with the k-th's expert (-1: none
// left) and key.
template <typename F, int EPL>
__device__ __forceinline__ void select_best(const F (&key)[EPL], int lane, int n, int& my_e, F& my_key) {
  uint32_t taken = 0u;
  my_e = -1;
  my_key = -(F)INFINITY;
  for (int k = 0; k < n; ++k) {
    F best = -(F)INFINITY;
    int at = 1 << 20;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (!((taken >> i) & 1u) && key[i] > best) {
        best = key[i];
        at = lane * EPL + i;
      }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const F ob = __shfl_xor_sync(FULL, best, off);
      const int oa = __shfl_xor_sync(FULL, at, off);
      if (ob > best || (ob == best && oa < at)) {
        best = ob;
        at = oa;
      }
    }
    if (!(best > -(F)INFINITY)) break;
    if (at / EPL == lane) taken |= 1u << (at % EPL);
    if (lane == k) {
      my_e = at;
      my_key = best;
    }
  }
}

// The row in fp64.
template <int EPL>
__device__ __noinline__ void route_row_f64(const RouteParams& p, const float (&x)[EPL], int lane, int& my_e) {
  double s[EPL], key[EPL], my_key;
  all_scores<double, EPL>(p, x, s);
  keys_of<double, EPL>(p, x, s, lane, key);
  if (p.n_groups > 1) {
    uint32_t kept;
    bool unsure;
    if (p.bias == nullptr && p.top2) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (!(x[i] > -INFINITY)) s[i] = -INFINITY;
      kept = keep_groups<double>(group_scores<double, EPL>(s, lane, p.E, p.n_groups, true), lane, p.n_groups,
                                 p.top_groups, 0.0, unsure);
    } else {
      kept = keep_groups<double>(group_scores<double, EPL>(key, lane, p.E, p.n_groups, p.top2 != 0), lane, p.n_groups,
                                 p.top_groups, 0.0, unsure);
    }
    drop_groups<double, EPL>(key, lane, p.E / p.n_groups, kept);
  }
  select_best<double, EPL>(key, lane, p.top_k, my_e, my_key);
}

__device__ __forceinline__ float ord_value(uint32_t k) {
  return k == 0u ? -INFINITY : __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k);
}

// fp32 error of a score: a sigmoid's from ex2 (2 units, and its argument's
// rounding, |x| 2^-24 times s (1 - s) < 0.25 / |x|), one addition and one
// reciprocal, below 2^-22, of which twice is allowed for; a softmax's from the
// same and a sum of up to 1024 terms (32 a lane, 5 steps: 36 roundings), below
// 2.6e-6 of the row's largest score, of which 3.8e-6 is allowed for.
constexpr float SIGMOID_ERR = 4.76837158203125e-07f;  // 2^-21
constexpr float SOFTMAX_ERR = 3.814697265625e-06f;    // 2^-18, of the row's largest score
constexpr float SUM_ERR = 1.1920928955078125e-07f;    // 2^-23: two roundings

__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Returns the scores' error bound.
template <int EPL>
__device__ __forceinline__ float fast_scores(const RouteParams& p, const float (&x)[EPL], float (&s)[EPL]) {
  if (p.softmax) {
    float m = -INFINITY, z = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) m = x[i] > m ? x[i] : m;
    m = ord_value(redux_max(m > -INFINITY ? ord_key(m) : 0u));
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      s[i] = x[i] > -INFINITY ? (x[i] == m ? 1.f : __expf(x[i] - m)) : 0.f;
      z += s[i];
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(FULL, z, off);
    const float r = rcp_approx(z);
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] *= r;
    return SOFTMAX_ERR * r;  // the largest score is 1 / z
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) s[i] = rcp_approx(1.f + __expf(-x[i]));
  return SIGMOID_ERR;
}

// A softmax row's largest logit and the sum of exp(x - largest) in fp64.
template <int EPL>
__device__ __noinline__ void softmax_sum_f64(const float (&x)[EPL], float& m, double& z) {
  m = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; ++i) m = x[i] > m ? x[i] : m;
  m = ord_value(redux_max(m > -INFINITY ? ord_key(m) : 0u));
  z = 0.0;
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (x[i] > -INFINITY) z += x[i] == m ? 1.0 : exp((double)x[i] - (double)m);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(FULL, z, off);
}
// One expert's score in fp64; m and z of its row, for a softmax.
__device__ __forceinline__ double score_f64(const RouteParams& p, float x, float m, double z) {
  if (p.softmax) return (x == m ? 1.0 : exp((double)x - (double)m)) / z;
  return 1.0 / (1.0 + exp(-(double)x));
}

// Decides the groups in fp64 from each group's two best experts, one value a
// lane.  val: the fp32 values' keys.  False where fp32 does not
// tell which experts those are, or where there are more than 32.
template <int EPL>
__device__ __noinline__ bool refine_groups(const RouteParams& p, const float (&x)[EPL], const uint32_t (&val)[EPL],
                                           float err, int lane, uint32_t& mask) {
  const int G = p.n_groups, size = p.E / G, take = p.top2 ? 2 : 1;
  if (G * take > 32) return false;
  int mine = -1;  // expert of lane g * take + j
  for (int g = 0; g < G; ++g) {
    uint32_t done = 0u;
    float last = 0.f;
    for (int j = 0; j <= take; ++j) {  // one more than counts, to see how close it comes
      uint32_t best = 0u;
      int at = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane * EPL + i;
        if (e >= g * size && e < (g + 1) * size && !((done >> i) & 1u) && val[i] > best) {
          best = val[i];
          at = i;
        }
      }
      const uint32_t m = redux_max(best);
      if (m == 0u) break;
      const float v = ord_value(m);
      if (j == take) {
        if (!(last - v > 2.f * err + SUM_ERR * (fabsf(v) + fabsf(last)))) return false;
        break;
      }
      last = v;
      const int e = (int)redux_min(best == m ? (uint32_t)(lane * EPL + at) : 0xFFFFFFFFu);
      if (lane == g * take + j) mine = e;
      if (e / EPL == lane) done |= 1u << at;
    }
  }
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const float o = __shfl_sync(FULL, x[i], mine / EPL);
    if (mine % EPL == i) mx = o;
  }
  float m = 0.f;
  double z = 1.0, v = -INFINITY;
  if (p.softmax) softmax_sum_f64<EPL>(x, m, z);
  if (mine >= 0) v = score_f64(p, mx, m, z) + (p.bias != nullptr ? (double)__ldg(p.bias + mine) : 0.0);
  const double first = __shfl_sync(FULL, v, (lane * take) & 31), second = __shfl_sync(FULL, v, (lane * take + 1) & 31);
  double score = lane < G ? first : -INFINITY;
  if (lane < G && take == 2 && second > -INFINITY) score = first + second;
  bool unsure;
  mask = keep_groups<double>(score, lane, G, p.top_groups, 0.0, unsure);
  return true;
}

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// The lane's EPL values of a row of E, `none` beyond it; up to 16 bytes a load
// where the row is aligned for it.
template <int EPL, typename V>
__device__ __forceinline__ void load_experts(const V* row, bool aligned, int lane, int E, float none, float (&x)[EPL]) {
  constexpr int N = EPL * sizeof(V) < 16 ? EPL : 16 / sizeof(V);  // of a load
  struct alignas(N * sizeof(V)) Chunk {
    V v[N];
  };
#pragma unroll
  for (int c = 0; c < EPL; c += N) {
    const int e = lane * EPL + c;
    if (aligned && e + N <= E) {
      const Chunk u = *reinterpret_cast<const Chunk*>(row + e);
#pragma unroll
      for (int i = 0; i < N; ++i) x[c + i] = as_f32(u.v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[c + i] = e + i < E ? as_f32(row[e + i]) : none;
    }
  }
}

// Selection with fp32 scores: my_e of lane k = the k-th expert (-1: none).
// False where fp32 does not decide it.
template <int EPL, typename V>
__device__ __forceinline__ bool route_row_f32(const RouteParams& p, const float (&x)[EPL], const V* row, int lane,
                                              int& my_e) {
  const bool biased = p.bias != nullptr;
  float err = 0.f;
  const bool sums = p.n_groups > 1 && p.top2;
  uint32_t key[EPL];  // choice, 0: not a candidate
  float s[EPL];
  if (biased || sums) err = fast_scores<EPL>(p, x, s);
  if (biased) {
    float bias[EPL];
    load_experts<EPL>(p.bias, true, lane, p.E, 0.f, bias);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float k = s[i] + bias[i];
      key[i] = (x[i] > -INFINITY && k > -INFINITY) ? ord_key(k) : 0u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = x[i] > -INFINITY ? ord_key(x[i]) : 0u;
  }
  // the groups' values: the keys, or without a bias the scores to be summed
  auto value = [&](int i) { return (sums && !biased) ? (key[i] != 0u ? ord_key(s[i]) : 0u) : key[i]; };
  const int G = p.n_groups, size = p.E / G;
  // Which groups stay (bit g * step of the mask), from their two best values g1,
  // g2, held by lane `leader` of group g at g * step; `member` is the lane's own group.
  auto decide = [&](uint32_t g1, uint32_t g2, int member, int step, uint32_t& mask) -> bool {
    const bool leader = lane == member * step && member < G;
    const float v1 = ord_value(g1), v2 = p.top2 && g2 != 0u ? ord_value(g2) : 0.f, score = v1 + v2;
    int rank = 0;
    for (int g = 0; g < G; ++g) {
      const float o = __shfl_sync(FULL, score, g * step);
      if (o > score || (o == score && g < member)) ++rank;
    }
    const bool kept = leader && rank < p.top_groups;
    const uint32_t leaders = __ballot_sync(FULL, kept);  // bit g * step
    if (biased || sums) {  // weakest kept group against strongest dropped one, each at its error's far end
      // Both keys' errors and roundings, the sum's and this one's: by the size of the
      // keys, which may nearly cancel.
      const float tol = 2.f * err + 1.5f * SUM_ERR * (fabsf(v1) + fabsf(v2));
      const bool some = leader && g1 != 0u;  // a group with candidates, also where their sum is beyond fp32
      const uint32_t low = some ? ord_key(fmaxf(score - tol, -INFINITY)) : 0u;  // fmaxf, fminf: NaN of two infinities
      const uint32_t high = some ? ord_key(fminf(score + tol, INFINITY)) : 0u;
      const uint32_t lo = redux_min(kept ? low : 0xFFFFFFFFu), hi = redux_max(kept ? 0u : high);
      if (hi != 0u && lo <= hi) {
        float xc[EPL];  // copies: what a call takes by address does not stay in registers
        uint32_t val[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          xc[i] = x[i];
          val[i] = value(i);
        }
        uint32_t better;
        if (!refine_groups<EPL>(p, xc, val, err, lane, better)) return false;
        mask = 0u;
        for (int g = 0; g < G; ++g) mask |= ((better >> g) & 1u) << (g * step);
        return true;
      }
    }
    mask = leaders;
    return true;
  };
  if (G > 1 && p.group_lanes == 0) {  // groups that do not fall on whole lanes
    uint32_t g1 = 0u, g2 = 0u;        // lane g: group g's two best
    for (int g = 0; g < G; ++g) {
      uint32_t a = 0u, b = 0u;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane * EPL + i;
        if (e >= g * size && e < (g + 1) * size) {
          const uint32_t k = value(i);
          b = max(b, min(a, k));
          a = max(a, k);
        }
      }
      const uint32_t m1 = redux_max(a);
      const uint32_t who = __ballot_sync(FULL, a == m1);
      const uint32_t m2 = redux_max(lane == __ffs(who) - 1 ? b : a);
      if (lane == g) {
        g1 = m1;
        g2 = m2;
      }
    }
    uint32_t mask;
    if (!decide(g1, g2, lane, 1, mask)) return false;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const uint32_t g = ((uint32_t)(lane * EPL + i) * p.recip) >> 20;
      if (!((mask >> (g & 31u)) & 1u)) key[i] = 0u;  // beyond the last expert the key is 0 already
    }
  }

  // The lane's two best; a lane that wins twice looks for its next one among the
  // rest.
  uint32_t best = 0u, second = 0u, done = 0u;
  int id = lane * EPL, id2 = id;  // their experts
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    if (key[i] > best) {
      second = best;
      id2 = id;
      best = key[i];
      id = lane * EPL + i;
    } else if (key[i] > second) {
      second = key[i];
      id2 = lane * EPL + i;
    }
  }
  if (G > 1 && p.group_lanes != 0) {  // a group is a run of whole lanes
    uint32_t a = best, b = second;
    if (sums && !biased) {
      a = b = 0u;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const uint32_t k = value(i);
        b = max(b, min(a, k));
        a = max(a, k);
      }
    }
    for (int off = 1; off < p.group_lanes; off <<= 1) {
      const uint32_t oa = __shfl_xor_sync(FULL, a, off), ob = __shfl_xor_sync(FULL, b, off);
      b = max(min(a, oa), max(b, ob));
      a = max(a, oa);
    }
    const int member = (int)(((uint32_t)(lane * EPL) * p.recip) >> 20);
    uint32_t mask;
    if (!decide(a, b, member, p.group_lanes, mask)) return false;
    // a lane that is never picked, so its keys are not looked at again
    if (!((mask >> ((member * p.group_lanes) & 31)) & 1u)) best = second = 0u;
  }
  my_e = -1;
  uint32_t my_key = 0u;
  int n = 0;
  auto pick = [&](uint32_t m) {  // m: the warp's best key
    const int e = (int)redux_min(best == m ? (uint32_t)id : 0xFFFFFFFFu);
    if (lane == n) {
      my_e = e;
      my_key = m;
    }
    ++n;
    const bool won = e == id && best == m;
    if (won) {
      done |= 1u << (id % EPL);
      best = second;
      id = id2;
      second = 0u;
    }
    if (EPL > 2 && __any_sync(FULL, won && best == 0u)) {
      if (won) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const uint32_t k = ((done >> i) & 1u) ? 0u : key[i];
          if (k > best) {
            best = k;
            id = lane * EPL + i;
          }
        }
      }
    }
  };
  uint32_t m = redux_max(best);
  while (n < p.top_k && m != 0u) {
    pick(m);
    m = redux_max(best);
  }
  if (biased && m != 0u) {
    // The picks go on as long as they could belong before the last one that
    // counts: candidates beyond are not in reach of fp32's error.
    const float last = ord_value(__shfl_sync(FULL, my_key, n - 1));
    while (n < 32 && m != 0u) {
      const float v = ord_value(m);
      if (last - v > 2.f * err + SUM_ERR * (fabsf(v) + fabsf(last))) break;
      pick(m);
      m = redux_max(best);
    }
    if (n == 32 && m != 0u) {
      // More candidates than lanes.  What is left in reach is in its place behind
      // the picks only where it is the same number as the last one that counts.
      const int le = __shfl_sync(FULL, my_e, p.top_k - 1);
      const float lx = as_f32(row[le]), lb = __ldg(p.bias + le);
      bool other = false;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const float v = ord_value(key[i]);
        if (((done >> i) & 1u) || key[i] == 0u || last - v > 2.f * err + SUM_ERR * (fabsf(v) + fabsf(last))) continue;
        other |= x[i] != lx || __ldg(p.bias + lane * EPL + i) != lb;
      }
      if (__any_sync(FULL, other)) return false;
    }
  }
  if (biased) {
    // Neighbours in the order must be further apart than their errors, unless
    // they are the same number: the same logit with the same bias.
    const float v = ord_value(my_key), nv = __shfl_down_sync(FULL, v, 1);
    const float bias = my_e >= 0 ? __ldg(p.bias + my_e) : 0.f, nb = __shfl_down_sync(FULL, bias, 1);
    const float mx = my_e >= 0 ? as_f32(row[my_e]) : 0.f;  // again, from the L1
    const float nx = __shfl_down_sync(FULL, mx, 1);
    const bool apart = v - nv > 2.f * err + SUM_ERR * (fabsf(v) + fabsf(nv)) || (mx == nx && bias == nb);
    if (!__all_sync(FULL, lane + 1 >= n || apart)) {
      if (n == 32) return false;  // more candidates than lanes
      // the candidates, one a lane, in fp64, and their order
      float top = 0.f;
      double z = 1.0, k = -INFINITY;
      if (p.softmax) {
        float xc[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) xc[i] = x[i];
        softmax_sum_f64<EPL>(xc, top, z);
      }
      if (lane < n) k = score_f64(p, mx, top, z) + (double)bias;
      int rank = 0, first = -1;
      for (int j = 0; j < n; ++j) {
        const double o = __shfl_sync(FULL, k, j);
        const int oe = __shfl_sync(FULL, my_e, j);
        if (o > k || (o == k && oe < my_e)) ++rank;
      }
      for (int j = 0; j < n; ++j) {
        const int r = __shfl_sync(FULL, rank, j), oe = __shfl_sync(FULL, my_e, j);
        if (r == lane) first = oe;
      }
      my_e = lane < n ? first : -1;
    }
    if (lane >= p.top_k) my_e = -1;
  }
  return true;
}

template <int EPL, bool BF16>
__global__ void __launch_bounds__(128) route_kernel(const RouteParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (t >= p.T) return;
  float x[EPL];
  using V = typename std::conditional<BF16, __nv_bfloat16, float>::type;
  const V* row = static_cast<const V*>(p.logits) + (size_t)t * (size_t)p.stride;
  load_experts<EPL>(row, p.wide_loads, lane, p.E, -INFINITY, x);
  int my_e;
  if (!route_row_f32<EPL>(p, x, row, lane, my_e)) {
    float xc[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) xc[i] = x[i];
    int e;
    route_row_f64<EPL>(p, xc, lane, e);
    my_e = e;
  }

  // Weights from the selected logits.  u is the score times a factor common to
  // the row that keeps the largest near 1, so that renormalising never divides
  // by zero, however low the logits are.
  const bool on = my_e >= 0;
  const float xs = on ? as_f32(row[my_e]) : -INFINITY;
  float ref = on ? (p.softmax ? xs : fminf(xs, 0.f)) : -INFINITY;
  if (p.renorm) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ref = fmaxf(ref, __shfl_xor_sync(FULL, ref, off));
  }
  float u = 0.f, den = 1.f;
  if (p.softmax) {
    if (!p.renorm) {
      float m = -INFINITY, z = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) m = x[i] > m ? x[i] : m;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, off));
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (x[i] > -INFINITY) z += x[i] == m ? 1.f : expf(x[i] - m);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(FULL, z, off);
      ref = m;
      den = z;
    }
    if (on) u = xs == ref ? 1.f : expf(xs - ref);
  } else if (on) {
    const float m = fminf(xs, 0.f);
    const float r = p.renorm ? ref : 0.f;
    u = (m == r ? 1.f : expf(m - r)) / (1.f + expf(-fabsf(xs)));
  }
  if (p.renorm) {
    den = u;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) den += __shfl_xor_sync(FULL, den, off);
  }
  if (lane < p.top_k) {
    p.ids[(size_t)t * p.top_k + lane] = my_e;
    p.w[(size_t)t * p.top_k + lane] = on ? p.scale * (u / den) : 0.f;
  }
}

// ---------------------------------------------------------------- grouping
// Stable counting sort of the pairs by expert, in one cluster of CTAs.  Every
// warp owns one stretch of consecutive pairs and a histogram of its own in
// shared memory; the histograms' sums in warp and CTA order (the CTAs read each
// other's totals) give each warp its first place in every expert's range, and a
// second pass over the stretch hands the places out in order.  No atomic
// decides an order, so the result is the same on every call.
//
// Bound by latency and by the scattered stores of the order, one line a lane:
// 49,152 pairs of 256 experts take one CTA 61 us, eight 8.4 us, sixteen 6.2 us; one
// cluster does all, so 2^20 pairs take 66 us.
constexpr int GP_WARPS = 32;
constexpr int GP_CTAS = 16;  // at most: more than the portable 8, within one GPC
constexpr int GP_HELD = 4;

template <int CTAS>  // of the cluster
__global__ void __launch_bounds__(GP_WARPS * 32) group_kernel(const int32_t* __restrict__ ids, int P, int E,
                                                              int32_t* __restrict__ offsets,
                                                              int32_t* __restrict__ order, int32_t* __restrict__ pos) {
  extern __shared__ int hist[];     // [GP_WARPS][E], [E] this CTA's totals, [E + 1] first places, [32] scan
  int* total = hist + GP_WARPS * E;
  int* first = total + E;
  int* scan = first + E + 1;
  uint32_t rank;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < GP_WARPS * E; i += GP_WARPS * 32) hist[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const int stretch = (P + CTAS * GP_WARPS * 32 - 1) / (CTAS * GP_WARPS * 32) * 32;  // pairs of a warp
  const long long lo = (long long)(rank * GP_WARPS + warp) * stretch;
  int* h = hist + warp * E;
  auto id_at = [&](int i) {  // of this lane's pair, -1: none or dropped
    const long long at = lo + i + lane;
    const int id = at < P ? __ldg(ids + at) : -1;
    return id >= 0 && id < E ? id : -1;
  };
  int held[GP_HELD];  // the first ids stay in registers for the second pass
#pragma unroll
  for (int i = 0; i < GP_HELD; ++i) held[i] = 32 * i < stretch ? id_at(32 * i) : -1;
#pragma unroll
  for (int i = 0; i < GP_HELD; ++i)
    if (held[i] >= 0) atomicAdd(&h[held[i]], 1);
  for (int i = 32 * GP_HELD; i < stretch; i += 32) {
    const int id = id_at(i);
    if (id >= 0) atomicAdd(&h[id], 1);
  }
  __syncthreads();
  if (tid < E) {  // exclusive sums over the warps; E <= 1024 threads
    int c[GP_WARPS], sum = 0;
#pragma unroll
    for (int w = 0; w < GP_WARPS; ++w) c[w] = hist[w * E + tid];
#pragma unroll
    for (int w = 0; w < GP_WARPS; ++w) {
      hist[w * E + tid] = sum;
      sum += c[w];
    }
    total[tid] = sum;
  }
  if (CTAS > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
  else __syncthreads();
  // per expert: all pairs, and those of the CTAs before this one
  int all = 0, before = 0;
  if (tid < E) {
    int v[CTAS];
    if (CTAS > 1) {
#pragma unroll
      for (uint32_t r = 0; r < CTAS; ++r) {
        uint32_t a;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(total + tid)), "r"(r));
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v[r]) : "r"(a) : "memory");
      }
    } else {
      v[0] = total[tid];
    }
#pragma unroll
    for (uint32_t r = 0; r < CTAS; ++r) {
      all += v[r];
      if (r < rank) before += v[r];
    }
  }
  // this thread has read the other CTAs' totals; they may leave once all have
  if (CTAS > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  int incl = all;  // inclusive sums over the experts
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(FULL, incl, off);
    if (lane >= off) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int v = scan[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(FULL, v, off);
      if (lane >= off) v += o;
    }
    scan[lane] = v;
  }
  __syncthreads();
  const int base = incl - all + (warp > 0 ? scan[warp - 1] : 0);
  if (tid < E) {
    first[tid] = base + before;
    if (rank == 0) offsets[tid] = base;
  }
  const int kept = scan[GP_WARPS - 1];
  if (tid == 0 && rank == 0) offsets[E] = kept;
  __syncthreads();
  auto hand_out = [&](int i, int id) {
    const long long at = lo + i + lane;
    // lanes with the same id, a ballot for each bit (match.any takes some 65
    // cycles of the SM); a dropped pair's -1 meets nobody that looks
    uint32_t peers = FULL;
    for (int bit = 0; (1 << bit) < E; ++bit) {
      const uint32_t on = __ballot_sync(FULL, (id >> bit) & 1);
      peers &= ((id >> bit) & 1) ? on : ~on;
    }
    peers &= __ballot_sync(FULL, id >= 0);
    int place = -1;
    if (id >= 0) place = first[id] + h[id] + __popc(peers & ((1u << lane) - 1u));
    __syncwarp();
    if (id >= 0 && lane == __ffs(peers) - 1) h[id] += __popc(peers);
    __syncwarp();
    if (at < P) pos[at] = place;
    if (place >= 0) order[place] = (int)at;
  };
#pragma unroll
  for (int i = 0; i < GP_HELD; ++i)
    if (32 * i < stretch) hand_out(32 * i, held[i]);
  for (int i = 32 * GP_HELD; i < stretch; i += 32) hand_out(i, id_at(i));
  for (long long i = kept + (long long)rank * GP_WARPS * 32 + tid; i < P; i += (long long)CTAS * GP_WARPS * 32) order[i] = -1;
  __syncwarp();
  if (CTAS > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int EPL>
cudaError_t launch_route_epl(RouteParams p, bool bf16, cudaStream_t st) {
  const int size = p.E / p.n_groups, lanes = size % EPL == 0 ? size / EPL : 0;
  p.group_lanes = (lanes & (lanes - 1)) == 0 ? lanes : 0;
  p.wide_loads = p.stride * (bf16 ? 2 : 4) % 16 == 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.T + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&cfg, route_kernel<EPL, true>, p)
              : cudaLaunchKernelEx(&cfg, route_kernel<EPL, false>, p);
}

}  // namespace

constexpr int group_smem(int E) { return (GP_WARPS * E + 2 * E + 1 + GP_WARPS) * 4; }

// CTAs that group n_pairs where the device places clusters of up to `most`.  One
// alone saves the exchange with the others (up to two ids a thread); few pairs
// make a cluster's fixed costs count: 8,192 pairs of 64, 256, 1,024 experts 3.9,
// 4.4, 6.3 us in eight, 4.0, 4.7, 8.4 in sixteen; 16,384 of 256 5.1 and 4.9.
static int group_ctas(int n_pairs, int most) {
  const int want = n_pairs <= 2 * GP_WARPS * 32 ? 1 : n_pairs <= 8192 ? 8 : GP_CTAS;
  return want < most ? want : most;
}

static cudaLaunchConfig_t group_config(int ctas, int E, cudaLaunchAttribute (&attr)[2], cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(GP_WARPS * 32);
  cfg.dynamicSmemBytes = (size_t)group_smem(E);
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// Whether the device (it may be a part of one) places clusters of so many.
template <int CTAS>
static bool group_placed() {
  if (CTAS > 8 &&
      cudaFuncSetAttribute(group_kernel<CTAS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return false;
  if (cudaFuncSetAttribute(group_kernel<CTAS>, cudaFuncAttributeMaxDynamicSharedMemorySize, group_smem(ROUTE_MAX_E)) !=
      cudaSuccess)
    return false;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = group_config(CTAS, ROUTE_MAX_E, attr, nullptr);
  int n = 0;
  return cudaOccupancyMaxActiveClusters(&n, group_kernel<CTAS>, &cfg) == cudaSuccess && n > 0;
}

cudaError_t route_kernels_init(int* group_most) {
  *group_most = 1;
  if (group_placed<8>()) *group_most = 8;
  if (*group_most == 8 && group_placed<GP_CTAS>()) *group_most = GP_CTAS;
  if (*group_most < GP_CTAS) (void)cudaGetLastError();  // a size that is not placed is no error of a later call
  return cudaFuncSetAttribute(group_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, group_smem(ROUTE_MAX_E));
}

cudaError_t launch_route(const RouteSpec& r, const void* logits, bool bf16, long long stride, int T, const float* bias,
                         int32_t* ids, float* w, cudaStream_t st) {
  RouteParams p;
  p.logits = logits;
  p.stride = stride;
  p.bias = bias;
  p.ids = ids;
  p.w = w;
  p.T = T;
  p.E = r.E;
  p.top_k = r.top_k;
  p.n_groups = r.n_groups;
  p.top_groups = r.top_groups;
  p.softmax = r.softmax;
  p.top2 = r.top2;
  p.renorm = r.renorm;
  p.scale = r.scale;
  p.recip = (uint32_t)(((1 << 20) + r.E / r.n_groups - 1) / (r.E / r.n_groups));
  if (r.E <= 64) return launch_route_epl<2>(p, bf16, st);
  if (r.E <= 128) return launch_route_epl<4>(p, bf16, st);
  if (r.E <= 256) return launch_route_epl<8>(p, bf16, st);
  if (r.E <= 512) return launch_route_epl<16>(p, bf16, st);
  return launch_route_epl<32>(p, bf16, st);
}

cudaError_t launch_group_pairs(const int32_t* ids, int P, int E, int32_t* offsets, int32_t* order, int32_t* pos,
                               int most, cudaStream_t st) {
  const int ctas = group_ctas(P, most);
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = group_config(ctas, E, attr, st);
  return ctas == 1   ? cudaLaunchKernelEx(&cfg, group_kernel<1>, ids, P, E, offsets, order, pos)
         : ctas == 8 ? cudaLaunchKernelEx(&cfg, group_kernel<8>, ids, P, E, offsets, order, pos)
                     : cudaLaunchKernelEx(&cfg, group_kernel<GP_CTAS>, ids, P, E, offsets, order, pos);
}

}  // namespace flint

// For the tests: the CTAs that group so many pairs where clusters of up to `most` are placed.
extern "C" int flint_group_pairs_ctas(int n_pairs, int most) { return flint::group_ctas(n_pairs, most); }
