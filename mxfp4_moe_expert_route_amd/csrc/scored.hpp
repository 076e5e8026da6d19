// Routing by scores: the rule, and one wave's work on one token.
//
// With l the token's logits and b the bias (optional):
//   s_e = 1 / (1 + exp(-l_e))  or  exp(l_e - max l) / sum_e' exp(l_e' - max l)
//   c_e = s_e + b_e
// An expert is available unless l_e or c_e is NaN or -Inf.  Groups are runs of
// E / groups experts; a group's value is the sum of its `best` (1 or 2)
// largest c among the available, and the `keep` groups of the largest values
// stay (a group without an available expert comes last, the lower index first
// on equal values).  Of their available experts the k with the largest c are
// taken, or with the largest l where there is no bias (s grows with l), the
// lower index first on equal values.  Weights: s_j, or s_j / sum_j' s_j' over
// the taken, times `scale`.  Where fewer than k are available the rest of the
// row is id -1 with weight 0.
//
// Choices are those of 64 bits: c next to 1 saturates in 32, and a choice that a
// rounding decides would differ between two ways to compute the same rule.  But
// 32 bits nearly always settle it.  A wave takes its first k + 2 candidates by
// fp32 values, orders them by their differences (order_of), which do not lose
// what the values lose, and keeps the first k if the last of them is further
// above whatever is no candidate than the values' errors; otherwise it chooses
// again in fp64.  8192 tokens of 384 experts in 8 groups: 10.7 us a wave a token, 7.7
// four tokens a wave (route_scored.hip), 36 in fp64 throughout; what bounds it are
// a wave's instructions.  Of such inputs two in three hold a token that is chosen
// in fp64, which ends the launch 0.5 to 1.5 later, with four tokens a wave 3.5 to 7.
#pragma once
#include "routing.hpp"

namespace mxm {

struct ScoreRule {
  int E, k;
  int groups, keep, best;
  int size;                // experts of a group
  int lanes_log2;          // lanes of a group: 64 / groups rounded up to a power of two
  bool sigmoid, norm;
  float scale;
};

hipError_t launch_route_scored(const float* logits, const float* bias, int T, const ScoreRule& r,
                               int32_t* ids, float* w, hipStream_t s);
// Routing that also counts, for every 32 tokens, how many took each expert (a byte
// an expert, into the grouping's workspace), and the grouping from those counts:
// ranges of 256 pairs, so calls of k = 8, whose workspace has the room.
constexpr int kCountTokens = 32;
constexpr int kCountExperts = 512;
bool route_scored_counts(int T, const ScoreRule& r, const float* logits, const float* bias);
hipError_t launch_route_scored_count(const float* logits, const float* bias, int T,
                                     const ScoreRule& r, int32_t* ids, float* w, uint32_t* bytes,
                                     hipStream_t s);
bool permute_counted_fits(int T, int E);
hipError_t launch_permute_counted(const int32_t* ids, int T, int E, int k, const uint32_t* bytes,
                                  int32_t* counts, int32_t* offsets, int32_t* sorted_pairs,
                                  int32_t* pair_to_row, hipStream_t s);
// routing and grouping in one workgroup, where it fits
bool route_scored_fusable(int T, const ScoreRule& r);
hipError_t launch_route_scored_permute(const float* logits, const float* bias, int T,
                                       const ScoreRule& r, int32_t* ids, float* w,
                                       int32_t* counts, int32_t* offsets, int32_t* sorted_pairs,
                                       int32_t* pair_to_row, hipStream_t s);

namespace {

__device__ __forceinline__ uint64_t order_key64(double v) {
  const uint64_t u = uint64_t(__double_as_longlong(v + 0.0));     // -0.0 ties with +0.0
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ double max_f64(double a, double b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  auto up = [&](int x) { v = max(v, uint32_t(x)); };
  up(__builtin_amdgcn_update_dpp(0, int(v), 0x111, 0xf, 0xf, true));   // row_shr:1
  up(__builtin_amdgcn_update_dpp(0, int(v), 0x112, 0xf, 0xf, true));   // row_shr:2
  up(__builtin_amdgcn_update_dpp(0, int(v), 0x114, 0xf, 0xf, true));   // row_shr:4
  up(__builtin_amdgcn_update_dpp(0, int(v), 0x118, 0xf, 0xf, true));   // row_shr:8
  up(__builtin_amdgcn_update_dpp(0, int(v), 0x142, 0xa, 0xf, true));   // row_bcast:15
  up(__builtin_amdgcn_update_dpp(0, int(v), 0x143, 0xc, 0xf, true));   // row_bcast:31
  return uint32_t(__builtin_amdgcn_readlane(int(v), kWave - 1));
}

// Sum over the wave in fp64, in the order of wave_sum_f32.
__device__ __forceinline__ double wave_sum_f64(double v) {
  auto add = [&](uint64_t x) { v += __longlong_as_double((long long)x); };
  add(dpp_u64<0x111, 0xf>(uint64_t(__double_as_longlong(v))));
  add(dpp_u64<0x112, 0xf>(uint64_t(__double_as_longlong(v))));
  add(dpp_u64<0x114, 0xf>(uint64_t(__double_as_longlong(v))));
  add(dpp_u64<0x118, 0xf>(uint64_t(__double_as_longlong(v))));
  add(dpp_u64<0x142, 0xa>(uint64_t(__double_as_longlong(v))));
  add(dpp_u64<0x143, 0xc>(uint64_t(__double_as_longlong(v))));
  const uint64_t u = uint64_t(__double_as_longlong(v));
  const uint32_t lo = __builtin_amdgcn_readlane(int(uint32_t(u)), kWave - 1);
  const uint32_t hi = __builtin_amdgcn_readlane(int(uint32_t(u >> 32)), kWave - 1);
  return __longlong_as_double((long long)((uint64_t(hi) << 32) | lo));
}

// v of lane ^ D where the lanes of each run of D already agree (D = 4 and 8
// mirror a run of 2 D)
template <int D>
__device__ __forceinline__ float across(float v) {
  if constexpr (D == 1) return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xb1, 0xf, 0xf, true));
  if constexpr (D == 2) return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4e, 0xf, 0xf, true));
  if constexpr (D == 4) return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xf, 0xf, true));
  if constexpr (D == 8) return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xf, 0xf, true));
  return __shfl_xor(v, D);
}

// exp(x) for x <= 0 to 2^-22, relative: the argument's product and its whole
// part in fp64, so that its size does not count.  Below fp32's range 0.
__device__ __forceinline__ float exp_down(double x) {
  const double t = x * 1.4426950408889634;
  const double n = rint(t);
  const float e = __builtin_ldexpf(__builtin_amdgcn_exp2f(float(t - n)), x > -120.0 ? int(n) : 0);
  return x > -120.0 ? e : 0.f;
}

__device__ __forceinline__ float lane_f32(float v, int src) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), src));
}

// Where a lane's experts are: lane (g << lanes_log2) + m holds the experts m,
// m + lanes, ... of group g, at most NPER of them, so a group's largest values
// meet in log2(lanes) steps for all groups at once.
struct ScorePlace {
  int lane, lanes, g, m;
  int e0;                                         // slot i holds expert e0 + lanes * i
  __device__ explicit ScorePlace(const ScoreRule& r)
      : lane(lane_id()), lanes(1 << r.lanes_log2), g(lane >> r.lanes_log2), m(lane & (lanes - 1)),
        e0(g * r.size + m) {}
};

__device__ __forceinline__ double lane_f64(double v, int src) {
  const uint64_t u = uint64_t(__double_as_longlong(v));
  const uint32_t lo = __builtin_amdgcn_readlane(int(uint32_t(u)), src);
  const uint32_t hi = __builtin_amdgcn_readlane(int(uint32_t(u >> 32)), src);
  return __longlong_as_double((long long)((uint64_t(hi) << 32) | lo));
}

// exp(l - top), and 1 at the top, be it infinite
__device__ __forceinline__ double exp_f64(float l, float top) {
  return exp(l == top ? 0.0 : double(l) - double(top));
}

__device__ __forceinline__ double score_f64(float l, float top, double total, bool sigmoid) {
  return sigmoid ? 1.0 / (1.0 + exp(-double(l))) : exp_f64(l, top) / total;
}

// The softmax's sum; one exponential at a time, for few registers.
template <int NPER>
__device__ __forceinline__ double total_f64(const float (&v)[NPER], float top) {
  double total = 0.0;
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const double e = exp_f64(v[i], top);
    total += v[i] > -__builtin_inff() ? e : 0.0;
    __builtin_amdgcn_sched_barrier(0);
  }
  return wave_sum_f64(total);
}

// The values c in fp64, -inf where an expert is not available.  v is NaN in
// slots without an expert, top the row's largest logit.
template <int NPER>
__device__ __forceinline__ void values_f64(const float (&v)[NPER], const float (&b)[NPER],
                                           float top, bool sigmoid, double (&c)[NPER]) {
  const double none = -__builtin_inf();
  double total = 1.0;
  if (!sigmoid) total = total_f64<NPER>(v, top);
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const double x = score_f64(v[i], top, total, sigmoid) + double(b[i]);
    c[i] = double(v[i]) > none && x > none ? x : none;
    if (i % 2) __builtin_amdgcn_sched_barrier(0);
  }
}

// Whether the lane's group stays, by values in fp64.
template <int NPER>
__device__ __forceinline__ bool keep_f64(const double (&c)[NPER], const ScoreRule& r,
                                         const ScorePlace& at) {
  const double none = -__builtin_inf();
  double a1 = none, a2 = none;                    // the two largest of the group
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    a2 = c[i] > a1 ? a1 : max_f64(a2, c[i]);
    a1 = max_f64(a1, c[i]);
  }
  for (int d = 1; d < at.lanes; d <<= 1) {
    const double o1 = __shfl_xor(a1, d), o2 = __shfl_xor(a2, d);
    a2 = o1 > a1 ? max_f64(a1, o2) : max_f64(a2, o1);
    a1 = max_f64(a1, o1);
  }
  const double value = r.best == 2 && a2 > none ? a1 + a2 : a1;
  int before = 0;
  for (int j = 0; j < r.groups; ++j) {
    const double o = lane_f64(value, j << r.lanes_log2);
    before += o > value || (o == value && j < at.g);
  }
  return before < r.keep;
}

// The choice in fp64; lanes 0..k-1 end with the j-th id, or -1.
template <int NPER>
__device__ __forceinline__ int choose_f64(const float (&v)[NPER], const float (&b)[NPER],
                                          bool biased, float top, const ScoreRule& r,
                                          const ScorePlace& at) {
  const double none = -__builtin_inf();
  double c[NPER];
  values_f64(v, b, top, r.sigmoid, c);
  const bool kept = r.groups == 1 || keep_f64(c, r, at);
  uint64_t key[NPER];
#pragma unroll
  for (int i = 0; i < NPER; ++i)
    key[i] = kept && c[i] > none ? order_key64(biased ? c[i] : double(v[i])) : 0ull;
  int my_id = -1;
  for (int j = 0; j < r.k; ++j) {
    uint64_t mine = key[0];
    int e = at.e0;
#pragma unroll
    for (int i = 1; i < NPER; ++i)
      if (key[i] > mine) mine = key[i], e = at.e0 + at.lanes * i;
    const uint64_t best = wave_max_u64(mine);
    if (best == 0ull) break;                      // no available expert is left
    const unsigned long long owners = __ballot(mine == best);
    int first;
    if (__popcll(owners) == 1) {
      first = __builtin_amdgcn_readlane(e, __ffsll((long long)owners) - 1);
    } else {
      first = mine == best ? e : 0x7fffffff;
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) first = min(first, __shfl_xor(first, d));
    }
#pragma unroll
    for (int i = 0; i < NPER; ++i)
      if (at.e0 + at.lanes * i == first && mine == best) key[i] = 0ull;
    if (at.lane == j) my_id = first;
  }
  return my_id;
}

// Descending order of N values by a fixed network (odd-even merges of the next
// power of two, without the places past N).
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&key)[N]) {
  constexpr int P = N <= 2 ? 2 : N <= 4 ? 4 : N <= 8 ? 8 : N <= 16 ? 16 : 32;
#pragma unroll
  for (int p = 1; p < P; p *= 2)
#pragma unroll
    for (int d = p; d >= 1; d /= 2)
#pragma unroll
      for (int j = d % p; j + d < P; j += 2 * d)
#pragma unroll
        for (int i = 0; i < d; ++i) {
          const int x = i + j, y = i + j + d;
          if (y < N && x / (2 * p) == y / (2 * p)) {
            const uint32_t hi = max(key[x], key[y]), lo = min(key[x], key[y]);
            key[x] = hi;
            key[y] = lo;
          }
        }
}

// The score of a pick to 2^-21 (softmax: and the error of the sum), and for a
// sigmoid u = 1 - s as exactly.
__device__ __forceinline__ float pick_score(float l, float top, float inv, bool sigmoid, float& u) {
  if (!sigmoid) return exp_down(l == top ? 0.0 : double(l) - double(top)) * inv;
  const float q = exp_down(-fabs(double(l)));
  const float a = __builtin_amdgcn_rcpf(1.f + q), b = q * a;
  u = l < 0.f ? a : b;
  return l < 0.f ? b : a;
}

__device__ __forceinline__ float lane_above(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x130, 0xf, 0xf, true));   // wave_shl:1
}

// Whether this lane's pick comes before the next lane's: 1, -1, or 0 where fp32
// does not tell.  With h the larger logit of the two and d their distance
//   sigmoid(h) - sigmoid(h - d) = s(h) u(h - d) (1 - exp(-d)),
//   softmax the same without u,
// a product of factors known however close the two scores are.  Its error, relative,
// in units of 2^-24: of an exponential 2.2 (its instruction 2, its argument 0.2), of
// 1/(1+q) 4.1 at most and of q/(1+q) 5.2 (the exponential's, a sum's 1, the
// reciprocal's 2, a product's 1; a score and a u are never both of the second form);
// of 1 - exp(-d) 7.6 at most: d's rounding 1, the series' last steps 2.3 and its
// rest d^8 / 8! 4.3, or 4.9 by the exponential; two products 2.  Together 19, and
// 24 are taken.  Softmax: the sum's 56 (below) in the place of a reciprocal's, 68
// together, and 128 are taken.  All lanes call it: a lane reads its neighbour's
// registers.
__device__ __forceinline__ int order_of(float l, float b, int id, float s, float u, bool biased,
                                        bool sigmoid) {
  const float nl = lane_above(l), nb = lane_above(b), ns = lane_above(s), nu = lane_above(u);
  const int ni = __float_as_int(lane_above(__int_as_float(id)));
  const int by_id = id < ni ? 1 : -1;
  if (!biased) return l > nl ? 1 : l < nl ? -1 : l == nl ? by_id : 0;
  const bool up = l >= nl;
  const float d = fabsf(l - nl);
  float t = 1.f - d * (1.f / 7.f);                // 1 - exp(-d), below 1/2 by its series
  t = 1.f - d * (1.f / 6.f) * t;
  t = 1.f - d * (1.f / 5.f) * t;
  t = 1.f - d * (1.f / 4.f) * t;
  t = 1.f - d * (1.f / 3.f) * t;
  t = d * (1.f - d * 0.5f * t);
  if (!(d < 0.5f)) t = 1.f - __builtin_amdgcn_exp2f(d * -1.4426950408889634f);
  float ds = (up ? s : ns) * t;
  if (sigmoid) ds *= up ? nu : u;
  const float db = b - nb;
  // values that fp64 does not tell apart are equal: left to it, as are scores that
  // fp32 holds with few digits
  const float err = (sigmoid ? 0x1.8p-20f : 0x1p-17f) * ds + 0x1p-22f * fabsf(db) +
                    0x1p-51f * (fabsf(s) + fabsf(b)) + 0x1p-140f;
  const float x = (up ? ds : -ds) + db;
  if (l == nl && b == nb) return by_id;
  return x > err ? 1 : x < -err ? -1 : 0;
}

// One token by one whole wave; lanes 0..k-1 end with the j-th choice and its
// weight.
template <int NPER>
__device__ __forceinline__ void score_token(const float* __restrict__ row,
                                            const float* __restrict__ bias, const ScoreRule& r,
                                            int& my_id, float& my_w) {
  constexpr int SB = NPER <= 2 ? 1 : NPER <= 4 ? 2 : NPER <= 8 ? 3 : NPER <= 16 ? 4 : 5;
  constexpr uint32_t kSlots = (1u << SB) - 1u;
  const float none = -__builtin_inff();
  const ScorePlace at(r);
  float v[NPER], b[NPER];
  const int held = at.g < r.groups ? (r.size - at.m + at.lanes - 1) >> r.lanes_log2 : 0;
  int place[NPER];
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    place[i] = min(at.e0 + (i << r.lanes_log2), r.E - 1);
    v[i] = row[place[i]];
    b[i] = 0.f;
  }
  if (bias) {
#pragma unroll
    for (int i = 0; i < NPER; ++i) b[i] = bias[place[i]];
  }
#pragma unroll
  for (int i = 0; i < NPER; ++i) v[i] = i < held ? v[i] : __builtin_nanf("");
  // fp32 values and a bound on the scores' error
  float top = none, total = 1.f, inv = 1.f;
  if (!r.sigmoid) {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      const uint32_t o = order_key(v[i]);         // of NaN: -inf's
      t = max(t, o);
    }
    t = wave_max_u32(t);
    top = key_value(t);
  }
  const bool scored = bias || r.groups > 1;       // else logits decide
  float c[NPER], ds = 0.f;
  if (r.sigmoid) {
    // |error| of s: s (1 - s) (1.25 2^-24 |l| + 2^-23) of the exponential, whose
    // instruction is off by a unit in the last place, and 1.5 2^-23 s of the sum
    // and the reciprocal, a unit too: below 1.9 2^-23 in all
    ds = 0x1p-22f;
#pragma unroll
    for (int i = 0; i < NPER; ++i)
      c[i] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v[i] * -1.4426950408889634f));
  } else if (r.norm && scored) {
    // with d = l - top, of exp(d): 2^-23 (|d| + 1) relative, so at most 2^-23 in
    // all; of the sum: 2^-23 (1 + the mean of |d| by weight, at most ln E, and half
    // of its 38 additions), 56 units of 2^-24 with the reciprocal's; of each s at
    // most 2^-23 (3 + 7 + 19) / total
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      const float d = v[i] == top ? 0.f : v[i] - top;
      const float e = __builtin_amdgcn_exp2f(d * 1.4426950408889634f);
      c[i] = v[i] > none ? e : 0.f;
      sum += c[i];
    }
    inv = __builtin_amdgcn_rcpf(wave_sum_f32(sum));
    ds = 0x1p-18f * inv;
#pragma unroll
    for (int i = 0; i < NPER; ++i) c[i] *= inv;
  } else if (!r.norm) {
    double sum = 0.0;                             // the weights' divisor too
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      const float e = exp_down(v[i] == top ? 0.0 : double(v[i]) - double(top));
      c[i] = v[i] > none ? e : 0.f;
      sum += double(c[i]);
    }
    total = float(wave_sum_f64(sum));
    inv = __builtin_amdgcn_rcpf(total);
    ds = 0x1p-20f * inv;
#pragma unroll
    for (int i = 0; i < NPER; ++i) c[i] *= inv;
  } else {
#pragma unroll
    for (int i = 0; i < NPER; ++i) c[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const float x = fmaxf(c[i] + b[i], none);     // NaN: none
    c[i] = v[i] > none ? x : none;
  }
  bool kept = true;
  if (r.groups > 1) {
    float a1 = none, a2 = none;                   // the two largest of the group
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      a2 = fmaxf(a2, fminf(a1, c[i]));
      a1 = fmaxf(a1, c[i]);
    }
    auto meet = [&](float o1, float o2) {
      a2 = fmaxf(fminf(a1, o1), fmaxf(a2, o2));
      a1 = fmaxf(a1, o1);
    };
    if (r.lanes_log2 > 0) meet(across<1>(a1), across<1>(a2));
    if (r.lanes_log2 > 1) meet(across<2>(a1), across<2>(a2));
    if (r.lanes_log2 > 2) meet(across<4>(a1), across<4>(a2));
    if (r.lanes_log2 > 3) meet(across<8>(a1), across<8>(a2));
    if (r.lanes_log2 > 4) meet(across<16>(a1), across<16>(a2));
    const bool two = r.best == 2 && a2 > none;
    const float value = two ? a1 + a2 : a1;
    // three roundings of 2^-24: the sums with the bias, the value, and lo and hi
    const float err = 2.f * ds + 0x1.8p-23f * (fabsf(a1) + (two ? fabsf(a2) : 0.f));
    const float lo = a1 > none ? value - err : none, hi = a1 > none ? value + err : none;
    int surely = 0, maybe = 0;                    // groups before this one
    for (int j = 0; j < r.groups; ++j) {
      surely += lane_f32(lo, j << r.lanes_log2) > hi;
      maybe += !(lane_f32(hi, j << r.lanes_log2) < lo);          // itself among them
    }
    kept = surely < r.keep;
    if (__any(kept && maybe - 1 >= r.keep && a1 > none)) {
      double x[NPER];
      values_f64(v, b, top, r.sigmoid, x);
      kept = keep_f64(x, r, at);
    }
  }
  // keys: the value's order image, its lowest bits the slot
  uint32_t key[NPER];
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    // no NaN and no -0 where available
    const uint32_t u = __float_as_uint(bias ? c[i] : v[i] + 0.f);
    const uint32_t image = u ^ (uint32_t(int(u) >> 31) | 0x80000000u);
    key[i] = kept && c[i] > none ? (image & ~kSlots) | (kSlots - i) : 0u;
  }
  sort_down(key);
  int my_key = 0, my_src = 0, found = 0;
  bool all = false;                               // every key of the wave is taken
  auto take = [&](int upto) {
    while (found < upto) {
      const uint32_t best = wave_max_u32(key[0]);
      if (best == 0u) {
        all = true;
        break;
      }
      const int src = __ffsll((long long)__ballot(key[0] == best)) - 1;
      if (at.lane == found) my_key = int(best), my_src = src;
      if (at.lane == src) {
#pragma unroll
        for (int i = 0; i + 1 < NPER; ++i) key[i] = key[i + 1];
        key[NPER - 1] = 0u;
      }
      ++found;
    }
  };
  auto id_of = [&]() {
    return !my_key ? -1
                   : (my_src >> r.lanes_log2) * r.size + (my_src & (at.lanes - 1)) +
                         (int(kSlots - (uint32_t(my_key) & kSlots)) << r.lanes_log2);
  };
  take(r.k + 2);                                  // and the two that are left first
  my_id = id_of();
  float l = row[max(my_id, 0)];
  float mb = bias ? bias[max(my_id, 0)] : 0.f;
  bool doubt = false;
  // the candidates' order by their differences, which fp32 has far more
  // exactly than the values; neighbours that stand the wrong way change places
  bool settled = false;
  float s = 0.f;
  for (int pass = 0; pass < 4 && !settled; ++pass) {
    float u = 1.f;
    if (bias) s = pick_score(l, top, inv, r.sigmoid, u);
    int way = order_of(l, mb, my_id, s, u, bias != nullptr, r.sigmoid);
    way = at.lane + 1 < found ? way : 1;
    if (__any(way == 0)) break;
    const unsigned long long bad = __ballot(way < 0);
    settled = bad == 0ull;
    if (!settled) {                             // of a run of wrong pairs the first
      const unsigned long long first = bad & ~(bad << 1);
      const int from = at.lane + int(first >> at.lane & 1) - int(first << 1 >> at.lane & 1);
      l = __shfl(l, from);
      mb = __shfl(mb, from);
      my_id = __shfl(my_id, from);
    }
  }
  doubt = !settled;
  // and whatever is no candidate has at most the last one's key
  if (settled && !all && found > r.k) {
    const float left = key_value(uint32_t(__builtin_amdgcn_readlane(my_key, found - 1)) | kSlots);
    const float x = bias ? lane_f32(s, r.k - 1) + lane_f32(mb, r.k - 1) : lane_f32(l, r.k - 1);
    const float err = bias ? 2.f * ds + 0x1p-22f * (fabsf(left) + fabsf(x)) : 0.f;
    doubt = !(x - left > err);
  }
  if (doubt) {
    my_id = choose_f64<NPER>(v, b, bias != nullptr, top, r, at);
    l = row[max(my_id, 0)];
  }
  // weights: renormalised ones are relative to the largest score, so that they
  // hold where every s underflows
  const bool has = at.lane < r.k && my_id >= 0;
  float p;
  if (r.sigmoid) {
    const float q = exp_down(-fabs(double(l)));
    float up = l < 0.f ? q : 1.f;
    if (r.norm) {
      const uint32_t most = wave_max_u32(has ? order_key(l) : 0u);
      const float lm = most ? key_value(most) : 0.f;
      if (lm < 0.f) up = l < lm ? exp_down(double(l) - double(lm)) : 1.f;
    }
    p = up / (1.f + q);
  } else if (r.norm) {
    const uint32_t most = wave_max_u32(has ? order_key(l) : 0u);
    const float lm = key_value(most);
    p = l == lm ? 1.f : exp_down(double(l) - double(lm));
  } else {
    p = (l == top ? 1.f : exp_down(double(l) - double(top))) / total;
  }
  p = has ? p : 0.f;
  if (r.norm) p /= wave_sum_f32(p);
  my_w = has ? p * r.scale : 0.f;
}

}  // namespace
}  // namespace mxm
