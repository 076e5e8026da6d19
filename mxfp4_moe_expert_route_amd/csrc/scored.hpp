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
// Choices compare values of 64 bits: c next to 1 saturates in 32, and a choice
// that a rounding decides would differ between two ways to compute the same
// rule.
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
// routing and grouping in one workgroup: T <= 16
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

__device__ __forceinline__ double wave_max_f64(double v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v = max_f64(v, __shfl_xor(v, d));
  return v;
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }

// One token by one whole wave.  Lane (g << lanes_log2) + m holds the experts
// m, m + lanes, ... of group g, at most NPER of them, so a group's largest
// values meet in log2(lanes) steps for all groups at once.  Lanes 0..k-1 end
// with the j-th choice and its weight.
template <int NPER>
__device__ __forceinline__ void score_token(const float* __restrict__ row,
                                            const float* __restrict__ bias, const ScoreRule& r,
                                            int& my_id, float& my_w) {
  const double none = -__builtin_inf();
  const int lane = lane_id();
  const int lanes = 1 << r.lanes_log2;
  const int g = lane >> r.lanes_log2, m = lane & (lanes - 1);
  const int e0 = g * r.size + m;                  // slot i holds expert e0 + lanes * i
  float v[NPER], b[NPER];
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const bool in = g < r.groups && m + lanes * i < r.size;
    v[i] = row[in ? e0 + lanes * i : 0];
    b[i] = bias ? bias[in ? e0 + lanes * i : 0] : 0.f;
    if (!in) v[i] = __builtin_nanf("");
  }
  // scores; c[i] = -inf: not available
  double c[NPER];
  double top = none, total = 0.0;
#pragma unroll
  for (int i = 0; i < NPER; ++i) top = v[i] > top ? double(v[i]) : top;
  top = wave_max_f64(top);
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const double l = v[i];
    const double s = r.sigmoid ? sigmoid64(l) : (l == top ? 1.0 : exp(l - top));
    c[i] = l > none ? s : 0.0;
    total += c[i];
  }
  total = wave_sum_f64(total);
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    c[i] = (r.sigmoid ? c[i] : c[i] / total) + double(b[i]);
    if (!(v[i] > none) || !(c[i] > none)) c[i] = none;
  }
  bool kept = g < r.groups;
  if (r.groups > 1) {
    double a1 = none, a2 = none;                  // the two largest of the group
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      a2 = c[i] > a1 ? a1 : max_f64(a2, c[i]);
      a1 = max_f64(a1, c[i]);
    }
    for (int d = 1; d < lanes; d <<= 1) {
      const double o1 = __shfl_xor(a1, d), o2 = __shfl_xor(a2, d);
      a2 = o1 > a1 ? max_f64(a1, o2) : max_f64(a2, o1);
      a1 = max_f64(a1, o1);
    }
    const double value = r.best == 2 && a2 > none ? a1 + a2 : a1;
    int before = 0;
    for (int j = 0; j < r.groups; ++j) {
      const double o = __shfl(value, j << r.lanes_log2);
      before += o > value || (o == value && j < g);
    }
    kept = kept && before < r.keep;
  }
  uint64_t key[NPER];
#pragma unroll
  for (int i = 0; i < NPER; ++i)
    key[i] = kept && c[i] > none ? order_key64(bias ? c[i] : double(v[i])) : 0ull;
  my_id = -1;
  float my_l = 0.f;
  int taken = 0;
  for (int j = 0; j < r.k; ++j) {
    uint64_t mine = key[0];
    int e = e0;
    float l = v[0];
#pragma unroll
    for (int i = 1; i < NPER; ++i)
      if (key[i] > mine) mine = key[i], e = e0 + lanes * i, l = v[i];
    const uint64_t best = wave_max_u64(mine);
    if (best == 0ull) break;                      // no available expert is left
    int first = mine == best ? e : 0x7fffffff;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) first = min(first, __shfl_xor(first, d));
    const unsigned long long owner = __ballot(mine == best && e == first);
    const float chosen = __shfl(l, __ffsll((long long)owner) - 1);
#pragma unroll
    for (int i = 0; i < NPER; ++i)
      if (e0 + lanes * i == first && key[i] == best) key[i] = 0ull;
    if (lane == j) my_id = first, my_l = chosen;
    ++taken;
  }
  // weights: renormalised ones are a softmax of log s over the taken, so that
  // they hold where every s underflows
  const bool has = lane < taken;
  const double l = my_l;
  double p;
  if (r.norm) {
    const double z = !has ? none : r.sigmoid ? fmin(l, 0.0) - log1p(exp(-fabs(l))) : l;
    const double zm = wave_max_f64(z);
    p = !has ? 0.0 : z == zm ? 1.0 : exp(z - zm);
    const double sum = wave_sum_f64(p);
    p = has ? p / sum : 0.0;
  } else {
    p = !has ? 0.0 : r.sigmoid ? sigmoid64(l) : (l == top ? 1.0 : exp(l - top)) / total;
  }
  my_w = float(p * double(r.scale));
}

}  // namespace
}  // namespace mxm
