// Routing by scores, alone and with the grouping of pairs by expert.  The rule
// and a wave's work on a token are in scored.hpp.
#include "scored.hpp"

namespace mxm {
namespace {

constexpr int kFusedWaves = 16;

template <int NPER>
__global__ __launch_bounds__(256) void k_route_scored(const float* __restrict__ logits,
                                                      const float* __restrict__ bias, int T,
                                                      ScoreRule r, int32_t* __restrict__ ids,
                                                      float* __restrict__ w) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;                                      // whole wave leaves together
  const int lane = lane_id();
  int my_id;
  float my_w;
  score_token<NPER>(logits + int64_t(t) * r.E, bias, r, my_id, my_w);
  if (lane < r.k) {
    ids[int64_t(t) * r.k + lane] = my_id;
    w[int64_t(t) * r.k + lane] = my_w;
  }
}

// Small batches: wave t routes token t, then the workgroup groups the pairs
// from the experts' token masks.  One launch and one round trip to memory fewer.
template <int NPER>
__global__ __launch_bounds__(kFusedWaves * kWave) void k_route_scored_permute(
    const float* __restrict__ logits, const float* __restrict__ bias, int T, ScoreRule r,
    int32_t* __restrict__ ids, float* __restrict__ w, int32_t* __restrict__ counts,
    int32_t* __restrict__ offsets, int32_t* __restrict__ sorted_pairs,
    int32_t* __restrict__ pair_to_row) {
  extern __shared__ int32_t smem[];               // mask [E], offsets [E + 1], ids [T k]
  __shared__ int32_t wave_sum[kFusedWaves];
  uint32_t* mask = reinterpret_cast<uint32_t*>(smem);
  int32_t* off_lds = smem + r.E;
  int32_t* lds_ids = smem + 2 * r.E + 1;
  for (int e = threadIdx.x; e < r.E; e += kFusedWaves * kWave) mask[e] = 0u;
  __syncthreads();
  const int t = threadIdx.x >> 6;
  const int lane = lane_id();
  if (t < T) {
    int my_id;
    float my_w;
    score_token<NPER>(logits + int64_t(t) * r.E, bias, r, my_id, my_w);
    if (lane < r.k) {
      ids[int64_t(t) * r.k + lane] = my_id;
      w[int64_t(t) * r.k + lane] = my_w;
      lds_ids[t * r.k + lane] = my_id;
      if (my_id >= 0) atomicOr(&mask[my_id], 1u << t);
    }
  }
  __syncthreads();
  group_small<kFusedWaves, true>(lds_ids, mask, T * r.k, r.E, r.k, counts, offsets, off_lds,
                                 sorted_pairs, pair_to_row, nullptr, nullptr, wave_sum);
}

// ---- four tokens a wave ------------------------------------------------------
//
// A wave a token spends most of its instructions on reductions that carry one
// value a lane.  With a row of 16 lanes a token they serve four tokens, and a
// reduction is four rotations that end in every lane.  The steps are those of
// score_token; a token that needs fp64, has fewer than k + 2 available experts or
// takes more than eight from one lane is left to it.
constexpr int kRowTokens = 4;                    // tokens a wave
constexpr int kRowPicks = 8;                     // largest k

template <int N>
__device__ __forceinline__ int row_ror(int v) {
  return __builtin_amdgcn_update_dpp(0, v, 0x120 + N, 0xf, 0xf, false);
}
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v) {
  v = max(v, uint32_t(row_ror<8>(int(v))));
  v = max(v, uint32_t(row_ror<4>(int(v))));
  v = max(v, uint32_t(row_ror<2>(int(v))));
  return max(v, uint32_t(row_ror<1>(int(v))));
}
__device__ __forceinline__ float row_sum_f32(float v) {
  v += __int_as_float(row_ror<8>(__float_as_int(v)));
  v += __int_as_float(row_ror<4>(__float_as_int(v)));
  v += __int_as_float(row_ror<2>(__float_as_int(v)));
  return v + __int_as_float(row_ror<1>(__float_as_int(v)));
}

// f(N) for the rotations N = 1 .. 15
template <int N = 1, class F>
__device__ __forceinline__ void rotations(F f) {
  f(std::integral_constant<int, N>());
  if constexpr (N < 15) rotations<N + 1>(f);
}

// a: the eight largest of a and b, both in descending order
__device__ __forceinline__ void merge_top8(uint32_t (&a)[8], const uint32_t* b) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = max(a[i], b[7 - i]);
#pragma unroll
  for (int d = 4; d >= 1; d /= 2)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & d)) {
        const uint32_t hi = max(a[i], a[i + d]), lo = min(a[i], a[i + d]);
        a[i] = hi;
        a[i + d] = lo;
      }
}

// lane (g << l2) + m of a row of 16 holds the experts 4 (m + (i << l2)) .. + 3 of
// group g, i = 0 .. NP / 4 - 1
template <int NP>
__device__ __forceinline__ void score_rows(const float* __restrict__ logits,
                                           const float* __restrict__ bias, int T, int t0,
                                           const ScoreRule& r, int32_t* __restrict__ ids,
                                           float* __restrict__ w, int32_t* hist) {
  constexpr int NV = NP / 4;
  constexpr uint32_t kSlots = 31;
  const float none = -__builtin_inff();
  const int lane = lane_id(), q = lane & 15;
  const int t = t0 + (lane >> 4);
  const float* row = logits + int64_t(min(t, T - 1)) * r.E;
  const int l2 = r.lanes_log2 - 2;
  const int g = q >> l2, m = q & ((1 << l2) - 1);
  const int e0 = g * r.size + 4 * m;
  float v[NP], c[NP];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(row + min(e0 + (i << (l2 + 2)), r.E - 4));
    const bool in = g < r.groups && 4 * (m + (i << l2)) < r.size;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * i + j] = in ? x[j] : none;
  }
  const bool scored = bias || r.groups > 1;
  float top = none, total = 1.f, ds = 0x1p-22f;
  if (!r.sigmoid) {
    uint32_t x = 0;
#pragma unroll
    for (int i = 0; i < NP; ++i) x = max(x, order_key(v[i]));
    top = key_value(row_max_u32(x));
  }
  if (r.sigmoid) {
#pragma unroll
    for (int i = 0; i < NP; ++i)
      c[i] = scored ? __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v[i] * -1.4426950408889634f)) : 0.f;
  } else {
    // the sum's 24 to 32 terms a lane and four rotations: below score_token's bound
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float d = v[i] == top ? 0.f : v[i] - top;
      const float e = __builtin_amdgcn_exp2f(d * 1.4426950408889634f);
      c[i] = v[i] > none ? e : 0.f;
      sum += c[i];
    }
    total = row_sum_f32(sum);
    const float inv = __builtin_amdgcn_rcpf(total);
    if (!r.norm) {                               // the weights' divisor, more exactly
      float more = 0.f;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float e = exp_down(v[i] == top ? 0.0 : double(v[i]) - double(top));
        more += v[i] > none ? e : 0.f;
      }
      total = row_sum_f32(more);
    }
    ds = 0x1p-18f * inv;
#pragma unroll
    for (int i = 0; i < NP; ++i) c[i] *= inv;
  }
  if (bias) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(bias + min(e0 + (i << (l2 + 2)), r.E - 4));
#pragma unroll
      for (int j = 0; j < 4; ++j) c[4 * i + j] = fmaxf(c[4 * i + j] + x[j], none);
    }
  }
#pragma unroll
  for (int i = 0; i < NP; ++i) c[i] = v[i] > none ? c[i] : none;
  bool kept = true, doubt = false;
  if (r.groups > 1) {
    float a1 = none, a2 = none;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      a2 = __builtin_amdgcn_fmed3f(a1, a2, c[i]);
      a1 = fmaxf(a1, c[i]);
    }
    auto meet = [&](float o1, float o2) {
      a2 = fmaxf(fminf(a1, o1), fmaxf(a2, o2));
      a1 = fmaxf(a1, o1);
    };
    if (l2 > 0) meet(across<1>(a1), across<1>(a2));
    if (l2 > 1) meet(across<2>(a1), across<2>(a2));
    if (l2 > 2) meet(across<4>(a1), across<4>(a2));
    const bool two = r.best == 2 && a2 > none;
    const float value = two ? a1 + a2 : a1;
    const float err = 2.f * ds + 0x1.8p-23f * (fabsf(a1) + (two ? fabsf(a2) : 0.f));
    const float lo = a1 > none ? value - err : none, hi = a1 > none ? value + err : none;
    int surely = 0, maybe = 0;                   // groups before this one
    rotations([&](auto n) {
      if ((decltype(n)::value & ((1 << l2) - 1)) == 0) {
        surely += __int_as_float(row_ror<decltype(n)::value>(__float_as_int(lo))) > hi;
        maybe += !(__int_as_float(row_ror<decltype(n)::value>(__float_as_int(hi))) < lo);
      }
    });
    kept = surely < r.keep;
    doubt = kept && maybe >= r.keep && a1 > none;
  }
  uint32_t a[8], key[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const uint32_t u = __float_as_uint(bias ? c[i] : v[i] + 0.f);
    const uint32_t image = u ^ (uint32_t(int(u) >> 31) | 0x80000000u);
    const uint32_t x = (image & ~kSlots) | (kSlots - i);
    key[i] = kept && c[i] > none ? x : 0u;
  }
#pragma unroll
  for (int o = 0; o < NP / 8; ++o) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = key[8 * o + i];
    sort_down(b);
    if (o == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = b[i];
    } else {
      merge_top8(a, b);
    }
  }
  const bool full = a[7] != 0u;                  // there may be more than these eight
  uint32_t my_key = 0;
  int my_src = 0;
  for (int j = 0; j < r.k + 2; ++j) {            // and the two that are left first
    const uint32_t best = row_max_u32(a[0]);
    const unsigned long long owners = __ballot(a[0] == best);
    const int src = __ffs(uint32_t(owners >> (lane & 48)) & 0xffffu) - 1;
    if (q == j) my_key = best, my_src = src;
    const bool pop = q == src;
#pragma unroll
    for (int i = 0; i < 7; ++i) a[i] = pop ? a[i + 1] : a[i];
    a[7] = pop ? 0u : a[7];
  }
  doubt = doubt || (full && NP > 8 && a[0] == 0u) || (q < r.k + 2 && my_key == 0u);
  const int slot = int(kSlots - (my_key & kSlots));
  int my_id = my_key ? (my_src >> l2) * r.size + 4 * (my_src & ((1 << l2) - 1)) +
                           ((slot >> 2) << (l2 + 2)) + (slot & 3)
                     : 0;
  float l = row[my_id], mb = bias ? bias[my_id] : 0.f, s = 0.f;
  const float inv = __builtin_amdgcn_rcpf(total);
  for (int pass = 0;; ++pass) {
    float u = 1.f;
    if (bias) s = pick_score(l, top, inv, r.sigmoid, u);
    int way = order_of(l, mb, my_id, s, u, bias != nullptr, r.sigmoid);
    way = q + 1 < r.k + 2 ? way : 1;
    doubt = doubt || way == 0 || (pass == 3 && way < 0);
    const unsigned long long bad = __ballot(way < 0);
    if (!bad || pass == 3) break;
    const unsigned long long first = bad & ~(bad << 1);
    const int from = lane + int(first >> lane & 1) - int(first << 1 >> lane & 1);
    l = __shfl(l, from);
    mb = __shfl(mb, from);
    my_id = __shfl(my_id, from);
  }
  const float most = key_value(uint32_t(__shfl(int(my_key), (lane & 48) + r.k + 1)) | kSlots);
  if (q == r.k - 1) {
    const float x = bias ? s + mb : l;
    const float err = bias ? 2.f * ds + 0x1p-22f * (fabsf(most) + fabsf(x)) : 0.f;
    doubt = doubt || !(x - most > err);
  }
  const bool has = q < r.k;
  float p;
  if (r.sigmoid) {
    const float z = exp_down(-fabs(double(l)));
    float up = l < 0.f ? z : 1.f;
    if (r.norm) {
      const float lm = key_value(row_max_u32(has ? order_key(l) : 0u));
      if (lm < 0.f) up = l < lm ? exp_down(double(l) - double(lm)) : 1.f;
    }
    p = up / (1.f + z);
  } else if (r.norm) {
    const float lm = key_value(row_max_u32(has ? order_key(l) : 0u));
    p = exp_down(l == lm ? 0.0 : double(l) - double(lm));
  } else {
    p = exp_down(l == top ? 0.0 : double(l) - double(top)) / total;
  }
  p = has ? p : 0.f;
  if (r.norm) p /= row_sum_f32(p);
  const unsigned long long left = __ballot(doubt);
  const bool mine = ((left >> (lane & 48)) & 0xffffull) != 0;
  if (has && t < T && !mine) {
    ids[int64_t(t) * r.k + q] = my_id;
    w[int64_t(t) * r.k + q] = p * r.scale;
    if (hist) atomicAdd(&hist[my_id], 1);
  }
  for (int i = 0; i < kRowTokens; ++i) {
    if (t0 + i >= T || !((left >> (16 * i)) & 0xffffull)) continue;
    int id;
    float f;
    score_token<NP / 4>(logits + int64_t(t0 + i) * r.E, bias, r, id, f);
    if (lane < r.k) {
      ids[int64_t(t0 + i) * r.k + lane] = id;
      w[int64_t(t0 + i) * r.k + lane] = f;
      if (hist && id >= 0) atomicAdd(&hist[id], 1);
    }
  }
}

template <int NP>
__global__ __launch_bounds__(256) void k_route_scored_rows(const float* __restrict__ logits,
                                                           const float* __restrict__ bias, int T,
                                                           ScoreRule r, int32_t* __restrict__ ids,
                                                           float* __restrict__ w) {
  const int t0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * kRowTokens;
  if (t0 < T) score_rows<NP>(logits, bias, T, t0, r, ids, w, nullptr);
}

// and how many of the workgroup's 32 tokens took each expert, a byte an expert:
// the first step of the grouping
template <int NP>
__global__ __launch_bounds__(kCountTokens / kRowTokens * kWave) void k_route_scored_count(
    const float* __restrict__ logits, const float* __restrict__ bias, int T, ScoreRule r,
    int32_t* __restrict__ ids, float* __restrict__ w, uint32_t* __restrict__ bytes) {
  constexpr int NT = kCountTokens / kRowTokens * kWave;
  __shared__ int32_t hist[kCountExperts];
  for (int e = threadIdx.x; e < r.E; e += NT) hist[e] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * kCountTokens + (threadIdx.x >> 6) * kRowTokens;
  if (t0 < T) score_rows<NP>(logits, bias, T, t0, r, ids, w, hist);
  __syncthreads();
  for (int i = threadIdx.x; i < r.E / 4; i += NT)
    bytes[size_t(blockIdx.x) * (r.E / 4) + i] =
        hist[4 * i] | hist[4 * i + 1] << 8 | hist[4 * i + 2] << 16 | hist[4 * i + 3] << 24;
}

// experts that a lane holds
int per_lane(const ScoreRule& r) { return (r.size + (1 << r.lanes_log2) - 1) >> r.lanes_log2; }

// The kernel of four tokens a wave: whole vectors of logits, four lanes a group at
// least, of 32 experts at most.  In us, it and a wave a token, 384 experts in 8
// groups: 2048 tokens 6.3 and 5.5, 4096 6.5 and 7.1, 8192 7.7 and 10.6; with a token
// left to score_token, as in two of three inputs of 8192, 11 to 15 and 11 to 12.
bool takes_rows(int T, const ScoreRule& r, const float* logits, const float* bias) {
  return T >= 4096 && r.k <= kRowPicks && r.lanes_log2 >= 2 && per_lane(r) <= 8 && r.size % 4 == 0 &&
         r.keep * r.size >= r.k + 2 && reinterpret_cast<uintptr_t>(logits) % 16 == 0 &&
         reinterpret_cast<uintptr_t>(bias) % 16 == 0;
}

// f(experts that a lane of such a row holds)
template <class F>
void by_row_size(const ScoreRule& r, F f) {
  const int n = per_lane(r);
  if (n <= 2) f(std::integral_constant<int, 8>());
  else if (n <= 4) f(std::integral_constant<int, 16>());
  else if (n <= 6) f(std::integral_constant<int, 24>());
  else f(std::integral_constant<int, 32>());
}

}  // namespace

hipError_t launch_route_scored(const float* logits, const float* bias, int T, const ScoreRule& r,
                               int32_t* ids, float* w, hipStream_t s) {
  const int n = per_lane(r);
  const bool rows = takes_rows(T, r, logits, bias);
  // a launch has fewer than 2^32 threads
  constexpr int kMost = 1 << 25;
  for (int64_t t0 = 0; t0 < T; t0 += kMost) {
    const int nt = int(T - t0 < kMost ? T - t0 : kMost);
    auto go = [&](auto per) {
      k_route_scored<decltype(per)::value><<<(nt + 3) / 4, 256, 0, s>>>(
          logits + t0 * r.E, bias, nt, r, ids + t0 * r.k, w + t0 * r.k);
    };
    if (rows)
      by_row_size(r, [&](auto per) {
        k_route_scored_rows<decltype(per)::value><<<(nt + 15) / 16, 256, 0, s>>>(
            logits + t0 * r.E, bias, nt, r, ids + t0 * r.k, w + t0 * r.k);
      });
    else if (n <= 2) go(std::integral_constant<int, 2>());
    else if (n <= 4) go(std::integral_constant<int, 4>());
    else if (n <= 6) go(std::integral_constant<int, 6>());
    else if (n <= 8) go(std::integral_constant<int, 8>());
    else if (n <= 16) go(std::integral_constant<int, 16>());
    else go(std::integral_constant<int, 32>());
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

bool route_scored_counts(int T, const ScoreRule& r, const float* logits, const float* bias) {
  return takes_rows(T, r, logits, bias) && r.k == 8 && permute_counted_fits(T, r.E);
}

hipError_t launch_route_scored_count(const float* logits, const float* bias, int T,
                                     const ScoreRule& r, int32_t* ids, float* w, uint32_t* bytes,
                                     hipStream_t s) {
  by_row_size(r, [&](auto per) {
    k_route_scored_count<decltype(per)::value>
        <<<(T + kCountTokens - 1) / kCountTokens, kCountTokens / kRowTokens * kWave, 0, s>>>(
            logits, bias, T, r, ids, w, bytes);
  });
  return hipGetLastError();
}

// 16 waves leave a lane 128 registers: enough for eight experts each
bool route_scored_fusable(int T, const ScoreRule& r) { return T <= kFusedWaves && per_lane(r) <= 8; }

hipError_t launch_route_scored_permute(const float* logits, const float* bias, int T,
                                       const ScoreRule& r, int32_t* ids, float* w,
                                       int32_t* counts, int32_t* offsets, int32_t* sorted_pairs,
                                       int32_t* pair_to_row, hipStream_t s) {
  const size_t lds = (size_t(2) * r.E + 1 + size_t(T) * r.k) * sizeof(int32_t);
  const int n = per_lane(r);
  auto go = [&](auto per) {
    k_route_scored_permute<decltype(per)::value><<<1, kFusedWaves * kWave, lds, s>>>(
        logits, bias, T, r, ids, w, counts, offsets, sorted_pairs, pair_to_row);
  };
  if (n <= 2) go(std::integral_constant<int, 2>());
  else if (n <= 4) go(std::integral_constant<int, 4>());
  else if (n <= 6) go(std::integral_constant<int, 6>());
  else go(std::integral_constant<int, 8>());
  return hipGetLastError();
}

}  // namespace mxm
