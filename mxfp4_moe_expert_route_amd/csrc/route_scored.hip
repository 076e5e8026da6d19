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

// experts that a lane holds
int per_lane(const ScoreRule& r) { return (r.size + (1 << r.lanes_log2) - 1) >> r.lanes_log2; }

}  // namespace

hipError_t launch_route_scored(const float* logits, const float* bias, int T, const ScoreRule& r,
                               int32_t* ids, float* w, hipStream_t s) {
  const int n = per_lane(r);
  // a launch has fewer than 2^32 threads
  constexpr int kMost = 1 << 25;
  for (int64_t t0 = 0; t0 < T; t0 += kMost) {
    const int nt = int(T - t0 < kMost ? T - t0 : kMost);
    auto go = [&](auto per) {
      k_route_scored<decltype(per)::value><<<(nt + 3) / 4, 256, 0, s>>>(
          logits + t0 * r.E, bias, nt, r, ids + t0 * r.k, w + t0 * r.k);
    };
    if (n <= 2) go(std::integral_constant<int, 2>());
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
