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
  const int lane = lane_id();
  for (int t = blockIdx.x * 4 + (threadIdx.x >> 6); t < T; t += gridDim.x * 4) {
    int my_id;
    float my_w;
    score_token<NPER>(logits + int64_t(t) * r.E, bias, r, my_id, my_w);
    if (lane < r.k) {
      ids[int64_t(t) * r.k + lane] = my_id;
      w[int64_t(t) * r.k + lane] = my_w;
    }
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

// f<NPER>() for the experts that a lane holds
template <class F>
hipError_t by_size(const ScoreRule& r, F f) {
  const int n = (r.size + (1 << r.lanes_log2) - 1) >> r.lanes_log2;
  if (n <= 2) return f(std::integral_constant<int, 2>());
  if (n <= 4) return f(std::integral_constant<int, 4>());
  if (n <= 6) return f(std::integral_constant<int, 6>());
  if (n <= 8) return f(std::integral_constant<int, 8>());
  if (n <= 16) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
}

}  // namespace

hipError_t launch_route_scored(const float* logits, const float* bias, int T, const ScoreRule& r,
                               int32_t* ids, float* w, hipStream_t s) {
  const int grid = T / 4 + 1 < 65536 ? (T + 3) / 4 : 65536;
  return by_size(r, [&](auto n) {
    k_route_scored<decltype(n)::value><<<grid, 256, 0, s>>>(logits, bias, T, r, ids, w);
    return hipGetLastError();
  });
}

hipError_t launch_route_scored_permute(const float* logits, const float* bias, int T,
                                       const ScoreRule& r, int32_t* ids, float* w,
                                       int32_t* counts, int32_t* offsets, int32_t* sorted_pairs,
                                       int32_t* pair_to_row, hipStream_t s) {
  const size_t lds = (size_t(2) * r.E + 1 + size_t(T) * r.k) * sizeof(int32_t);
  return by_size(r, [&](auto n) {
    k_route_scored_permute<decltype(n)::value><<<1, kFusedWaves * kWave, lds, s>>>(
        logits, bias, T, r, ids, w, counts, offsets, sorted_pairs, pair_to_row);
    return hipGetLastError();
  });
}

}  // namespace mxm
