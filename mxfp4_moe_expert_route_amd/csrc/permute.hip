// Token-to-expert permutation: counts, offsets, sorted pair lists.  The
// algorithm is permute_block in routing.hpp; this file launches it as one
// workgroup of 4 waves (up to 1024 pairs) or 16 (up to 8192), and above that
// as one workgroup per range of pairs (one kernel or three, below).
#include "scored.hpp"

namespace mxm {
namespace {

template <int NW>
__global__ __launch_bounds__(NW * kWave) void k_permute(const int32_t* __restrict__ ids, int R,
                                                        int E, int32_t* __restrict__ counts,
                                                        int32_t* __restrict__ offsets,
                                                        int32_t* __restrict__ sorted_pairs,
                                                        int32_t* __restrict__ pair_to_row) {
  extern __shared__ int32_t smem[];
  __shared__ int32_t wave_sum[NW];
  permute_block<NW>(ids, 0, R, E, nullptr, counts, offsets, sorted_pairs, pair_to_row, smem,
                    wave_sum);
}

// Large batches: the pairs are cut into ranges of kRangePairs (more for very
// large R, so at most kMaxRanges ranges) handled by one workgroup each.
//  k_perm_hist     per-range expert histograms -> ws[range][E]
//  k_perm_scan     one workgroup: counts, offsets, and ws[range][e] replaced
//                  by the first row of expert e for that range (offsets[e]
//                  plus the counts of the earlier ranges)
//  k_perm_scatter  per range: permute_block from those bases
// Ranges, waves and lanes keep pair order, so the lists are the single
// workgroup's lists bit for bit.
constexpr int kRangePairs = 1024;
constexpr int kMaxRanges = 1024;
constexpr int kSingleMaxPairs = 8192;

__device__ __forceinline__ void range_of(int R, int nr, int b, int& r0, int& r1) {
  const int cb = (R + nr - 1) / nr;
  r0 = min(R, b * cb);
  r1 = min(R, r0 + cb);
}

__global__ __launch_bounds__(256) void k_perm_hist(const int32_t* __restrict__ ids, int R, int E,
                                                   int nr, int32_t* __restrict__ ws) {
  extern __shared__ int32_t hist[];
  int r0, r1;
  range_of(R, nr, blockIdx.x, r0, r1);
  for (int e = threadIdx.x; e < E; e += 256) hist[e] = 0;
  __syncthreads();
  for (int p = r0 + threadIdx.x; p < r1; p += 256) {
    const int id = ids[p];
    if (unsigned(id) < unsigned(E)) atomicAdd(&hist[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 256) ws[size_t(blockIdx.x) * E + e] = hist[e];
}

// one thread per expert (E <= 1024); a thread's counts over the ranges are
// read 16 at a time, all loads of a batch in flight together
constexpr int kScanBatch = 16;

__global__ __launch_bounds__(1024) void k_perm_scan(int E, int nr, int32_t* __restrict__ ws,
                                                    int32_t* __restrict__ counts,
                                                    int32_t* __restrict__ offsets) {
  __shared__ int32_t wave_tot[1024 / kWave];
  const int e = threadIdx.x, lane = lane_id(), wave = e / kWave;
  int total = 0;
  if (e < E)
    for (int b0 = 0; b0 < nr; b0 += kScanBatch) {
      int v[kScanBatch];
#pragma unroll
      for (int i = 0; i < kScanBatch; ++i) v[i] = b0 + i < nr ? ws[size_t(b0 + i) * E + e] : 0;
#pragma unroll
      for (int i = 0; i < kScanBatch; ++i) total += v[i];
    }
  const int incl = wave_incl_scan(total);
  if (lane == kWave - 1) wave_tot[wave] = incl;
  __syncthreads();
  int run = incl - total, all = 0;
  for (int w = 0; w < 1024 / kWave; ++w) {
    run += w < wave ? wave_tot[w] : 0;
    all += wave_tot[w];
  }
  if (e < E) {
    counts[e] = total;
    offsets[e] = run;
    for (int b0 = 0; b0 < nr; b0 += kScanBatch) {
      int v[kScanBatch];
#pragma unroll
      for (int i = 0; i < kScanBatch; ++i) v[i] = b0 + i < nr ? ws[size_t(b0 + i) * E + e] : 0;
#pragma unroll
      for (int i = 0; i < kScanBatch; ++i) {
        if (b0 + i < nr) ws[size_t(b0 + i) * E + e] = run;
        run += v[i];
      }
    }
  }
  if (e == 0) offsets[E] = all;
}

__global__ __launch_bounds__(4 * kWave) void k_perm_scatter(const int32_t* __restrict__ ids,
                                                            int R, int E, int nr,
                                                            const int32_t* __restrict__ ws,
                                                            int32_t* __restrict__ sorted_pairs,
                                                            int32_t* __restrict__ pair_to_row) {
  extern __shared__ int32_t smem[];
  __shared__ int32_t wave_sum[4];
  int r0, r1;
  range_of(R, nr, blockIdx.x, r0, r1);
  permute_block<4>(ids, r0, r1, E, ws + size_t(blockIdx.x) * E, nullptr, nullptr, sorted_pairs,
                   pair_to_row, smem, wave_sum);
}

// One launch for calls with k >= 4 up to one_max_pairs(E) pairs: every workgroup
// counts all pairs for itself, those before its range apart, which gives it the
// offsets and its bases.  Lanes that meet on one counter take turns (two cycles a
// lane), so there are eight copies of the counters: lanes of a run of eight have
// one each, and so have eight lanes of those eight apart, whether a token's ids are
// all the same or all tokens have the same ids.  In us, 65536 pairs of 384 experts,
// so, with one copy and in three launches: distinct ids in each token 11.7, 12.9 and
// 14.6; all ids the same 14.0, 61 and 15.3.
constexpr int kOneWaves = 16;
constexpr int kOneRange = 256;
constexpr int kOneBatch = 16;                    // ids a thread loads together
constexpr int kOneCopies = 8;

// Counting grows with the pairs, the three launches' scan with pairs times experts.
// In us, one launch and three, distinct ids: 8 experts, 65536 pairs 10.9 and 11.4,
// 131072 17.4 and 14.9; 384 experts, 98304 14.0 and 17.0 (all ids the same 17.6 and
// 17.7), 131072 17.6 and 19.6 (22 and 20); 1024 experts, 131072 18.2 and 26.
int one_max_pairs(int E) {
  const int most = 65536 + 128 * E;
  return most < 131072 ? most : 131072;
}

// A copy's counter holds the pairs before the range in its lower 16 bits and the
// others above: eight lanes of a wave share a copy, so neither passes 131072 / 8.
// Ints from one copy to the next: odd, so that an expert's lie in different banks.
__host__ __device__ constexpr int one_copy(int E) { return E | 1; }

// bases and permute_block's tables, before them, in the same place, the copies
// (k >= 4 experts at least, so 18 E ints are more than 8 (E + 1))
size_t one_lds(int E) { return size_t(1 + kOneWaves + 1) * E * sizeof(int32_t); }

// From how many pairs of expert threadIdx.x lie before the range and how many in it
// or past it (0 from E on; E <= 1024): counts, offsets, and in base[0, E) the range's
// first row of each expert.  By the whole workgroup, whose threads may read what
// lies at base until they call it.
__device__ __forceinline__ void bases_from_counts(int before, int rest, int32_t* base, int E,
                                                  int32_t* counts, int32_t* offsets,
                                                  int32_t* wave_sum) {
  const int tid = threadIdx.x, lane = lane_id(), wave = tid >> 6;
  const int total = before + rest;
  const int incl = wave_incl_scan(total);
  if (lane == kWave - 1) wave_sum[wave] = incl;
  __syncthreads();
  int run = incl - total, all = 0;
  for (int w = 0; w < kOneWaves; ++w) {
    run += w < wave ? wave_sum[w] : 0;
    all += wave_sum[w];
  }
  if (tid < E) {
    base[tid] = run + before;
    if (blockIdx.x == 0) {
      counts[tid] = total;
      offsets[tid] = run;
    }
  }
  if (tid == 0 && blockIdx.x == 0) offsets[E] = all;
  __syncthreads();
}

__global__ __launch_bounds__(kOneWaves * kWave) void k_perm_one(const int32_t* __restrict__ ids,
                                                                int R, int E, int nr,
                                                                int32_t* __restrict__ counts,
                                                                int32_t* __restrict__ offsets,
                                                                int32_t* __restrict__ sorted_pairs,
                                                                int32_t* __restrict__ pair_to_row) {
  constexpr int NT = kOneWaves * kWave;
  extern __shared__ int32_t smem[];
  __shared__ int32_t wave_sum[kOneWaves];
  const int tid = threadIdx.x;
  int r0, r1;
  range_of(R, nr, blockIdx.x, r0, r1);
  const int copy = one_copy(E);
  int32_t* mine = smem + ((lane_id() + (lane_id() >> 3)) & (kOneCopies - 1)) * copy;
  for (int e = tid; e < kOneCopies * copy; e += NT) smem[e] = 0;
  __syncthreads();
  for (int p0 = tid; p0 < R; p0 += NT * kOneBatch) {
    int id[kOneBatch];
#pragma unroll
    for (int i = 0; i < kOneBatch; ++i) id[i] = ids[min(p0 + NT * i, R - 1)];
#pragma unroll
    for (int i = 0; i < kOneBatch; ++i) {
      const int p = p0 + NT * i;
      if (p < R && unsigned(id[i]) < unsigned(E)) atomicAdd(&mine[id[i]], p < r0 ? 1 : 1 << 16);
    }
  }
  __syncthreads();
  int before = 0, rest = 0;
  if (tid < E) {
#pragma unroll
    for (int c = 0; c < kOneCopies; ++c) {
      const int n = smem[c * copy + tid];
      before += n & 0xffff;
      rest += n >> 16;
    }
  }
  bases_from_counts(before, rest, smem, E, counts, offsets, wave_sum);
  permute_block<kOneWaves>(ids, r0, r1, E, smem, nullptr, nullptr, sorted_pairs, pair_to_row,
                           smem + E, wave_sum);
}

// The same from the counts of every kCountTokens tokens, a byte an expert (E a
// multiple of 4, up to kCountExperts), that the routing left: four experts a
// thread, two sums of 16 bits to a register.  A token's experts are all different,
// so within the range a pair's rank is the number of lower bits in its expert's
// mask of tokens.
__global__ __launch_bounds__(kOneWaves * kWave) void k_perm_counted(
    const int32_t* __restrict__ ids, int R, int E, int k, const uint32_t* __restrict__ bytes, int rows,
    int32_t* __restrict__ counts, int32_t* __restrict__ offsets, int32_t* __restrict__ sorted_pairs,
    int32_t* __restrict__ pair_to_row) {
  constexpr int NT = kOneWaves * kWave;
  extern __shared__ int32_t smem[];
  __shared__ int32_t wave_sum[kOneWaves];
  __shared__ uint32_t part[4][kCountExperts / 4];        // even and odd experts, before and from here on
  uint32_t* mask = reinterpret_cast<uint32_t*>(smem + E);
  const int tid = threadIdx.x, cols = E / 4, here = blockIdx.x;
  const int pair = here * kCountTokens * k + tid;          // of the first kCountTokens k threads
  const bool owns = tid < kCountTokens * k && pair < R;
  const int id = owns ? ids[pair] : -1;
  for (int i = tid; i < kCountExperts; i += NT) (&part[0][0])[i] = 0u;
  for (int i = tid; i < E; i += NT) mask[i] = 0u;
  __syncthreads();
  const bool valid = unsigned(id) < unsigned(E);
  if (valid) atomicOr(&mask[id], 1u << (tid / k));
  const int col = tid % cols, parts = NT / cols, mine = tid / cols;
  if (mine < parts) {
    uint32_t s[4] = {0u, 0u, 0u, 0u};
    for (int b0 = mine; b0 < rows; b0 += parts * kOneBatch) {
      uint32_t v[kOneBatch];
#pragma unroll
      for (int i = 0; i < kOneBatch; ++i)
        v[i] = bytes[size_t(min(b0 + parts * i, rows - 1)) * cols + col];
#pragma unroll
      for (int i = 0; i < kOneBatch; ++i) {
        const int b = b0 + parts * i;
        const uint32_t x = b < rows ? v[i] : 0u;
        const uint32_t even = x & 0x00ff00ffu, odd = x >> 8 & 0x00ff00ffu;
        s[0] += b < here ? even : 0u;
        s[1] += b < here ? odd : 0u;
        s[2] += b < here ? 0u : even;
        s[3] += b < here ? 0u : odd;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) atomicAdd(&part[i][col], s[i]);
  }
  __syncthreads();
  int before = 0, rest = 0;
  if (tid < E) {
    const int i = tid >> 2, shift = (tid & 2) * 8;
    before = part[tid & 1][i] >> shift & 0xffff;
    rest = part[2 + (tid & 1)][i] >> shift & 0xffff;
  }
  bases_from_counts(before, rest, smem, E, counts, offsets, wave_sum);
  if (valid) {
    const int row = smem[id] + __popc(mask[id] & ((1u << (tid / k)) - 1u));
    sorted_pairs[row] = pair;
    pair_to_row[pair] = row;
  } else if (owns) {
    pair_to_row[pair] = -1;
  }
}

int ranges_for(int64_t R) {
  if (R <= kSingleMaxPairs) return 0;
  const int64_t n = (R + kRangePairs - 1) / kRangePairs;
  return int(n < kMaxRanges ? n : kMaxRanges);
}

}  // namespace

// an expert's count fits 16 bits, and the bytes fit the workspace of three launches
constexpr int kCountedTokens = 1 << 14;

bool permute_counted_fits(int T, int E) {
  return T <= kCountedTokens && E % 4 == 0 && E <= kCountExperts;
}

hipError_t launch_permute_counted(const int32_t* ids, int T, int E, int k, const uint32_t* bytes,
                                  int32_t* counts, int32_t* offsets, int32_t* sorted_pairs,
                                  int32_t* pair_to_row, hipStream_t s) {
  const int rows = (T + kCountTokens - 1) / kCountTokens;
  k_perm_counted<<<rows, kOneWaves * kWave, size_t(2) * E * sizeof(int32_t), s>>>(ids, T * k, E, k, bytes, rows, counts, offsets,
                                                            sorted_pairs, pair_to_row);
  return hipGetLastError();
}

size_t permute_workspace_bytes(int T, int E, int k) {
  return size_t(ranges_for(int64_t(T) * k)) * E * sizeof(int32_t);
}

hipError_t launch_permute(const int32_t* ids, int T, int E, int k, int32_t* counts,
                          int32_t* offsets, int32_t* sorted_pairs, int32_t* pair_to_row,
                          void* workspace, hipStream_t s) {
  const int R = T * k;
  const int nr = ranges_for(R);
  if (nr > 0 && k >= 4 && R <= one_max_pairs(E)) {
    static std::atomic<bool> set[kMaxDevices];   // 18 E ints, E up to 1024: above 64 KB
    const hipError_t e = lds_limit_once(reinterpret_cast<const void*>(&k_perm_one), int(one_lds(1024)), set);
    if (e != hipSuccess) return e;
    const int n = (R + kOneRange - 1) / kOneRange < 256 ? (R + kOneRange - 1) / kOneRange : 256;
    k_perm_one<<<n, kOneWaves * kWave, one_lds(E), s>>>(ids, R, E, n, counts, offsets, sorted_pairs, pair_to_row);
    return hipGetLastError();
  }
  if (nr > 0) {
    int32_t* ws = static_cast<int32_t*>(workspace);
    k_perm_hist<<<nr, 256, size_t(E) * sizeof(int32_t), s>>>(ids, R, E, nr, ws);
    k_perm_scan<<<1, 1024, 0, s>>>(E, nr, ws, counts, offsets);
    k_perm_scatter<<<nr, 4 * kWave, size_t(5) * E * sizeof(int32_t), s>>>(ids, R, E, nr, ws,
                                                                          sorted_pairs, pair_to_row);
    return hipGetLastError();
  }
  if (R <= 1024) {                // 5 E ints: within the default 64 KB for E <= 1024
    k_permute<4><<<1, 4 * kWave, size_t(5) * E * sizeof(int32_t), s>>>(
        ids, R, E, counts, offsets, sorted_pairs, pair_to_row);
    return hipGetLastError();
  }
  static std::atomic<bool> lds_set[kMaxDevices];   // 17 E ints, E up to 1024: above 64 KB
  const hipError_t e = lds_limit_once(reinterpret_cast<const void*>(&k_permute<16>),
                                      int(17 * 1024 * sizeof(int32_t)), lds_set);
  if (e != hipSuccess) return e;
  k_permute<16><<<1, 16 * kWave, size_t(17) * E * sizeof(int32_t), s>>>(
      ids, R, E, counts, offsets, sorted_pairs, pair_to_row);
  return hipGetLastError();
}

}  // namespace mxm
