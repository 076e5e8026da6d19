// Low-rank adapters of many requests beside a shared projection: what the
// kernels and the entry points share.
#pragma once
#include "common.hpp"

namespace mxm {

// y[row, n] += scale[s] sum_j b[s, n, j] sum_k a[s, j, k] x[row, k] for the rows
// sorted_rows[p], offsets[s] <= p < offsets[s + 1], of every adapter s
struct LoraProblem {
  const uint16_t* x;
  const int32_t* rows;
  const int32_t* offsets;
  const uint16_t* a;
  const uint16_t* b;
  const float* scale;      // or null: 1
  void* y;
  float* part;             // [splits, M, padded rank]: a x, in pieces of K
  int M, K, N, S, r;
  bool bf16;
};

size_t lora_workspace_bytes(int M, int K, int N, int S, int r);
hipError_t launch_lora(const LoraProblem& p, hipStream_t s);

}  // namespace mxm
