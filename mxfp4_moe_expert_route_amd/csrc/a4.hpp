// Products of two MXFP4 factors on the scaled matrix instructions: what the
// kernels of mxfp4_gemm and of the expert contractions on MXFP4 activations
// share.
//
// Both factors are stored alike: E2M1 codes [rows, K/2] and E8M0 block scales
// [rows, K/32], row-major, blocks along K.  v_mfma_scale_f32_16x16x128_f8f6f4
// takes exactly that: of each operand lane 16 g + r holds row r's block g of
// four (32 codes, 16 bytes) and, in the low byte of a register, that block's
// scale.  Nothing is converted: a product of two E2M1 values has at most six
// significant bits and the block factors are powers of two, so every product
// is exact and only the fp32 sums round.
//
// Throughout, "weights" (W) are the factor whose rows become output columns
// and operand A of the instruction, "rows" (X) the other one, operand B: lane
// 16 g + r of the result holds columns 4 g .. 4 g + 3 of row r.
//
// Scale byte 255 (NaN) makes every product of its block NaN and byte 0 is
// 2^-127; the instruction takes both as they are.
#pragma once
#include "common.hpp"

namespace mxm {
namespace a4 {

typedef __attribute__((ext_vector_type(8))) int i32x8;

constexpr int kFp4 = 4;                        // operand format code: E2M1

// acc += X (operand B) times W (operand A); scales in the low byte of sw, sx
__device__ __forceinline__ f32x4 mfma(uint4 w, uint32_t sw, uint4 x, uint32_t sx, f32x4 acc) {
  const i32x8 a = {int(w.x), int(w.y), int(w.z), int(w.w), 0, 0, 0, 0};
  const i32x8 b = {int(x.x), int(x.y), int(x.z), int(x.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, kFp4, kFp4, 0, int(sw), 0,
                                                          int(sx));
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// Which contraction, and what becomes of the sums.
enum Kind { kGemm, kGateUp, kDown };
enum Out { kF32, kBf16, kMx };

// One contraction.  kGemm: out [M, N] = X [M, K] W [N, K]^T.  kGateUp: row r
// of expert e is X row pairs[r] / k, W is [E, 2 N, K] (N gate rows, then N up
// rows), out [R, N] the SwiGLU of the two.  kDown: row r is X row r, W is
// [E, N, K].  Grouped kinds take the experts with lo <= rows < hi.
struct Problem {
  const uint8_t* xc;
  const uint8_t* xs;
  const uint8_t* wc;
  const uint8_t* ws;
  const int32_t* pairs;
  const int32_t* offsets;
  void* out;              // f32 or bf16 (kF32, kBf16)
  uint8_t* oc;            // kMx: codes [R, N/2]
  uint8_t* os;            // kMx: scales [R, N/32]
  int M;                  // rows of X (kGemm), T (kGateUp), R (kDown)
  int R;                  // rows of out
  int N, K, E, k;
  int lo, hi;
};

// Operands straight from memory: every shape.  Grouped units are low (16 rows;
// ms 1) or high (64 rows, 32 where h is packed); the product's are 16 cf
// columns x 16 ms rows: (1, 1), (1, 2), (2, 2) or (2, 4).
hipError_t launch_direct(Kind kind, Out out, const Problem& p, int ms, hipStream_t s);
hipError_t launch_direct_gemm(Out out, const Problem& p, int cf, int ms, hipStream_t s);
// Persistent, through LDS.  Grouped tiles are 32 ms rows tall, ms 1, 2 or 3
// (split: experts with more rows in a launch of their own, with taller tiles);
// the product's are 64 as columns x 32 ms rows: (4, 6), (2, 6), (2, 4), (2, 2)
// or (2, 1).
bool tiled_supported(Kind kind, const Problem& p);
hipError_t launch_tiled(Kind kind, Out out, const Problem& p, int ms, bool split, hipStream_t s);
hipError_t launch_tiled_gemm(Out out, const Problem& p, int as, int ms, hipStream_t s);

}  // namespace a4

// Verification of drafted tokens from probabilities.
size_t verify_probs_workspace_bytes(int B, int V);
hipError_t launch_verify_probs(const void* target, const void* draft, bool bf16,
                               const int32_t* tokens, const int32_t* draft_len,
                               const float* uniforms, int B, int L, int V, int32_t* accept_len,
                               int32_t* next_token, void* workspace, hipStream_t s);

}  // namespace mxm
