// C ABI of the products of two MXFP4 factors, of the layer on MXFP4
// activations and of verification from probabilities: host-side argument
// checks, then launches.  As in api.hip, every check runs before anything is
// enqueued and none of them touches the HIP runtime.
#include "../../include/mxfp4moe.h"

#include <cmath>

#include "a4.hpp"

namespace {

using mxm::a4::Problem;

constexpr int kMaxE = 1024;
constexpr int kMaxK = 32;
constexpr int kMaxH = 16384;
constexpr int kMaxI = 8192;
constexpr int kMaxGemmK = 1 << 20;
constexpr int kMaxGemmMN = 1 << 30;      // rows and columns are counted in 31 bits, past the last tile too
constexpr int kMaxVerifyL = 32;          // one lane of a wave per block position
constexpr int kMaxVerifyB = 1 << 20;     // a launch has fewer than 2^32 threads, 1024 a block
constexpr int kMaxVerifyV = 1 << 30;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int launched(hipError_t e) { return e == hipSuccess ? MXM_OK : MXM_ERR_LAUNCH; }

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

int check_ffn_shape(int T, int H, int I, int E, int k) {
  if (T < 0 || E < 1 || E > kMaxE || k < 1 || k > kMaxK || k > E) return MXM_ERR_SHAPE;
  if (int64_t(T) * k > INT32_MAX) return MXM_ERR_SHAPE;
  if (H < 32 || I < 32 || H % 32 || I % 32 || H > kMaxH || I > kMaxI) return MXM_ERR_SHAPE;
  return MXM_OK;
}

// parts of a block and a row's elements are counted in 31 bits
bool verify_probs_shape(int B, int L, int V) {
  return B >= 0 && B <= kMaxVerifyB && L >= 1 && L <= kMaxVerifyL && V >= 1 && V <= kMaxVerifyV;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Which kernel and tile a product takes: the one whose time, estimated from
// sizes alone, is least.  A direct unit costs the loads of its fragments, 70
// ns each per 256 of K and CU.  A tiled item costs the stages of its tile and
// its epilogue; a stage takes longer the more CUs are busy (they share L2 and
// power), so a last, partial round goes faster.  The constants are fits of
// measured times, to about 15%.  In us, by tile 256 x 192, 128 x 192, 128 x 128,
// 128 x 64, 128 x 32: 512 x 6144 x 2048 20.9, 14.0, 11.9, 13.8, 16.2; 333 x 4096
// x 6144 35.8, 23.4, 19.1, 15.7, 26.3; 260 x 2049 x 2048 18.3, 11.8, 9.8, 8.3,
// 7.5; 4096 x 4096 x 4096 58, 53, 55, 67, 113; 8192 x 4096 x 6144 131, 170 by the
// first two.  Direct: 8 x 4096 x 6144 5 (11 by 128 x 32).
hipError_t product(mxm::a4::Out out, const Problem& p, hipStream_t s) {
  struct Tile {
    int a, ms;
    double idle, busy, item;             // tiled: us per stage of 256 of K, per item
  };
  constexpr Tile kDirect[] = {{1, 1}, {1, 2}, {2, 2}, {2, 4}};
  constexpr Tile kTiled[] = {{4, 6, 0.93, 1.4, 8.0},
                             {2, 6, 0.60, 0.9, 3.2},
                             {2, 4, 0.42, 0.64, 2.7},
                             {2, 2, 0.40, 0.40, 1.6},
                             {2, 1, 0.35, 0.35, 1.0}};
  constexpr int kCus = 256;
  const double chunks = double(ceil_div(p.K, 256));
  double best = 1e30;
  const Tile* t = nullptr;
  bool tiled = false;
  for (const Tile& c : kDirect) {
    const int64_t units = ceil_div(p.N, 16 * c.a) * ceil_div(p.M, 16 * c.ms);
    const double us = 2.3 + double(ceil_div(units, kCus)) * (0.07 * chunks * (c.a + c.ms) + 0.1);
    if (us < best) best = us, t = &c;
  }
  if (mxm::a4::tiled_supported(mxm::a4::kGemm, p)) {
    for (const Tile& c : kTiled) {
      const int64_t items = ceil_div(p.N, 64 * c.a) * ceil_div(p.M, 32 * c.ms);
      const double last = double(items % kCus) / kCus;
      const double us = 4.3 + double(ceil_div(items, kCus)) * c.item + double(items / kCus) * chunks * c.busy +
                        (last > 0 ? chunks * (c.idle + last * (c.busy - c.idle)) : 0.0);
      if (us < best) best = us, t = &c, tiled = true;
    }
  }
  return tiled ? mxm::a4::launch_tiled_gemm(out, p, t->a, t->ms, s)
               : mxm::a4::launch_direct_gemm(out, p, t->a, t->ms, s);
}

// The same for the experts' contractions, for a uniform routing.  A row tile is
// as tall as a typical expert (mean rows and a standard deviation): a taller
// one multiplies rows that are not there, a shorter one reads the weights
// again.  Page-shaped gate/up, tiles of 32, 64, 96 and 192 rows: 841, 900, 958,
// 1154 us at 512 tokens (11 rows an expert); 1372, 933, 1005, 1181 at 2048 (43);
// 2085, 1483, 1211, 1256 at 4096 (85); 3921, 2217, 1678, 1390 at 8192 (171).
// Routing is skewed as a rule, so the experts that outgrow the tile go to a
// taller one in a launch of their own: Zipf-routed, 512 tokens take 544 us so
// and 637 with 32-row tiles alone.  Where there is nothing for it that launch
// costs about 4 us: small calls and batches with few rows an expert do without.
// A gate/up item of K below 800 is mostly start and end, which the estimate
// misses: there the tiled kernel takes over where a typical expert has more rows
// than a direct unit, 64.  In us, direct and tiled, 384 experts of 2 2048
// columns, 8 of them a token: K = 544, 8 tokens 22 and 36, 1536 258 and 261, 3040
// 383 and 298; K = 768, 8 tokens 27 and 29, 8192 859 and 438.
hipError_t grouped(mxm::a4::Kind kind, mxm::a4::Out out, const Problem& p, hipStream_t s) {
  const bool gu = kind == mxm::a4::kGateUp;
  const int groups = p.R < p.E ? p.R : p.E;
  const double mean = double(p.R) / groups;
  const int64_t tall = int64_t(mean + std::sqrt(mean));
  const double chunks = double(ceil_div(p.K, 256));
  constexpr int kCus = 256;
  double best = 1e30;
  int ms = 1;
  bool tiled = false;
  for (int m = 1; m <= 4; m += 3) {
    const bool mx = out == mxm::a4::kMx;
    const int64_t units = groups * ceil_div(tall < 1 ? 1 : tall, mx && m > 1 ? 32 : 16 * m) *
                          ceil_div(p.N, mx ? 32 : 16);
    const int frags = (gu ? 2 : 1) * (mx ? 2 : 1) + (mx && m > 1 ? 2 : m);
    const double us = 2.3 + double(ceil_div(units, kCus)) * (0.07 * chunks * frags + 0.8);
    if (us < best) best = us, ms = m;
  }
  if (mxm::a4::tiled_supported(kind, p) && !(gu && p.K < 800 && tall <= 64)) {
    constexpr double kStage[] = {1.35, 1.45, 1.5};   // us per stage of 256 of K
    for (int m = 1; m <= 3; ++m) {
      const int64_t items = groups * ceil_div(tall < 1 ? 1 : tall, 32 * m) * ceil_div(p.N, gu ? 128 : 256);
      const double us = 3.0 + double(ceil_div(items, kCus)) * (chunks * kStage[m - 1] + 1.2 * m);
      if (us < best) best = us, ms = m, tiled = true;
    }
  }
  if (!tiled) return mxm::a4::launch_direct(kind, out, p, ms, s);
  const bool split = mean >= 4 && best > 60;
  if (split) ms = tall <= 32 ? 1 : tall <= 64 ? 2 : 3;
  return mxm::a4::launch_tiled(kind, out, p, ms, split, s);
}

}  // namespace

extern "C" {

int mxfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
               const uint8_t* b_scales, int M, int N, int K, void* c, int c_dtype, void* stream) {
  if (c_dtype != MXM_F32 && c_dtype != MXM_BF16) return MXM_ERR_DTYPE;
  if (M < 0 || N < 0 || M > kMaxGemmMN || N > kMaxGemmMN) return MXM_ERR_SHAPE;
  if (K < 32 || K % 32 || K > kMaxGemmK) return MXM_ERR_SHAPE;
  if (M == 0 || N == 0) return MXM_OK;
  if (!a_codes || !a_scales || !b_codes || !b_scales || !c) return MXM_ERR_NULL;
  if (!aligned(a_codes, 16) || !aligned(b_codes, 16) || !aligned(c, c_dtype == MXM_F32 ? 4 : 2))
    return MXM_ERR_ALIGN;
  Problem p{};
  p.xc = a_codes; p.xs = a_scales; p.wc = b_codes; p.ws = b_scales;
  p.out = c;
  p.M = M; p.R = M; p.N = N; p.K = K; p.E = 1; p.k = 1;
  p.lo = 1; p.hi = INT32_MAX;
  return launched(product(c_dtype == MXM_F32 ? mxm::a4::kF32 : mxm::a4::kBf16, p,
                          as_stream(stream)));
}

int moe_mxfp4_a4_gate_up_swiglu(const uint8_t* x_codes, const uint8_t* x_scales,
                                const int32_t* sorted_pairs, const int32_t* offsets, int T, int H,
                                int I, int E, int k, const uint8_t* w13_codes,
                                const uint8_t* w13_scales, uint16_t* h_bf16, uint8_t* h_codes,
                                uint8_t* h_scales, void* stream) {
  const int st = check_ffn_shape(T, H, I, E, k);
  if (st != MXM_OK) return st;
  if (T == 0) return MXM_OK;
  const bool mx = h_codes || h_scales;
  if (!x_codes || !x_scales || !sorted_pairs || !offsets || !w13_codes || !w13_scales ||
      (mx ? !h_codes || !h_scales || h_bf16 : !h_bf16))
    return MXM_ERR_NULL;
  if (!aligned(x_codes, 16) || !aligned(w13_codes, 16) || !aligned(h_bf16, 16) ||
      !aligned(h_codes, 16) || !aligned(sorted_pairs, 4) || !aligned(offsets, 4))
    return MXM_ERR_ALIGN;
  Problem p{};
  p.xc = x_codes; p.xs = x_scales; p.wc = w13_codes; p.ws = w13_scales;
  p.pairs = sorted_pairs; p.offsets = offsets;
  p.out = h_bf16; p.oc = h_codes; p.os = h_scales;
  p.M = T; p.R = T * k; p.N = I; p.K = H; p.E = E; p.k = k;
  p.lo = 1; p.hi = INT32_MAX;
  return launched(grouped(mxm::a4::kGateUp, mx ? mxm::a4::kMx : mxm::a4::kBf16, p,
                          as_stream(stream)));
}

int moe_mxfp4_a4_down(const uint8_t* h_codes, const uint8_t* h_scales, const int32_t* offsets,
                      int T, int H, int I, int E, int k, const uint8_t* w2_codes,
                      const uint8_t* w2_scales, float* y, void* stream) {
  const int st = check_ffn_shape(T, H, I, E, k);
  if (st != MXM_OK) return st;
  if (T == 0) return MXM_OK;
  if (!h_codes || !h_scales || !offsets || !w2_codes || !w2_scales || !y) return MXM_ERR_NULL;
  if (!aligned(h_codes, 16) || !aligned(w2_codes, 16) || !aligned(y, 16) || !aligned(offsets, 4))
    return MXM_ERR_ALIGN;
  Problem p{};
  p.xc = h_codes; p.xs = h_scales; p.wc = w2_codes; p.ws = w2_scales;
  p.offsets = offsets;
  p.out = y;
  p.M = T * k; p.R = T * k; p.N = H; p.K = I; p.E = E; p.k = k;
  p.lo = 1; p.hi = INT32_MAX;
  return launched(grouped(mxm::a4::kDown, mxm::a4::kF32, p, as_stream(stream)));
}

int moe_mxfp4_a4_layer(const uint16_t* x_bf16, const float* logits, int T, int H, int I, int E,
                       int k, const uint8_t* w13_codes, const uint8_t* w13_scales,
                       const uint8_t* w2_codes, const uint8_t* w2_scales, int32_t* topk_ids,
                       float* topk_w, int32_t* counts, int32_t* offsets, int32_t* sorted_pairs,
                       int32_t* pair_to_row, uint8_t* x_codes, uint8_t* x_scales,
                       uint8_t* h_codes, uint8_t* h_scales, float* y, float* out,
                       void* workspace, size_t workspace_bytes, void* stream) {
  // check everything before enqueuing anything
  int st = check_ffn_shape(T, H, I, E, k);
  if (st != MXM_OK) return st;
  const size_t need = moe_permute_workspace_bytes(T, E, k);
  if (workspace_bytes < need) return MXM_ERR_WORKSPACE;
  if (T == 0) return MXM_OK;
  if (!x_bf16 || !logits || !w13_codes || !w13_scales || !w2_codes || !w2_scales || !topk_ids ||
      !topk_w || !counts || !offsets || !sorted_pairs || !pair_to_row || !x_codes || !x_scales ||
      !h_codes || !h_scales || !y || !out || (need > 0 && !workspace))
    return MXM_ERR_NULL;
  if (!aligned(x_bf16, 16) || !aligned(w13_codes, 16) || !aligned(w2_codes, 16) ||
      !aligned(x_codes, 16) || !aligned(h_codes, 16) || !aligned(y, 16) || !aligned(out, 16) ||
      !aligned(logits, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) ||
      !aligned(counts, 4) || !aligned(offsets, 4) || !aligned(sorted_pairs, 4) ||
      !aligned(pair_to_row, 4) || !aligned(workspace, 4))
    return MXM_ERR_ALIGN;
  if ((st = moe_route_permute(logits, T, E, k, topk_ids, topk_w, counts, offsets, sorted_pairs,
                              pair_to_row, workspace, workspace_bytes, stream)) != MXM_OK)
    return st;
  if ((st = mxfp4_pack(x_bf16, MXM_BF16, T, H, x_codes, x_scales, stream)) != MXM_OK) return st;
  if ((st = moe_mxfp4_a4_gate_up_swiglu(x_codes, x_scales, sorted_pairs, offsets, T, H, I, E, k,
                                        w13_codes, w13_scales, nullptr, h_codes, h_scales,
                                        stream)) != MXM_OK)
    return st;
  if ((st = moe_mxfp4_a4_down(h_codes, h_scales, offsets, T, H, I, E, k, w2_codes, w2_scales, y,
                              stream)) != MXM_OK)
    return st;
  return moe_combine(y, topk_w, pair_to_row, T, H, k, out, stream);
}

size_t dflash_verify_probs_workspace_bytes(int B, int L, int V) {
  if (B == 0 || !verify_probs_shape(B, L, V)) return 0;
  return mxm::verify_probs_workspace_bytes(B, V);
}

int dflash_verify_probs(const void* target_probs, const void* draft_probs, int dtype,
                        const int32_t* draft_tokens, const int32_t* draft_len,
                        const float* uniforms, int B, int L, int V, int32_t* accept_len,
                        int32_t* next_token, void* workspace, size_t workspace_bytes,
                        void* stream) {
  if (dtype != MXM_F32 && dtype != MXM_BF16) return MXM_ERR_DTYPE;
  if (!verify_probs_shape(B, L, V)) return MXM_ERR_SHAPE;
  if (B == 0) return MXM_OK;
  const size_t need = dflash_verify_probs_workspace_bytes(B, L, V);
  if (workspace_bytes < need) return MXM_ERR_WORKSPACE;
  if (!target_probs || !draft_probs || !draft_tokens || !uniforms || !accept_len || !next_token ||
      (need > 0 && !workspace))
    return MXM_ERR_NULL;
  const uintptr_t size = dtype == MXM_F32 ? 4 : 2;
  if (!aligned(target_probs, size) || !aligned(draft_probs, size) || !aligned(draft_tokens, 4) ||
      !aligned(draft_len, 4) || !aligned(uniforms, 4) || !aligned(accept_len, 4) ||
      !aligned(next_token, 4) || !aligned(workspace, 8))
    return MXM_ERR_ALIGN;
  return launched(mxm::launch_verify_probs(target_probs, draft_probs, dtype == MXM_BF16,
                                           draft_tokens, draft_len, uniforms, B, L, V, accept_len,
                                           next_token, workspace, as_stream(stream)));
}

}  // extern "C"
