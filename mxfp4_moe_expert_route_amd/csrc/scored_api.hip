// C ABI of routing by scores, of the layer that routes so and of low-rank
// adapters: host-side argument checks, then launches.  As in api.hip, every
// check runs before anything is enqueued and none of them touches the HIP
// runtime.
#include "../../include/mxfp4moe.h"

#include <cmath>

#include "lora.hpp"
#include "scored.hpp"

namespace {

constexpr int kMaxE = 1024;
constexpr int kMaxK = 32;
constexpr int kMaxH = 16384;
constexpr int kMaxI = 8192;
constexpr int kMaxGroups = 64;           // one lane of a wave at least a group
constexpr int kMaxLoraM = 1 << 20;
constexpr int kMaxLoraKN = 1 << 17;
constexpr int kMaxAdapters = 1024;       // as many as moe_permute groups by
constexpr int kMaxRank = 128;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int launched(hipError_t e) { return e == hipSuccess ? MXM_OK : MXM_ERR_LAUNCH; }

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

int check_rule(int T, int E, int k, int score, int groups, int topk_groups, int group_best,
               float scale) {
  if (score != MXM_SCORE_SOFTMAX && score != MXM_SCORE_SIGMOID) return MXM_ERR_DTYPE;
  if (T < 0 || E < 1 || E > kMaxE || k < 1 || k > kMaxK) return MXM_ERR_SHAPE;
  if (int64_t(T) * k > INT32_MAX) return MXM_ERR_SHAPE;
  if (groups < 1 || groups > kMaxGroups || E % groups || topk_groups < 1 || topk_groups > groups ||
      group_best < 1 || group_best > 2 || int64_t(topk_groups) * (E / groups) < k)
    return MXM_ERR_SHAPE;
  if (!std::isfinite(scale)) return MXM_ERR_SHAPE;
  return MXM_OK;
}

mxm::ScoreRule rule(int E, int k, int score, int groups, int topk_groups, int group_best,
                    int renormalise, float scale) {
  mxm::ScoreRule r{};
  r.E = E; r.k = k;
  r.groups = groups; r.keep = topk_groups; r.best = group_best;
  r.size = E / groups;
  r.lanes_log2 = 6;
  while ((groups << r.lanes_log2) > 64) --r.lanes_log2;
  r.sigmoid = score == MXM_SCORE_SIGMOID;
  r.norm = renormalise != 0;
  r.scale = scale;
  return r;
}

bool lora_shape(int M, int K, int N, int S, int r) {
  return M >= 0 && M <= kMaxLoraM && K >= 8 && K <= kMaxLoraKN && K % 8 == 0 && N >= 0 &&
         N <= kMaxLoraKN && S >= 1 && S <= kMaxAdapters && r >= 1 && r <= kMaxRank;
}

}  // namespace

extern "C" {

int moe_route_scored(const float* logits, const float* bias, int T, int E, int k, int score,
                     int groups, int topk_groups, int group_best, int renormalise, float scale,
                     int32_t* topk_ids, float* topk_w, void* stream) {
  const int st = check_rule(T, E, k, score, groups, topk_groups, group_best, scale);
  if (st != MXM_OK) return st;
  if (T == 0) return MXM_OK;
  if (!logits || !topk_ids || !topk_w) return MXM_ERR_NULL;
  if (!aligned(logits, 4) || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4))
    return MXM_ERR_ALIGN;
  return launched(mxm::launch_route_scored(
      logits, bias, T, rule(E, k, score, groups, topk_groups, group_best, renormalise, scale),
      topk_ids, topk_w, as_stream(stream)));
}

int moe_route_scored_permute(const float* logits, const float* bias, int T, int E, int k,
                             int score, int groups, int topk_groups, int group_best,
                             int renormalise, float scale, int32_t* topk_ids, float* topk_w,
                             int32_t* counts, int32_t* offsets, int32_t* sorted_pairs,
                             int32_t* pair_to_row, void* workspace, size_t workspace_bytes,
                             void* stream) {
  const int st = check_rule(T, E, k, score, groups, topk_groups, group_best, scale);
  if (st != MXM_OK) return st;
  const size_t need = moe_permute_workspace_bytes(T, E, k);
  if (workspace_bytes < need) return MXM_ERR_WORKSPACE;
  if (T == 0) return MXM_OK;
  if (!logits || !topk_ids || !topk_w || !counts || !offsets || !sorted_pairs || !pair_to_row ||
      (need > 0 && !workspace))
    return MXM_ERR_NULL;
  if (!aligned(logits, 4) || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) ||
      !aligned(counts, 4) || !aligned(offsets, 4) || !aligned(sorted_pairs, 4) ||
      !aligned(pair_to_row, 4) || !aligned(workspace, 4))
    return MXM_ERR_ALIGN;
  const hipStream_t s = as_stream(stream);
  const mxm::ScoreRule r = rule(E, k, score, groups, topk_groups, group_best, renormalise, scale);
  if (mxm::route_scored_fusable(T, r))
    return launched(mxm::launch_route_scored_permute(logits, bias, T, r, topk_ids, topk_w, counts,
                                                     offsets, sorted_pairs, pair_to_row, s));
  if (need > 0 && mxm::route_scored_counts(T, r, logits, bias)) {
    uint32_t* bytes = static_cast<uint32_t*>(workspace);
    if (mxm::launch_route_scored_count(logits, bias, T, r, topk_ids, topk_w, bytes, s) != hipSuccess)
      return MXM_ERR_LAUNCH;
    return launched(mxm::launch_permute_counted(topk_ids, T, E, k, bytes, counts, offsets,
                                                sorted_pairs, pair_to_row, s));
  }
  if (mxm::launch_route_scored(logits, bias, T, r, topk_ids, topk_w, s) != hipSuccess)
    return MXM_ERR_LAUNCH;
  return launched(mxm::launch_permute(topk_ids, T, E, k, counts, offsets, sorted_pairs,
                                      pair_to_row, workspace, s));
}

int moe_mxfp4_scored_layer(const uint16_t* x_bf16, const float* logits, const float* bias, int T,
                           int H, int I, int E, int k, int score, int groups, int topk_groups,
                           int group_best, int renormalise, float scale,
                           const uint8_t* w13_codes, const uint8_t* w13_scales,
                           const uint8_t* w2_codes, const uint8_t* w2_scales, int32_t* topk_ids,
                           float* topk_w, int32_t* counts, int32_t* offsets,
                           int32_t* sorted_pairs, int32_t* pair_to_row, uint16_t* h_bf16,
                           float* y, float* out, void* workspace, size_t workspace_bytes,
                           void* stream) {
  // check everything before enqueuing anything
  int st = check_rule(T, E, k, score, groups, topk_groups, group_best, scale);
  if (st != MXM_OK) return st;
  if (H < 32 || I < 32 || H % 32 || I % 32 || H > kMaxH || I > kMaxI) return MXM_ERR_SHAPE;
  if (int64_t(T) * k * int64_t(H > I ? H : I) > (int64_t(1) << 40)) return MXM_ERR_SHAPE;
  const size_t need = moe_permute_workspace_bytes(T, E, k);
  if (workspace_bytes < need) return MXM_ERR_WORKSPACE;
  if (T == 0) return MXM_OK;
  if (!x_bf16 || !logits || !w13_codes || !w13_scales || !w2_codes || !w2_scales || !topk_ids ||
      !topk_w || !counts || !offsets || !sorted_pairs || !pair_to_row || !h_bf16 || !y || !out ||
      (need > 0 && !workspace))
    return MXM_ERR_NULL;
  if (!aligned(x_bf16, 16) || !aligned(w13_codes, 16) || !aligned(w2_codes, 16) ||
      !aligned(w13_scales, 16) || !aligned(w2_scales, 16) || !aligned(h_bf16, 16) ||
      !aligned(y, 16) || !aligned(out, 16) || !aligned(logits, 4) || !aligned(bias, 4) ||
      !aligned(topk_ids, 4) || !aligned(topk_w, 4) || !aligned(counts, 4) ||
      !aligned(offsets, 4) || !aligned(sorted_pairs, 4) || !aligned(pair_to_row, 4) ||
      !aligned(workspace, 4))
    return MXM_ERR_ALIGN;
  if ((st = moe_route_scored_permute(logits, bias, T, E, k, score, groups, topk_groups, group_best,
                                     renormalise, scale, topk_ids, topk_w, counts, offsets,
                                     sorted_pairs, pair_to_row, workspace, workspace_bytes,
                                     stream)) != MXM_OK)
    return st;
  if ((st = moe_mxfp4_gate_up_swiglu(x_bf16, sorted_pairs, offsets, T, H, I, E, k, w13_codes,
                                     w13_scales, h_bf16, stream)) != MXM_OK)
    return st;
  if ((st = moe_mxfp4_down(h_bf16, offsets, T, H, I, E, k, w2_codes, w2_scales, y, stream)) !=
      MXM_OK)
    return st;
  return moe_combine(y, topk_w, pair_to_row, T, H, k, out, stream);
}

size_t lora_add_workspace_bytes(int M, int K, int N, int S, int r) {
  if (!lora_shape(M, K, N, S, r) || M == 0 || N == 0) return 0;
  return mxm::lora_workspace_bytes(M, K, N, S, r);
}

int lora_add(const uint16_t* x_bf16, const int32_t* sorted_rows, const int32_t* offsets, int M,
             int K, int N, int S, int r, const uint16_t* a_bf16, const uint16_t* b_bf16,
             const float* scale, void* y, int y_dtype, void* workspace, size_t workspace_bytes,
             void* stream) {
  if (y_dtype != MXM_F32 && y_dtype != MXM_BF16) return MXM_ERR_DTYPE;
  if (!lora_shape(M, K, N, S, r)) return MXM_ERR_SHAPE;
  if (M == 0 || N == 0) return MXM_OK;
  const size_t need = mxm::lora_workspace_bytes(M, K, N, S, r);
  if (workspace_bytes < need) return MXM_ERR_WORKSPACE;
  if (!x_bf16 || !sorted_rows || !offsets || !a_bf16 || !b_bf16 || !y || (need > 0 && !workspace))
    return MXM_ERR_NULL;
  if (!aligned(x_bf16, 16) || !aligned(a_bf16, 16) || !aligned(b_bf16, 16) ||
      !aligned(workspace, 16) || !aligned(sorted_rows, 4) || !aligned(offsets, 4) ||
      !aligned(scale, 4) || !aligned(y, y_dtype == MXM_F32 ? 4 : 2))
    return MXM_ERR_ALIGN;
  mxm::LoraProblem p{};
  p.x = x_bf16; p.rows = sorted_rows; p.offsets = offsets;
  p.a = a_bf16; p.b = b_bf16; p.scale = scale;
  p.y = y; p.part = static_cast<float*>(workspace);
  p.M = M; p.K = K; p.N = N; p.S = S; p.r = r;
  p.bf16 = y_dtype == MXM_BF16;
  return launched(mxm::launch_lora(p, as_stream(stream)));
}

}  // extern "C"
