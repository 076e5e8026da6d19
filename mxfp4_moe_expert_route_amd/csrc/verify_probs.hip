// Verification of drafted tokens from probabilities: acceptance of a block's
// leading tokens and the draw of the next one.
//
// The rule ("MiMo-V2.5-Pro-FP4-DFlash" model card, §3: rejection sampling
// keeps the drafted block's verification lossless): token i is accepted when
// u_i q_i(d_i) < p_i(d_i); after the n accepted ones the next token is drawn
// from max(0, p_n - q_n), or from p_n where the whole block was accepted or
// that difference is zero everywhere, as the smallest token whose running
// sum of weights exceeds u_L times their sum.
//
// Decisions are made in fp64: products and differences of two fp32 (or bf16)
// values are exact there, and a sum over a vocabulary of 2^18 is off by at
// most 2^-35 of itself, so a draw depends on the order of summation only
// where u_L falls within that of a boundary.  Sums run in a fixed order.
//
// Of the (L + 1) V probabilities of a block only the drafted tokens' entries
// and the two rows at position n are read.  Two launches: the weights' sums
// over parts of row n, by workgroups that each find n themselves (2 L loads,
// cheaper than a launch), then one workgroup per block that finds the part
// holding the draw and reads it again.
#include "a4.hpp"

namespace mxm {
namespace {

constexpr int kT = 256;
constexpr int kWavesV = kT / kWave;
constexpr int kMaxParts = 128;
constexpr int kMinPart = 4 * kT;               // elements a part is worth a workgroup for

struct Sums {
  double w, p;                                 // of max(0, p - q), of p
};

// Parts per row: enough workgroups to fill the CUs, none below kMinPart.
int parts_of(int B, int V) {
  int n = (4 * 256 + B - 1) / B;
  const int most = (V + kMinPart - 1) / kMinPart;
  n = n < most ? n : most;
  return n < 1 ? 1 : (n > kMaxParts ? kMaxParts : n);
}

__device__ __forceinline__ float value(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float value(const uint16_t* p, int64_t i) {
  return __uint_as_float(uint32_t(p[i]) << 16);
}

// A probability: what is not a positive finite number counts as none.
__device__ __forceinline__ double clean(float v) {
  return v > 0.f && v < INFINITY ? double(v) : 0.0;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// Accepted tokens of block b (every wave computes it; uniform result).
template <typename T>
__device__ __forceinline__ int accepted(const T* target, const T* draft, const int32_t* tokens,
                                        const float* uniforms, int len, int b, int L, int V) {
  const int lane = lane_id();
  bool fail = false;
  if (lane < len) {
    const int64_t at = int64_t(b) * L + lane;
    const int d = tokens[at];
    fail = true;
    if (d >= 0 && d < V) {
      const double pd = clean(value(target, (at + b) * V + d));
      const double qd = clean(value(draft, at * V + d));
      fail = !(double(uniforms[at + b]) * qd < pd);
    }
  }
  const unsigned long long m = __ballot(fail);
  return __builtin_amdgcn_readfirstlane(m ? __ffsll((long long)m) - 1 : len);
}

__device__ __forceinline__ int block_len(const int32_t* draft_len, int b, int L) {
  return draft_len ? min(max(draft_len[b], 0), L) : L;
}

template <typename T>
__global__ __launch_bounds__(kT) void k_vp_sums(const T* __restrict__ target,
                                                const T* __restrict__ draft,
                                                const int32_t* __restrict__ tokens,
                                                const int32_t* __restrict__ draft_len,
                                                const float* __restrict__ uniforms, int L, int V,
                                                int span, int parts, Sums* __restrict__ sums,
                                                int32_t* __restrict__ accept_len) {
  __shared__ Sums ws[kWavesV];
  const int b = blockIdx.x / parts, part = blockIdx.x - b * parts, tid = threadIdx.x;
  const int len = block_len(draft_len, b, L);
  const int n = accepted(target, draft, tokens, uniforms, len, b, L, V);
  const bool residual = n < len;
  const T* p = target + (int64_t(b) * (L + 1) + n) * V;
  const T* q = draft + (int64_t(b) * L + (residual ? n : 0)) * V;
  const int v0 = part * span, v1 = min(v0 + span, V);
  double sw = 0.0, sp = 0.0;
  for (int v = v0 + tid; v < v1; v += kT) {
    const double pv = clean(value(p, v));
    const double qv = residual ? clean(value(q, v)) : 0.0;
    sp += pv;
    sw += pv > qv ? pv - qv : 0.0;
  }
  sw = wave_sum(sw);
  sp = wave_sum(sp);
  if (lane_id() == 0) ws[tid / kWave] = Sums{sw, sp};
  __syncthreads();
  if (tid == 0) {
    Sums t = ws[0];
#pragma unroll
    for (int w = 1; w < kWavesV; ++w) {
      t.w += ws[w].w;
      t.p += ws[w].p;
    }
    sums[blockIdx.x] = t;
    if (part == 0) accept_len[b] = n;
  }
}

template <typename T>
__global__ __launch_bounds__(kT) void k_vp_draw(const T* __restrict__ target,
                                                const T* __restrict__ draft,
                                                const int32_t* __restrict__ draft_len,
                                                const float* __restrict__ uniforms, int L, int V,
                                                int span, int parts,
                                                const Sums* __restrict__ sums,
                                                const int32_t* __restrict__ accept_len,
                                                int32_t* __restrict__ next_token) {
  __shared__ Sums ps[kMaxParts];
  __shared__ double wtot[kWavesV];
  __shared__ double sbase, sgoal;
  __shared__ int spart, ssecond;
  __shared__ unsigned long long first_m[kWavesV], pos_m[kWavesV];
  const int b = blockIdx.x, tid = threadIdx.x;
  const int len = block_len(draft_len, b, L);
  const int n = accept_len[b];
  for (int i = tid; i < parts; i += kT) ps[i] = sums[int64_t(b) * parts + i];
  __syncthreads();
  if (tid == 0) {
    double tw = 0.0, tp = 0.0;
    for (int i = 0; i < parts; ++i) {
      tw += ps[i].w;
      tp += ps[i].p;
    }
    const bool residual = n < len && tw > 0.0;       // else p_n itself
    const double total = residual ? tw : tp;
    const double goal = double(uniforms[int64_t(b) * (L + 1) + L]) * total;
    double run = 0.0, base = 0.0;
    int at = -1;
    for (int i = 0; i < parts; ++i) {
      const double s = residual ? ps[i].w : ps[i].p;
      if (s > 0.0) {
        at = i;                                      // the last part with weight, failing a hit
        base = run;
        if (goal < run + s) break;
      }
      run += s;
    }
    spart = at;
    ssecond = residual;
    sbase = base;
    sgoal = goal;
  }
  __syncthreads();
  const int part = spart;
  if (part < 0) {                                    // no token has probability
    if (tid == 0) next_token[b] = -1;
    return;
  }
  const bool residual = ssecond != 0;
  const double goal = sgoal;
  const T* p = target + (int64_t(b) * (L + 1) + n) * V;
  const T* q = draft + (int64_t(b) * L + (residual ? n : 0)) * V;
  const int v0 = part * span, v1 = min(v0 + span, V);
  // thread t owns a run of `each` tokens, so thread order is token order
  const int each = (v1 - v0 + kT - 1) / kT;
  const int a0 = min(v0 + tid * each, v1), a1 = min(a0 + each, v1);
  auto weight = [&](int v) {
    const double pv = clean(value(p, v));
    const double qv = residual ? clean(value(q, v)) : 0.0;
    return pv > qv ? pv - qv : 0.0;
  };
  double own = 0.0;
  for (int v = a0; v < a1; ++v) own += weight(v);
  // exclusive prefix over threads
  double incl = own;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const double o = __shfl_up(incl, d);
    if (lane_id() >= d) incl += o;
  }
  if (lane_id() == kWave - 1) wtot[tid / kWave] = incl;
  __syncthreads();
  double before = sbase;
  for (int w = 0; w < tid / kWave; ++w) before += wtot[w];
  const bool pos = own > 0.0;
  const unsigned long long fm = __ballot(pos && goal < before + incl);
  const unsigned long long pm = __ballot(pos);
  if (lane_id() == 0) {
    first_m[tid / kWave] = fm;
    pos_m[tid / kWave] = pm;
  }
  __syncthreads();
  int claim = -1;
  for (int w = 0; w < kWavesV && claim < 0; ++w)
    if (first_m[w]) claim = w * kWave + __ffsll((long long)first_m[w]) - 1;
  for (int w = kWavesV - 1; w >= 0 && claim < 0; --w)      // rounding: the last with weight
    if (pos_m[w]) claim = w * kWave + 63 - __clzll((long long)pos_m[w]);
  if (tid == claim) {
    double run = before + incl - own;
    int last = -1;
    for (int v = a0; v < a1; ++v) {
      const double x = weight(v);
      if (x > 0.0) {
        last = v;
        run += x;
        if (run > goal) break;
      }
    }
    next_token[b] = last;
  }
}

template <typename T>
hipError_t launch_typed(const void* target, const void* draft, const int32_t* tokens,
                        const int32_t* draft_len, const float* uniforms, int B, int L, int V,
                        int32_t* accept_len, int32_t* next_token, void* workspace, hipStream_t s) {
  const int parts = parts_of(B, V);
  const int span = (V + parts - 1) / parts;
  Sums* sums = static_cast<Sums*>(workspace);
  const T* p = static_cast<const T*>(target);
  const T* q = static_cast<const T*>(draft);
  k_vp_sums<T><<<unsigned(B) * unsigned(parts), kT, 0, s>>>(p, q, tokens, draft_len, uniforms, L, V,
                                                            span, parts, sums, accept_len);
  k_vp_draw<T><<<unsigned(B), kT, 0, s>>>(p, q, draft_len, uniforms, L, V, span, parts, sums,
                                          accept_len, next_token);
  return hipGetLastError();
}

}  // namespace

// one pair of sums per block and part
size_t verify_probs_workspace_bytes(int B, int V) {
  return size_t(B) * parts_of(B, V) * sizeof(Sums);
}

hipError_t launch_verify_probs(const void* target, const void* draft, bool bf16,
                               const int32_t* tokens, const int32_t* draft_len,
                               const float* uniforms, int B, int L, int V, int32_t* accept_len,
                               int32_t* next_token, void* workspace, hipStream_t s) {
  return bf16 ? launch_typed<uint16_t>(target, draft, tokens, draft_len, uniforms, B, L, V,
                                       accept_len, next_token, workspace, s)
              : launch_typed<float>(target, draft, tokens, draft_len, uniforms, B, L, V, accept_len,
                                    next_token, workspace, s);
}

}  // namespace mxm
