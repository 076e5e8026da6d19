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
// values are exact there (differences up to 2^-53 of the larger), and a sum
// over a vocabulary of 2^18 is off by at most 2^-35 of itself, so a draw
// depends on the order of summation only where u_L falls within that of a
// boundary.  Sums run in a fixed order.
//
// Of the (L + 1) V probabilities of a block only the drafted tokens' entries
// and the two rows at position n are read.  Up to 8192 tokens a workgroup per
// block does it all, with its threads' weights in registers (64 blocks of 2048
// tokens 4.0 us, 3 of 8192 6.7).  Beyond that two launches: the sums of a row's
// parts, a wave each, by workgroups that each find n themselves (2 L loads,
// cheaper than a launch); then the draw, a workgroup per block, which finds the
// part that holds it and reads that one again, into registers.  One block of
// 152064 tokens takes 8.4 us and 64 of them in bf16 16.5, latency of the two
// launches' dependent loads for the most part; 1024 take 135, 4.6 TB/s, as fast
// as a large copy.  (A workgroup per block throughout takes over 16 us for one
// block and 150 for 1024.)
#include "a4.hpp"

namespace mxm {
namespace {

constexpr int kSplitT = 256;                   // threads of a summing workgroup
constexpr int kDrawT = 512;
constexpr int kOneT = 1024;                    // threads where one workgroup does it all
constexpr int kMaxParts = 256;
constexpr int kOwn = 8;                        // weights a thread holds in registers

// one launch, no workspace
bool is_small(int V) { return V <= kOneT * kOwn; }

// Parts per row where two launches are taken: about sixteen waves a CU, at
// least 512 tokens a wave, and no more in a part than the draw takes at once.
int parts_of(int B, int V) {
  int n = 4096 / B;
  const int most = (V + 511) / 512, least = (V + kDrawT * kOwn - 1) / (kDrawT * kOwn);
  n = n < most ? n : most;
  n = n > least ? n : least;
  n = (n + 3) / 4 * 4;                         // whole summing workgroups
  return n < kMaxParts ? n : kMaxParts;
}

// Elements per part: whole 16-byte vectors of either type.
__host__ __device__ __forceinline__ int span_of(int V, int parts) {
  return ((V + parts - 1) / parts + 7) & ~7;
}

__device__ __forceinline__ float value(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float value(const uint16_t* p, int64_t i) {
  return __uint_as_float(uint32_t(p[i]) << 16);
}

// A probability: what is not a positive finite number counts as none.
__device__ __forceinline__ float clean(float v) {
  return __float_as_uint(v) - 1u < 0x7f7fffffu ? v : 0.f;
}

// max(0, p - q), or p (q = 0)
__device__ __forceinline__ double weight(float p, float q) {
  return fmax(double(clean(p)) - double(clean(q)), 0.0);
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// W consecutive values from element i (a multiple of W of an aligned row).
template <int W>
__device__ __forceinline__ void load(const float* p, int i, float (&v)[W]) {
  if constexpr (W == 1) {
    v[0] = p[i];
  } else {
    const float4 x = *reinterpret_cast<const float4*>(p + i);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  }
}
template <int W>
__device__ __forceinline__ void load(const uint16_t* p, int i, float (&v)[W]) {
  if constexpr (W == 1) {
    v[0] = value(p, i);
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(p + i);
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(u[k] << 16);
      v[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
    }
  }
}

// The kOwn values from element i on; those from `end` on are 0.  vec: the row
// is aligned and `end` a multiple of the vector.
template <class T>
__device__ __forceinline__ void load_run(const T* p, int i, int end, bool vec, float (&v)[kOwn]) {
  constexpr int kW = 16 / int(sizeof(T));
#pragma unroll
  for (int k = 0; k < kOwn; ++k) v[k] = 0.f;
  if (vec) {
#pragma unroll
    for (int h = 0; h < kOwn; h += kW) {
      if (i + h < end) {
        float x[kW];
        load<kW>(p, i + h, x);
#pragma unroll
        for (int k = 0; k < kW; ++k) v[h + k] = x[k];
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < kOwn; ++k)
      if (i + k < end) v[k] = value(p, i + k);
  }
}

// One wave's sum of the weights of tokens v0 .. v1 - 1; q may be NULL (0).
// Loads of a round are issued together: a part's time is their latency.
template <int W, class T>
__device__ __forceinline__ double part_sum(const T* p, const T* q, int v0, int v1) {
  constexpr int kU = W == 1 ? 8 : 5;
  double s = 0.0;
  for (int base = v0; base < v1; base += kWave * W * kU) {
    float pv[kU][W], qv[kU][W];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = base + (u * kWave + lane_id()) * W;
#pragma unroll
      for (int k = 0; k < W; ++k) pv[u][k] = qv[u][k] = 0.f;
      if (i < v1) {
        load<W>(p, i, pv[u]);
        if (q) load<W>(q, i, qv[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int k = 0; k < W; ++k) s += weight(pv[u][k], qv[u][k]);
  }
  return wave_sum(s);
}

// The same, by whole vectors where the rows allow it (V a multiple of 8 for
// bf16, 4 for fp32, and aligned tensors: then every row and part is).
template <class T>
__device__ __forceinline__ double part_sum(const T* p, const T* q, int v0, int v1, bool vec) {
  return vec ? part_sum<16 / int(sizeof(T))>(p, q, v0, v1) : part_sum<1>(p, q, v0, v1);
}

// One block's inputs.
template <class T>
struct Block {
  const T* target;                             // [L+1, V]
  const T* draft;                              // [L, V]
  const int32_t* tokens;
  const float* u;
  int len, L, V;

  __device__ __forceinline__ Block(const T* t, const T* d, const int32_t* tok,
                                   const int32_t* draft_len, const float* uni, int b, int L_, int V_)
      : target(t + int64_t(b) * (L_ + 1) * V_), draft(d + int64_t(b) * L_ * V_),
        tokens(tok + int64_t(b) * L_), u(uni + int64_t(b) * (L_ + 1)),
        len(draft_len ? min(max(draft_len[b], 0), L_) : L_), L(L_), V(V_) {}

  // Accepted tokens (every wave computes it; uniform result).  The loads do
  // not wait for the block's length.
  __device__ __forceinline__ int accepted() const {
    const int lane = lane_id();
    bool fail = false;
    if (lane < L) {
      const int d = tokens[lane];
      const float ui = u[lane];
      const bool inside = d >= 0 && d < V;
      const int64_t at = int64_t(lane) * V + (inside ? d : 0);
      const double pd = clean(value(target, at)), qd = clean(value(draft, at));
      fail = lane < len && !(inside && double(ui) * qd < pd);
    }
    const unsigned long long m = __ballot(fail);
    return __builtin_amdgcn_readfirstlane(m ? __ffsll((long long)m) - 1 : len);
  }
  __device__ __forceinline__ const T* p(int n) const { return target + int64_t(n) * V; }
  __device__ __forceinline__ const T* q(int n) const {
    return n < len ? draft + int64_t(n) * V : nullptr;
  }
};

// Inclusive prefix sum over the workgroup's threads; tot: one double per wave.
template <int NT>
__device__ __forceinline__ double block_prefix(double v, double* tot) {
  const int lane = lane_id(), wave = threadIdx.x / kWave;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const double o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();                             // tot is free
  if (lane == kWave - 1) tot[wave] = v;
  __syncthreads();
  double before = 0.0;
#pragma unroll
  for (int w = 0; w < NT / kWave; ++w)
    if (w < wave) before += tot[w];
  return before + v;
}

// The first thread for which `hit`, failing that the last for which `pos`
// (a goal rounded onto the total), failing that -1.
template <int NT>
__device__ __forceinline__ int claim(bool hit, bool pos, unsigned long long* m, bool* is_hit = nullptr) {
  constexpr int kW = NT / kWave;
  const unsigned long long h = __ballot(hit), p = __ballot(pos);
  __syncthreads();
  if (lane_id() == 0) {
    m[threadIdx.x / kWave] = h;
    m[kW + threadIdx.x / kWave] = p;
  }
  __syncthreads();
  int c = -1;
#pragma unroll
  for (int w = kW - 1; w >= 0; --w)
    if (m[w]) c = w * kWave + __ffsll((long long)m[w]) - 1;
  if (is_hit) *is_hit = c >= 0;
  if (c >= 0) return c;
#pragma unroll
  for (int w = 0; w < kW; ++w)
    if (m[kW + w]) c = w * kWave + 63 - __clzll((long long)m[kW + w]);
  return c;
}

template <int NT>
struct DrawLds {
  double sum[kMaxParts];
  double tot[NT / kWave];
  unsigned long long mask[2 * (NT / kWave)];
  double base;
};

// The draw from max(0, p - q), the sums of its parts given in s.sum.
template <int NT, class T>
__device__ __forceinline__ int draw(const T* p, const T* q, int V, int parts, int span, float u,
                                    bool vec, DrawLds<NT>& s) {
  static_assert(NT >= kMaxParts, "one thread per part");
  const int tid = threadIdx.x;
  for (;;) {
    const double own = tid < parts ? s.sum[tid] : 0.0;
    const double incl = block_prefix<NT>(own, s.tot);
    double total = 0.0;
#pragma unroll
    for (int w = 0; w < NT / kWave; ++w) total += s.tot[w];
    if (!(total > 0.0)) {
      if (!q) return -1;                       // no token has probability
      q = nullptr;                             // no difference: from p itself
      __syncthreads();
      for (int k = tid / kWave; k < parts; k += NT / kWave) {
        const double t = part_sum(p, q, min(k * span, V), min((k + 1) * span, V), vec);
        if (lane_id() == 0) s.sum[k] = t;
      }
      __syncthreads();
      continue;
    }
    const double goal = double(u) * total;
    const int part = claim<NT>(own > 0.0 && goal < incl, own > 0.0, s.mask);
    if (tid == part) s.base = incl - own;
    __syncthreads();
    // NT kOwn of the part's tokens at a time; a thread owns a run of kOwn, so
    // thread order is token order
    double base = s.base;
    const int v1 = min((part + 1) * span, V);
    int found = -1;
    for (int v0 = min(part * span, V); v0 < v1; v0 += NT * kOwn) {
      const int a0 = v0 + tid * kOwn;
      float pv[kOwn], qv[kOwn];
      load_run(p, a0, v1, vec, pv);
      load_run(q, a0, q ? v1 : 0, vec, qv);
      double run = 0.0;
#pragma unroll
      for (int k = 0; k < kOwn; ++k) run += weight(pv[k], qv[k]);
      const double end = base + block_prefix<NT>(run, s.tot);
      bool hit;
      const int c = claim<NT>(run > 0.0 && goal < end, run > 0.0, s.mask, &hit);
      if (c >= 0) found = -1;                  // a later token than any before
      if (tid == c) {
        double at = end - run;
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
          const double x = weight(pv[k], qv[k]);
          if (x > 0.0 && (found < 0 || !(at > goal))) {
            found = a0 + k;
            at += x;
          }
        }
      }
      if (hit) break;
#pragma unroll
      for (int w = 0; w < NT / kWave; ++w) base += s.tot[w];
    }
    return found;                              // one thread's alone
  }
}

template <class T>
__global__ __launch_bounds__(kSplitT) void k_vp_sums(
    const T* __restrict__ target, const T* __restrict__ draft, const int32_t* __restrict__ tokens,
    const int32_t* __restrict__ draft_len, const float* __restrict__ uniforms, int L, int V,
    int parts, int span, bool vec, double* __restrict__ sums, int32_t* __restrict__ accept_len) {
  const int groups = parts / (kSplitT / kWave);
  const int b = blockIdx.x / groups;
  const int part = (blockIdx.x - b * groups) * (kSplitT / kWave) + threadIdx.x / kWave;
  const Block<T> blk(target, draft, tokens, draft_len, uniforms, b, L, V);
  const int n = blk.accepted();
  const double s = part_sum(blk.p(n), blk.q(n), min(part * span, V), min((part + 1) * span, V), vec);
  if (lane_id() == 0) {
    sums[int64_t(b) * parts + part] = s;
    if (part == 0) accept_len[b] = n;
  }
}

template <class T>
__global__ __launch_bounds__(kDrawT) void k_vp_draw(
    const T* __restrict__ target, const T* __restrict__ draft, const int32_t* __restrict__ tokens,
    const int32_t* __restrict__ draft_len, const float* __restrict__ uniforms, int L, int V,
    int parts, int span, bool vec, const double* __restrict__ sums,
    const int32_t* __restrict__ accept_len, int32_t* __restrict__ next_token) {
  __shared__ DrawLds<kDrawT> s;
  const int b = blockIdx.x;
  const Block<T> blk(target, draft, tokens, draft_len, uniforms, b, L, V);
  const int n = accept_len[b];
  if (int(threadIdx.x) < parts) s.sum[threadIdx.x] = sums[int64_t(b) * parts + threadIdx.x];
  __syncthreads();
  const int t = draw<kDrawT>(blk.p(n), blk.q(n), V, parts, span, blk.u[L], vec, s);
  const bool any = __syncthreads_or(t >= 0);
  if (t >= 0 || (!any && threadIdx.x == 0)) next_token[b] = t;
}

// One workgroup per block and at most kOwn tokens per thread: thread t owns a
// run of them, so thread order is token order and one prefix sum finds the
// draw.
template <int NT, class T>
__global__ __launch_bounds__(NT) void k_vp_own(
    const T* __restrict__ target, const T* __restrict__ draft, const int32_t* __restrict__ tokens,
    const int32_t* __restrict__ draft_len, const float* __restrict__ uniforms, int L, int V,
    int each, bool vec, int32_t* __restrict__ accept_len, int32_t* __restrict__ next_token) {
  __shared__ double tot[NT / kWave];
  __shared__ unsigned long long mask[2 * (NT / kWave)];
  const int b = blockIdx.x, tid = threadIdx.x;
  const Block<T> blk(target, draft, tokens, draft_len, uniforms, b, L, V);
  const float u = blk.u[L];
  const int n = blk.accepted();
  const T* p = blk.p(n);
  const T* q = blk.q(n);
  const int a0 = min(tid * each, V), a1 = min(a0 + each, V);
  float pv[kOwn], qv[kOwn];
  load_run(p, a0, a1, vec, pv);
  load_run(q, a0, q ? a1 : 0, vec, qv);
  if (tid == 0) accept_len[b] = n;
  bool residual = q != nullptr;
  for (;;) {
    double run = 0.0;
#pragma unroll
    for (int k = 0; k < kOwn; ++k) run += weight(pv[k], residual ? qv[k] : 0.f);
    const double incl = block_prefix<NT>(run, tot);
    double total = 0.0;
#pragma unroll
    for (int k = 0; k < NT / kWave; ++k) total += tot[k];
    if (!(total > 0.0)) {
      if (!residual) {                         // no token has probability
        if (tid == 0) next_token[b] = -1;
        return;
      }
      residual = false;                        // no difference: from p itself
      continue;
    }
    const double goal = double(u) * total;
    const int c = claim<NT>(run > 0.0 && goal < incl, run > 0.0, mask);
    if (tid == c) {
      int found = -1;
      double at = incl - run;
#pragma unroll
      for (int k = 0; k < kOwn; ++k) {
        const double x = weight(pv[k], residual ? qv[k] : 0.f);
        if (x > 0.0 && (found < 0 || !(at > goal))) {
          found = a0 + k;
          at += x;
        }
      }
      next_token[b] = found;
    }
    return;
  }
}

template <class T>
hipError_t launch_typed(const void* target, const void* draft, const int32_t* tokens,
                        const int32_t* draft_len, const float* uniforms, int B, int L, int V,
                        int32_t* accept_len, int32_t* next_token, void* workspace, hipStream_t s) {
  const T* p = static_cast<const T*>(target);
  const T* q = static_cast<const T*>(draft);
  const bool vec = V % (16 / int(sizeof(T))) == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(q) % 16 == 0;
  if (is_small(V)) {
    // whole vectors a thread, or as few tokens as there are threads for
    const bool few = V <= kSplitT * kOwn;
    const int nt = few ? kSplitT : kOneT;
    (few ? k_vp_own<kSplitT, T> : k_vp_own<kOneT, T>)<<<unsigned(B), unsigned(nt), 0, s>>>(
        p, q, tokens, draft_len, uniforms, L, V, vec ? kOwn : (V + nt - 1) / nt, vec, accept_len,
        next_token);
    return hipGetLastError();
  }
  const int parts = parts_of(B, V), span = span_of(V, parts);
  double* sums = static_cast<double*>(workspace);
  const unsigned groups = unsigned(parts / (kSplitT / kWave));
  k_vp_sums<T><<<unsigned(B) * groups, kSplitT, 0, s>>>(p, q, tokens, draft_len, uniforms, L, V,
                                                        parts, span, vec, sums, accept_len);
  k_vp_draw<T><<<unsigned(B), kDrawT, 0, s>>>(p, q, tokens, draft_len, uniforms, L, V, parts, span,
                                              vec, sums, accept_len, next_token);
  return hipGetLastError();
}

}  // namespace

// the parts' sums, where two launches are taken
size_t verify_probs_workspace_bytes(int B, int V) {
  return is_small(V) ? 0 : size_t(B) * parts_of(B, V) * sizeof(double);
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
