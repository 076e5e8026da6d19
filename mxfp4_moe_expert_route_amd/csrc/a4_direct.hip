// Contractions of two MXFP4 factors without staging: every wave loads its
// operands from memory straight into the registers of the scaled matrix
// instructions.  Takes every shape.
//
// A unit is 16 CF output columns x 16 MS rows over the whole of K.  Where K is
// long (SPLIT) a workgroup's eight waves deal its 256-element chunks (a chunk
// is one 128-byte line of codes per row) among themselves and their partial
// sums meet in LDS, added in wave order, so results do not depend on timing:
// splitting K rather than the columns keeps every byte of a unit in flight at
// once, and with few rows the cost is the latency of the weight bytes, not
// their number (8 x 4096 x 6144: 5 us for 12.6 MB).  Where K is a few chunks,
// each wave has a unit to itself.
#include "a4.hpp"
#include "mx_pack.hpp"

namespace mxm {
namespace a4 {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * kWave;
constexpr int kChunkBlocks = 8;                // MX blocks per chunk (256 of K)
// K in one chunk is one wave's work; up to four are where there are units for
// half the waves the GPU holds (a long K goes faster split, 2785 x 29 x 544 in
// 3.2 instead of 5.6 us; many short units alone, 1272 x 2927 x 192 in 7.4
// instead of 20)
constexpr int kAloneChunks = 4;
constexpr int kAloneUnits = 1024;

template <bool LINES>
struct Frag {
  uint4 c[2];            // this lane's blocks g and 4 + g of the chunk
  uint32_t s[2];         // and their scale bytes
};

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

// Store at an address aligned to its elements alone (a row may start anywhere).
// T is a vector type of the compiler: a class such as uint2 is not packed.
template <class T>
__device__ __forceinline__ void store_any(void* p, const T& v) {
  struct __attribute__((packed, aligned(2))) U {
    T v;
  };
  static_assert(alignof(U) == 2, "the store may not claim more alignment than it has");
  static_cast<U*>(p)->v = v;
}

// Chunk `ch` of the row at (codes, scales).  LINES: K is whole chunks and the
// scale rows are 8-byte aligned.  Blocks past the end of K load as zeros under
// scale 1: they add nothing, whatever the other factor holds.
template <bool LINES>
__device__ __forceinline__ Frag<LINES> load_frag(const uint8_t* codes, const uint8_t* scales,
                                                 int ch, int nblk) {
  const int g = lane_id() >> 4;
  Frag<LINES> f;
  if constexpr (LINES) {
    f.c[0] = *reinterpret_cast<const uint4*>(codes + 128 * int64_t(ch) + 16 * g);
    f.c[1] = *reinterpret_cast<const uint4*>(codes + 128 * int64_t(ch) + 64 + 16 * g);
    const uint2 s = *reinterpret_cast<const uint2*>(scales + 8 * ch);
    f.s[0] = s.x >> (8 * g);
    f.s[1] = s.y >> (8 * g);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int b = kChunkBlocks * ch + 4 * h + g;
      const int bc = min(b, nblk - 1);
      f.c[h] = *reinterpret_cast<const uint4*>(codes + 16 * int64_t(bc));
      f.s[h] = scales[bc];
      if (b >= nblk) {
        f.c[h] = make_uint4(0u, 0u, 0u, 0u);
        f.s[h] = 127u;
      }
    }
  }
  return f;
}

// CF: 16-column groups per unit; MS: 16-row groups per unit.
template <Kind KIND, Out OUT, int CF, int MS, bool LINES, bool SPLIT>
__global__ __launch_bounds__(kThreads) void k_direct(Problem p) {
  constexpr int WF = KIND == kGateUp ? 2 * CF : CF;        // weight fragments
  __shared__ f32x4 part[SPLIT ? kWaves : 1][SPLIT ? WF * MS : 1][kWave];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = lane_id();
  const int r16 = lane & 15, g = lane >> 4;
  const int nblk = p.K / 32;
  const int64_t crow = p.K / 2;
  const int nch = (nblk + kChunkBlocks - 1) / kChunkBlocks;
  const int ncol = (p.N + 16 * CF - 1) / (16 * CF);

  const int64_t first = SPLIT ? int64_t(blockIdx.x) : int64_t(blockIdx.x) * kWaves + wave;
  const int64_t stride = SPLIT ? int64_t(gridDim.x) : int64_t(gridDim.x) * kWaves;
  for (int64_t slot = first;; slot += stride) {
    const int tau = int(slot / ncol);
    const int n0 = int(slot - int64_t(tau) * ncol) * 16 * CF;
    Tile t;
    if constexpr (KIND == kGemm) {
      t.e = 0;
      t.row0 = tau * 16 * MS;
      t.rows = min(16 * MS, p.M - t.row0);
      if (t.rows <= 0) break;
    } else {
      if (!find_tile(p.offsets, p.E, 16 * MS, tau, t, p.lo, p.hi)) break;
    }

    const uint8_t* xc[MS];
    const uint8_t* xs[MS];
#pragma unroll
    for (int m = 0; m < MS; ++m) {
      int64_t row = t.row0 + min(16 * m + r16, t.rows - 1);
      if constexpr (KIND == kGateUp) row = p.pairs[row] / p.k;
      xc[m] = p.xc + row * crow;
      xs[m] = p.xs + row * nblk;
    }
    const uint8_t* wc[WF];
    const uint8_t* ws[WF];
#pragma unroll
    for (int a = 0; a < WF; ++a) {
      const int n = min(n0 + 16 * (a % CF) + r16, p.N - 1);
      const int64_t row = KIND == kGateUp ? (int64_t(t.e) * 2 + a / CF) * p.N + n
                                          : int64_t(t.e) * p.N + n;
      wc[a] = p.wc + row * crow;
      ws[a] = p.ws + row * nblk;
    }

    f32x4 acc[WF][MS];
#pragma unroll
    for (int a = 0; a < WF; ++a)
#pragma unroll
      for (int m = 0; m < MS; ++m) acc[a][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int ch = SPLIT ? wave : 0; ch < nch; ch += SPLIT ? kWaves : 1) {
      Frag<LINES> w[WF], x[MS];
#pragma unroll
      for (int a = 0; a < WF; ++a) w[a] = load_frag<LINES>(wc[a], ws[a], ch, nblk);
#pragma unroll
      for (int m = 0; m < MS; ++m) x[m] = load_frag<LINES>(xc[m], xs[m], ch, nblk);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int a = 0; a < WF; ++a)
#pragma unroll
          for (int m = 0; m < MS; ++m)
            acc[a][m] = mfma(w[a].c[h], w[a].s[h], x[m].c[h], x[m].s[h], acc[a][m]);
    }
    if constexpr (SPLIT) {
#pragma unroll
      for (int a = 0; a < WF; ++a)
#pragma unroll
        for (int m = 0; m < MS; ++m) part[wave][a * MS + m][lane] = acc[a][m];
      __syncthreads();
    }

    // lane: columns 4g .. 4g+3 of row r16; a split unit's row groups are dealt
    // over the waves
    auto total = [&](int a, int m) {
      if constexpr (SPLIT) {
        f32x4 v = part[0][a * MS + m][lane];
#pragma unroll
        for (int q = 1; q < kWaves; ++q) v += part[q][a * MS + m][lane];
        return v;
      } else {
        return acc[a][m];
      }
    };
#pragma unroll
    for (int m = 0; m < MS; ++m) {
      if (SPLIT && m % kWaves != wave) continue;
      const int64_t row = int64_t(t.row0) + 16 * m + r16;
      const bool live = 16 * m + r16 < t.rows;
      if constexpr (OUT == kMx) {
        static_assert(OUT != kMx || CF == 2, "an MX block is two 16-column groups");
        // h rounded to bf16, then packed: the block's 32 columns are this
        // lane's eight and those of lanes +-16, +-32
        uint32_t v[2][4];
        uint32_t amax = 0;
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const f32x4 gv = total(a, m), uv = total(a + CF, m);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[a][i] = f32_to_bf16_rne(silu_mul(gv[i], uv[i])) << 16;
            amax = max(amax, v[a][i] & 0x7fffffffu);
          }
        }
        amax = max(amax, uint32_t(__shfl_xor(int(amax), 16)));
        amax = max(amax, uint32_t(__shfl_xor(int(amax), 32)));
        const bool bad = amax >= 0x7f800000u;            // Inf or NaN in the block
        const uint32_t e = bad ? 255u : mx_scale_byte(amax);
        const MxThresholds th(bad ? 0u : e);
        if (live) {
          uint8_t* oc = p.oc + row * (p.N / 2) + n0 / 2;
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            uint32_t c = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) c |= th.code(v[a][i]) << (4 * i);
            *reinterpret_cast<uint16_t*>(oc + 8 * a + 2 * g) = uint16_t(bad ? 0u : c);
          }
          if (g == 0) p.os[row * (p.N / 32) + n0 / 32] = uint8_t(e);
        }
      } else {
#pragma unroll
        for (int a = 0; a < CF; ++a) {
          f32x4 v = total(a, m);
          if constexpr (KIND == kGateUp) {
            const f32x4 u = total(a + CF, m);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = silu_mul(v[i], u[i]);
          }
          if (!live) continue;
          const int n = n0 + 16 * a + 4 * g;
          if constexpr (OUT == kF32) {
            float* o = static_cast<float*>(p.out) + row * p.N + n;
            if (n + 4 <= p.N) {
              store_any(o, v);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (n + i < p.N) o[i] = v[i];
            }
          } else {
            uint16_t* o = static_cast<uint16_t*>(p.out) + row * p.N + n;
            uint32_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = f32_to_bf16_rne(v[i]);
            if (n + 4 <= p.N) {
              store_any(o, u32x2{b[0] | (b[1] << 16), b[2] | (b[3] << 16)});
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (n + i < p.N) o[i] = uint16_t(b[i]);
            }
          }
        }
      }
    }
    if constexpr (SPLIT) __syncthreads();      // the sums are read: LDS is free
  }
}

template <Kind KIND, Out OUT, int CF, int MS>
hipError_t launch(const Problem& p, hipStream_t s) {
  const bool lines = p.K % 256 == 0 && reinterpret_cast<uintptr_t>(p.xs) % 8 == 0 &&
                     reinterpret_cast<uintptr_t>(p.ws) % 8 == 0;
  const int64_t ncol = (p.N + 16 * CF - 1) / (16 * CF);
  // row tiles: exact for a product, at most one partial tile per expert else
  const int64_t full = p.R / (16 * MS);
  const int64_t tiles = KIND == kGemm ? (int64_t(p.M) + 16 * MS - 1) / (16 * MS)
                                      : full + (p.R < p.E ? p.R : p.E);
  const int64_t slots = tiles * ncol;
  const int64_t chunks = (p.K + 255) / 256;
  const bool split = chunks > kAloneChunks || (chunks > 1 && slots <= kAloneUnits);
  const int64_t groups = split ? slots : (slots + kWaves - 1) / kWaves;
  const int64_t cap = int64_t(device_cus()) * 4;
  const unsigned grid = unsigned(groups < cap ? groups : cap);
  if (split) {
    if (lines) k_direct<KIND, OUT, CF, MS, true, true><<<grid, kThreads, 0, s>>>(p);
    else k_direct<KIND, OUT, CF, MS, false, true><<<grid, kThreads, 0, s>>>(p);
  } else {
    if (lines) k_direct<KIND, OUT, CF, MS, true, false><<<grid, kThreads, 0, s>>>(p);
    else k_direct<KIND, OUT, CF, MS, false, false><<<grid, kThreads, 0, s>>>(p);
  }
  return hipGetLastError();
}

template <Out OUT>
hipError_t launch_gemm(const Problem& p, int cf, int ms, hipStream_t s) {
  if (cf == 1) return ms == 1 ? launch<kGemm, OUT, 1, 1>(p, s) : launch<kGemm, OUT, 1, 2>(p, s);
  return ms == 2 ? launch<kGemm, OUT, 2, 2>(p, s) : launch<kGemm, OUT, 2, 4>(p, s);
}

}  // namespace

hipError_t launch_direct(Kind kind, Out out, const Problem& p, int ms, hipStream_t s) {
  if (kind == kDown) return ms == 1 ? launch<kDown, kF32, 1, 1>(p, s) : launch<kDown, kF32, 1, 4>(p, s);
  if (out == kMx)
    return ms == 1 ? launch<kGateUp, kMx, 2, 1>(p, s) : launch<kGateUp, kMx, 2, 2>(p, s);
  return ms == 1 ? launch<kGateUp, kBf16, 1, 1>(p, s) : launch<kGateUp, kBf16, 1, 4>(p, s);
}

hipError_t launch_direct_gemm(Out out, const Problem& p, int cf, int ms, hipStream_t s) {
  return out == kBf16 ? launch_gemm<kBf16>(p, cf, ms, s) : launch_gemm<kF32>(p, cf, ms, s);
}

}  // namespace a4
}  // namespace mxm
