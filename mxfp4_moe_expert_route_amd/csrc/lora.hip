// Low-rank adapters of many requests: t = A_s x, then y += scale_s B_s t.
//
// Rows come grouped by adapter (the lists of moe_permute), so a tile of rows
// has one adapter and both steps are small matrix products on
// v_mfma_f32_16x16x32_bf16.
#include "lora.hpp"

namespace mxm {
namespace {

constexpr int kWaves = 4;
constexpr int kCols = 64;            // columns of y a wave holds at a time

// rank padded to a size that the kernels are made for
int padded(int r) { return r <= 8 ? 8 : r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }

int tile_rows(const LoraProblem& p) {
  const int mean = p.M / (p.M < p.S ? p.M : p.S);
  return mean <= 16 ? 1 : mean <= 32 || p.r > 64 ? 2 : 4;
}

int64_t most_tiles(const LoraProblem& p, int mt) {
  const int64_t n = p.M / mt + int64_t(p.S);
  return n < p.M ? n : p.M;
}

// pieces of K, one workgroup each
int k_splits(const LoraProblem& p) {
  const int64_t tiles = most_tiles(p, 16 * tile_rows(p));
  int n = 1;
  while (n < 16 && tiles * n < 512 && p.K >= 2 * n * 256) n *= 2;
  return n;
}

__device__ __forceinline__ f32x4 mfma(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}

// The row of y and x at sorted position pos, or -1.
__device__ __forceinline__ int row_at(const LoraProblem& p, const Tile& t, int i) {
  const int pos = t.row0 + i;
  if (i >= t.rows || unsigned(pos) >= unsigned(p.M)) return -1;
  const int row = p.rows[pos];
  return unsigned(row) < unsigned(p.M) ? row : -1;
}

// t = A_s x for a tile of 16 MS rows and one piece of K.  The workgroup's waves
// take steps of 32 of K in turn and add up through LDS.  Of an operand lane
// 16 g + i holds row i (of A: operand A, of x: operand B), K 8 g .. 8 g + 7; lane
// 16 g + c of the result holds ranks 4 g .. 4 g + 3 of row c.
template <int RP, int MS>
__global__ __launch_bounds__(kWaves * kWave) void k_lora_shrink(LoraProblem p, int piece) {
  constexpr int NR = (RP + 15) / 16;
  __shared__ __attribute__((aligned(16))) float red[kWaves - 1][MS * 16][NR * 16];
  Tile t;
  if (!find_tile(p.offsets, p.S, 16 * MS, blockIdx.x, t)) return;
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  const uint16_t* xr[MS];
#pragma unroll
  for (int m = 0; m < MS; ++m) xr[m] = p.x + size_t(max(row_at(p, t, 16 * m + c), 0)) * p.K + 8 * g;
  const uint16_t* ar[NR];
#pragma unroll
  for (int j = 0; j < NR; ++j)
    ar[j] = p.a + (size_t(t.e) * p.r + min(16 * j + c, p.r - 1)) * p.K + 8 * g;
  f32x4 acc[MS][NR];
#pragma unroll
  for (int m = 0; m < MS; ++m)
#pragma unroll
    for (int j = 0; j < NR; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int k1 = min(p.K, int(blockIdx.y + 1) * piece);
  for (int k = blockIdx.y * piece + 32 * wave; k < k1; k += 32 * kWaves) {
    const bool in = k + 8 * g < k1;
    const int kk = in ? k : 0;
    uint4 xv[MS], av[NR];
#pragma unroll
    for (int m = 0; m < MS; ++m) {
      const uint4 v = *reinterpret_cast<const uint4*>(xr[m] + (in ? kk : -8 * g));
      xv[m] = in ? v : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      const uint4 v = *reinterpret_cast<const uint4*>(ar[j] + (in ? kk : -8 * g));
      av[j] = in && 16 * j + c < p.r ? v : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int m = 0; m < MS; ++m)
#pragma unroll
      for (int j = 0; j < NR; ++j) acc[m][j] = mfma(av[j], xv[m], acc[m][j]);
  }
  if (wave > 0) {
#pragma unroll
    for (int m = 0; m < MS; ++m)
#pragma unroll
      for (int j = 0; j < NR; ++j)
        *reinterpret_cast<f32x4*>(&red[wave - 1][16 * m + c][16 * j + 4 * g]) = acc[m][j];
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int m = 0; m < MS; ++m) {
    const int i = 16 * m + c;
    const int pos = t.row0 + i;
    const bool ok = i < t.rows && unsigned(pos) < unsigned(p.M);
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      f32x4 v = acc[m][j];
#pragma unroll
      for (int w = 0; w < kWaves - 1; ++w)
        v += *reinterpret_cast<const f32x4*>(&red[w][i][16 * j + 4 * g]);
      if (ok && 16 * j + 4 * g < RP)
        *reinterpret_cast<f32x4*>(p.part + (size_t(blockIdx.y) * p.M + pos) * RP + 16 * j + 4 * g) = v;
    }
  }
}

// Eight elements of row n of B from rank 8 q on; 0 past the rank.
template <bool VEC>
__device__ __forceinline__ uint4 load_b(const uint16_t* row, int q, int r) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if constexpr (VEC) {
    if (8 * q < r) v = *reinterpret_cast<const uint4*>(row + 8 * q);
  } else {
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = 8 * q + i < r ? row[8 * q + i] : 0;
    v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
  }
  return v;
}

// y += scale B_s t for a tile of 16 MS rows and 64 columns a wave.  t is fp32
// and B bf16: t is cut into three bf16 of 8 bits each by truncation, which is
// exact, and the three meet the same B along the instruction's K: octet q of K
// is octet q % (RP / 8) of the rank in part q / (RP / 8).  Product j of four
// takes the columns 16 (i / 4) + 4 j + i % 4 as its rows i, so lane 16 g + c ends
// with the 16 columns from 16 g on of row c.
template <int RP, int MS, bool BF16, bool VECB, bool VECY>
__global__ __launch_bounds__(kWaves * kWave) void k_lora_expand(LoraProblem p, int splits) {
  constexpr int OCT = RP / 8, NM = (3 * OCT + 3) / 4;
  constexpr int LD = 32 * NM + 8;                // bf16 a row in LDS
  __shared__ __attribute__((aligned(16))) uint16_t ts[MS * 16][LD];
  Tile t;
  if (!find_tile(p.offsets, p.S, 16 * MS, blockIdx.x, t)) return;
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  const float scale = p.scale ? p.scale[t.e] : 1.f;
  for (int i = threadIdx.x; i < MS * 16 * RP; i += kWaves * kWave) {
    const int row = i / RP, j = i % RP, pos = t.row0 + row;
    float v = 0.f;
    // past the rank an infinite x times the padding's 0 is NaN
    if (j < p.r && row < t.rows && unsigned(pos) < unsigned(p.M))
      for (int s = 0; s < splits; ++s) v += p.part[(size_t(s) * p.M + pos) * RP + j];
    v *= scale;
    const uint32_t hi = __float_as_uint(v) & 0xffff0000u;
    // an infinite or NaN t has no parts below
    const bool fin = (hi & 0x7f800000u) != 0x7f800000u;
    const float rest = fin ? v - __uint_as_float(hi) : 0.f;
    const uint32_t mid = __float_as_uint(rest) & 0xffff0000u;
    const float low = rest - __uint_as_float(mid);
    ts[row][j] = uint16_t(hi >> 16);
    ts[row][RP + j] = uint16_t(mid >> 16);
    ts[row][2 * RP + j] = uint16_t(__float_as_uint(low) >> 16);
  }
  if constexpr (3 * RP < 32 * NM) {
    for (int i = threadIdx.x; i < MS * 16 * (32 * NM - 3 * RP); i += kWaves * kWave)
      ts[i / (32 * NM - 3 * RP)][3 * RP + i % (32 * NM - 3 * RP)] = 0;
  }
  __syncthreads();
  int row[MS];
#pragma unroll
  for (int m = 0; m < MS; ++m) row[m] = row_at(p, t, 16 * m + c);
  for (int n0 = (blockIdx.y * kWaves + wave) * kCols; n0 < p.N; n0 += gridDim.y * kWaves * kCols) {
    f32x4 acc[MS][4];
#pragma unroll
    for (int m = 0; m < MS; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = min(n0 + 16 * (c >> 2) + 4 * j + (c & 3), p.N - 1);
      const uint16_t* br = p.b + (size_t(t.e) * p.N + n) * p.r;
#pragma unroll
      for (int q = 0; q < NM; ++q) {
        const int oct = 4 * q + g;
        const uint4 bv = oct < 3 * OCT ? load_b<VECB>(br, oct % OCT, p.r) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int m = 0; m < MS; ++m)
          acc[m][j] = mfma(bv, *reinterpret_cast<const uint4*>(&ts[16 * m + c][32 * q + 8 * g]), acc[m][j]);
      }
    }
#pragma unroll
    for (int m = 0; m < MS; ++m) {
      if (row[m] < 0) continue;
      const int n = n0 + 16 * g;
      if constexpr (BF16) {
        uint16_t* y = static_cast<uint16_t*>(p.y) + size_t(row[m]) * p.N + n;
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const float d[8] = {acc[m][j][0], acc[m][j][1], acc[m][j][2], acc[m][j][3],
                              acc[m][j + 1][0], acc[m][j + 1][1], acc[m][j + 1][2], acc[m][j + 1][3]};
          if (VECY) {
            if (n + 4 * j >= p.N) continue;
            uint4 v = *reinterpret_cast<const uint4*>(y + 4 * j);
            uint32_t* u = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              u[q] = f32_to_bf16_rne(__uint_as_float(u[q] << 16) + d[2 * q]) |
                     f32_to_bf16_rne(__uint_as_float(u[q] & 0xffff0000u) + d[2 * q + 1]) << 16;
            *reinterpret_cast<uint4*>(y + 4 * j) = v;
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (n + 4 * j + q < p.N)
                y[4 * j + q] = uint16_t(f32_to_bf16_rne(__uint_as_float(uint32_t(y[4 * j + q]) << 16) + d[q]));
          }
        }
      } else {
        float* y = static_cast<float*>(p.y) + size_t(row[m]) * p.N + n;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (VECY) {
            if (n + 4 * j < p.N) *reinterpret_cast<f32x4*>(y + 4 * j) += acc[m][j];
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (n + 4 * j + q < p.N) y[4 * j + q] += acc[m][j][q];
          }
        }
      }
    }
  }
}

template <int RP, int MS>
hipError_t launch(const LoraProblem& p, hipStream_t s) {
  const unsigned tiles = unsigned(most_tiles(p, 16 * MS));
  const int splits = k_splits(p);
  const int unit = 32 * kWaves;
  const int piece = ((p.K + splits - 1) / splits + unit - 1) / unit * unit;
  k_lora_shrink<RP, MS><<<dim3(tiles, splits), kWaves * kWave, 0, s>>>(p, piece);
  // a launch has fewer than 2^32 threads: workgroups go on to further columns
  const unsigned cols = unsigned((p.N + kWaves * kCols - 1) / (kWaves * kCols));
  const unsigned most = (1u << 23) / tiles;
  const dim3 grid(tiles, cols < most ? cols : most);
  const bool vb = p.r % 8 == 0;
  const bool vy = (p.N * (p.bf16 ? 2 : 4)) % 16 == 0 && reinterpret_cast<uintptr_t>(p.y) % 16 == 0;
  auto go = [&](auto bf, auto vecb, auto vecy) {
    k_lora_expand<RP, MS, decltype(bf)::value, decltype(vecb)::value, decltype(vecy)::value>
        <<<grid, kWaves * kWave, 0, s>>>(p, splits);
  };
  const std::true_type yes;
  const std::false_type no;
  if (p.bf16) {
    if (vb) { if (vy) go(yes, yes, yes); else go(yes, yes, no); }
    else { if (vy) go(yes, no, yes); else go(yes, no, no); }
  } else {
    if (vb) { if (vy) go(no, yes, yes); else go(no, yes, no); }
    else { if (vy) go(no, no, yes); else go(no, no, no); }
  }
  return hipGetLastError();
}

template <int RP>
hipError_t launch_r(const LoraProblem& p, hipStream_t s) {
  const int ms = tile_rows(p);
  if (ms == 1) return launch<RP, 1>(p, s);
  if (ms == 2) return launch<RP, 2>(p, s);
  return launch<RP, RP == 128 ? 2 : 4>(p, s);
}

}  // namespace

size_t lora_workspace_bytes(int M, int K, int N, int S, int r) {
  LoraProblem p{};
  p.M = M; p.K = K; p.N = N; p.S = S; p.r = r;
  return size_t(k_splits(p)) * M * padded(r) * sizeof(float);
}

hipError_t launch_lora(const LoraProblem& p, hipStream_t s) {
  switch (padded(p.r)) {
    case 8: return launch_r<8>(p, s);
    case 16: return launch_r<16>(p, s);
    case 32: return launch_r<32>(p, s);
    case 64: return launch_r<64>(p, s);
    default: return launch_r<128>(p, s);
  }
}

}  // namespace mxm
