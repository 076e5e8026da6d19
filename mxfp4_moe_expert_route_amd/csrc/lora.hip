// Low-rank adapters of many requests: t = A_s x, then y += scale_s B_s t.
//
// Rows come grouped by adapter (the lists of moe_permute), so a tile of rows
// has one adapter and both steps are small matrix products on
// v_mfma_f32_16x16x32_bf16.  Operations are few (2 r (K + N) a row); what counts is
// the bytes of x and y for many rows, of A and B for few, and for the smallest calls
// the launch.  8 rows of K = 6144, N = 4096, rank 16: 8.6 us, a launch and a chain of
// four loads; 8192 rows of rank 64: 50 us where the caches hold x and y, 70 (3.4 TB/s)
// where they do not.
#include "lora.hpp"

namespace mxm {
namespace {

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2v;

constexpr int kWaves = 4;
constexpr int kCols = 64;            // columns of y a wave holds at a time

// rank padded to a size that the kernels are made for
int padded(int r) { return r <= 8 ? 8 : r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }

int64_t most_tiles(const LoraProblem& p, int rows) {
  const int64_t n = p.M / rows + int64_t(p.S);
  return n < p.M ? n : p.M;
}

int padded_tiles(int r) { return (padded(r) + 15) / 16; }

// Rows of a tile for the kernel that takes both steps, whose workgroups have a CU to
// themselves: as few as fill the chip once, or twice, ..., where every adapter's
// last tile may be nearly empty, and 48 at most; or 16, where fewer would do.  A
// tile more than the chip holds costs another round: 8192 rows of 8 adapters by
// chance, rank 64, tiles of 32 rows 106 us, of 34 75; of 64 adapters 126 and 82.
constexpr int kCus = 256;
constexpr int kMostRows = 48;
int fused_rows(const LoraProblem& p, int* holds = nullptr) {
  const int64_t groups = p.M < p.S ? p.M : p.S;
  for (int places = kCus;; places += kCus) {
    if (places <= groups) continue;
    const int64_t rows = (p.M + places - groups - 1) / (places - groups);
    if (rows > kMostRows) continue;
    if (holds) *holds = places;
    return rows < 16 ? 16 : int(rows);
  }
}

// Ranges of columns for it: one round of workgroups, those without rows too, which
// take a CU until they know it.  2048 rows of K = 6144 in one range 20.7 us, in two
// (272 workgroups) 17.1; 512 rows of 32 adapters in four ranges (256) 10.3, in five
// 15.6.
int col_ranges(const LoraProblem& p, int rows) {
  const int64_t tiles = most_tiles(p, rows), cols = (p.N + kCols - 1) / kCols;
  int64_t ranges = (kCus - 1 + tiles) / tiles;
  if (ranges > 1 && tiles * ranges > kCus + 32) --ranges;
  return int(ranges < cols ? ranges : cols);
}

// Rows of a tile for the two kernels of a step each.
int step_rows(const LoraProblem& p) { return p.M >= 32 * (p.M < p.S ? p.M : p.S) ? 32 : 16; }

// pieces of K, one workgroup each, until there are two for every CU
int k_splits(const LoraProblem& p) {
  const int64_t tiles = most_tiles(p, step_rows(p));
  int n = 1;
  while (n < 16 && tiles * n < 512 && p.K >= 2 * n * 256) n *= 2;
  return n;
}

__device__ __forceinline__ f32x4 mfma(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}

constexpr int kChiplets = 8;
constexpr int kMostAdapters = 1024;

// The tile of workgroup blockIdx.x, by all W waves of it; false if it has none.  Tiles
// have `rows` rows; where there is one range of columns (near), a row tile less than MS
// if as many rounds of `places` workgroups hold those.  Workgroups go to the eight
// chiplets in turn, each with a cache of its own: each then gets a run of
// neighbouring tiles, which share A_s and B_s (4096 rows of 32 adapters, rank 32,
// fp32: 51 us without that, 47 with).  Up to 64 adapters every wave finds the tile
// alone; of more each thread takes a few (512 rows of 1024 adapters, K = N = 2048: 33 us
// 64 at a time in every wave, 18 so).
template <int W, int MS>
__device__ __forceinline__ bool place_tile(const LoraProblem& p, int rows, int places, bool near, Tile& t) {
  constexpr int kEach = kMostAdapters / (W * kWave);
  constexpr int kLess = MS > 1 ? 16 * (MS - 1) : 16;
  __shared__ int32_t sums[2][W];
  __shared__ int32_t found[3];
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const bool alone = p.S <= kWave;
  const int e0 = alone ? lane : int(threadIdx.x) * kEach;
  int off[kEach], cnt[kEach], n = 0, l = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = e0 + i;
    const bool in = e < p.S && (i == 0 || !alone);
    off[i] = in ? p.offsets[e] : 0;
    cnt[i] = in ? max(p.offsets[e + 1] - off[i], 0) : 0;
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    n += (cnt[i] + rows - 1) / rows;
    l += (cnt[i] + kLess - 1) / kLess;
  }
  int n_to = wave_incl_scan(n), l_to = wave_incl_scan(l);
  int tiles = __builtin_amdgcn_readlane(n_to, kWave - 1), less = __builtin_amdgcn_readlane(l_to, kWave - 1);
  if (!alone) {
    if (lane == kWave - 1) {
      sums[0][wave] = n_to;
      sums[1][wave] = l_to;
    }
    __syncthreads();
    tiles = less = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < wave) {
        n_to += sums[0][w];
        l_to += sums[1][w];
      }
      tiles += sums[0][w];
      less += sums[1][w];
    }
  }
  int first = n_to - n;
  if (MS > 1 && near && less <= places) {
    tiles = less;
    rows = kLess;
    first = l_to - l;
  }
  int at = blockIdx.x;
  if (at >= tiles) return false;                 // the whole workgroup
  if (near) {
    const int x = at % kChiplets, left = tiles % kChiplets;
    at = x * (tiles / kChiplets) + min(x, left) + at / kChiplets;
  }
  bool mine = false;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int k = (cnt[i] + rows - 1) / rows;
    if (at >= first && at < first + k) {
      mine = true;
      t.e = e0 + i;
      t.row0 = off[i] + (at - first) * rows;
      t.rows = min(rows, cnt[i] - (at - first) * rows);
    }
    first += k;
  }
  if (alone) {
    const int src = __ffsll((long long)__ballot(mine)) - 1;
    t.e = __builtin_amdgcn_readlane(t.e, src);
    t.row0 = __builtin_amdgcn_readlane(t.row0, src);
    t.rows = __builtin_amdgcn_readlane(t.rows, src);
    return true;
  }
  if (mine) {
    found[0] = t.e;
    found[1] = t.row0;
    found[2] = t.rows;
  }
  __syncthreads();
  t.e = __builtin_amdgcn_readfirstlane(found[0]);
  t.row0 = __builtin_amdgcn_readfirstlane(found[1]);
  t.rows = __builtin_amdgcn_readfirstlane(found[2]);
  return true;
}

// The row of y and x at sorted position pos, or -1.
__device__ __forceinline__ int row_at(const LoraProblem& p, const Tile& t, int i) {
  const int pos = t.row0 + i;
  if (i >= t.rows || unsigned(pos) >= unsigned(p.M)) return -1;
  const int row = p.rows[pos];
  return unsigned(row) < unsigned(p.M) ? row : -1;
}

// acc += A_s x over the K of [k0, k1) that are a wave's: steps of 32, STRIDE apart.
// A load takes 64 bytes of each of 16 rows by four neighbouring lanes; straight
// in the operands' order, a row a lane, the vector cache gives less than half of
// that rate (8.4 of 18.5 TB/s where it hits L2).  So each 1 KB block goes through
// `stage`, (MS + NR) KB of LDS that no other wave touches: piece q of row i at
// 256 q + 16 (i ^ 4 q), so that sixteen lanes read one window of 256 bytes and
// sixteen lanes write to sixteen different bank groups.  Of an
// operand lane 16 g + i holds row i (of A: operand A, of x: operand B), K 8 g ..
// 8 g + 7; lane 16 g + c of the result holds ranks 4 g .. 4 g + 3 of row c.  Rows
// past the tile and ranks past the last repeat others and are not used.
template <int NR, int MS, bool Few = false>
__device__ __forceinline__ void shrink_part(const LoraProblem& p, const Tile& t, int k0, int k1,
                                            int stride, char* stage, f32x4 (&acc)[MS][NR]) {
  constexpr int R = MS + NR;
  // steps whose loads go out together: more, where few waves have the registers
  constexpr int U = Few ? 4 : R <= 2 ? 6 : R <= 3 ? 4 : R <= 5 ? 3 : 2;
  const int lane = lane_id();
  const int lr = lane >> 2, lp = lane & 3;       // loading: row and piece
  const int c = lane & 15, g = lane >> 4;
  const uint16_t* src[R];
#pragma unroll
  for (int m = 0; m < MS; ++m)
    src[m] = p.x + size_t(max(row_at(p, t, min(16 * m + lr, t.rows - 1)), 0)) * p.K;
#pragma unroll
  for (int j = 0; j < NR; ++j)
    src[MS + j] = p.a + (size_t(t.e) * p.r + min(16 * j + lr, p.r - 1)) * p.K;
  char* put = stage + 256 * lp + 16 * (lr ^ (4 * lp));
  const char* get = stage + 256 * g + 16 * (c ^ (4 * g));
  for (int k = k0; k < k1; k += stride * U) {
    uint4 v[U][R];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = k + stride * u + 8 * lp;
#pragma unroll
      for (int i = 0; i < R; ++i)
        v[u][i] = *reinterpret_cast<const uint4*>(src[i] + (at < k1 ? at : 0));
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k + stride * u >= k1) break;           // wave-uniform
      const bool in = k + stride * u + 8 * lp < k1;
      uint4 o[R];
#pragma unroll
      for (int i = 0; i < R; ++i)
        *reinterpret_cast<uint4*>(put + 1024 * i) = in ? v[u][i] : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < R; ++i) o[i] = *reinterpret_cast<const uint4*>(get + 1024 * i);
#pragma unroll
      for (int j = 0; j < NR; ++j)
#pragma unroll
        for (int m = 0; m < MS; ++m) acc[m][j] = mfma(o[MS + j], o[m], acc[m][j]);
    }
  }
}

template <int NR, int MS>
__device__ __forceinline__ void clear(f32x4 (&acc)[MS][NR]) {
#pragma unroll
  for (int m = 0; m < MS; ++m)
#pragma unroll
    for (int j = 0; j < NR; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// t = A_s x for a tile of 16 MS rows and one piece of K, into `part`.  The
// workgroup's waves take steps in turn and add up through LDS.
template <int RP, int MS>
__global__ __launch_bounds__(kWaves * kWave) void k_lora_shrink(LoraProblem p, int piece) {
  constexpr int NR = (RP + 15) / 16;
  constexpr int kStage = (MS + NR) * 1024, kRed = MS * NR * 1024;
  constexpr int kBytes = kWaves * kStage > (kWaves - 1) * kRed ? kWaves * kStage : (kWaves - 1) * kRed;
  __shared__ __attribute__((aligned(16))) char lds[kBytes];
  Tile t{};
  if (!place_tile<kWaves, 1>(p, 16 * MS, 0, false, t)) return;
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  f32x4 acc[MS][NR];
  clear(acc);
  shrink_part(p, t, blockIdx.y * piece + 32 * wave, min(p.K, int(blockIdx.y + 1) * piece),
              32 * kWaves, lds + wave * kStage, acc);
  __syncthreads();                               // `red` lies where the stages were
  f32x4* red = reinterpret_cast<f32x4*>(lds);
  if (wave > 0) {
#pragma unroll
    for (int m = 0; m < MS; ++m)
#pragma unroll
      for (int j = 0; j < NR; ++j) red[((wave - 1) * MS * NR + m * NR + j) * kWave + lane] = acc[m][j];
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
      for (int w = 0; w < kWaves - 1; ++w) v += red[(w * MS * NR + m * NR + j) * kWave + lane];
      if (ok && 16 * j + 4 * g < RP)
        *reinterpret_cast<f32x4*>(p.part + (size_t(blockIdx.y) * p.M + pos) * RP + 16 * j + 4 * g) = v;
    }
  }
}

// Four neighbouring elements of y as they lie in memory.
template <bool BF16>
using RawY = std::conditional_t<BF16, u32x2, f32x4>;

// Columns past the last repeat it, and are not stored.  Loads and stores with the
// non-temporal hint are faster for a y that no cache holds (8192 rows of rank 16 48
// us, 54 without) and slower for one that the projection has just written, which
// the memory-side cache holds (44 against 40, N = 6144 56 against 42): no hint.
template <bool BF16, bool VEC>
__device__ __forceinline__ RawY<BF16> load_y(const void* y, size_t at, int n, int N) {
  if constexpr (VEC) {
    n = min(n, N - 4);                           // N is a multiple of 4
    const RawY<BF16>* q;
    if constexpr (BF16) {
      q = reinterpret_cast<const RawY<BF16>*>(static_cast<const uint16_t*>(y) + at + n);
    } else {
      q = reinterpret_cast<const RawY<BF16>*>(static_cast<const float*>(y) + at + n);
    }
    return *q;
  } else if constexpr (BF16) {
    const uint16_t* q = static_cast<const uint16_t*>(y) + at;
    const uint32_t v0 = q[min(n, N - 1)], v1 = q[min(n + 1, N - 1)], v2 = q[min(n + 2, N - 1)], v3 = q[min(n + 3, N - 1)];
    return u32x2{v0 | v1 << 16, v2 | v3 << 16};
  } else {
    const float* q = static_cast<const float*>(y) + at;
    return f32x4{q[min(n, N - 1)], q[min(n + 1, N - 1)], q[min(n + 2, N - 1)], q[min(n + 3, N - 1)]};
  }
}

__device__ __forceinline__ f32x4 as_f32(u32x2 u) {
  return f32x4{__uint_as_float(u[0] << 16), __uint_as_float(u[0] & 0xffff0000u),
               __uint_as_float(u[1] << 16), __uint_as_float(u[1] & 0xffff0000u)};
}
__device__ __forceinline__ f32x4 as_f32(f32x4 v) { return v; }

template <bool BF16, bool VEC>
__device__ __forceinline__ void store_y(void* y, size_t at, int n, int N, f32x4 v) {
  RawY<BF16> u;
  if constexpr (BF16) {
    const bf16x2v lo = __builtin_convertvector(f32x2{v[0], v[1]}, bf16x2v);      // to nearest even
    const bf16x2v hi = __builtin_convertvector(f32x2{v[2], v[3]}, bf16x2v);
    u = u32x2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
  } else {
    u = v;
  }
  if constexpr (VEC) {
    if (n >= N) return;
    RawY<BF16>* q;
    if constexpr (BF16) {
      q = reinterpret_cast<RawY<BF16>*>(static_cast<uint16_t*>(y) + at);
    } else {
      q = reinterpret_cast<RawY<BF16>*>(static_cast<float*>(y) + at);
    }
    *q = u;
  } else if constexpr (BF16) {
    uint16_t* q = static_cast<uint16_t*>(y) + at;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) q[i] = uint16_t(u[i >> 1] >> 16 * (i & 1));
  } else {
    float* q = static_cast<float*>(y) + at;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) q[i] = u[i];
  }
}

// y += scale B_s t for a tile of 16 MS rows and 64 columns a wave.  t is fp32
// and B bf16: t is cut into three bf16 of 8 bits each by truncation, which is
// exact, and the three meet the same B along the instruction's K: octet q of K
// is octet q % (RP / 8) of the rank in part q / (RP / 8).  Product j of four
// takes the columns 4 c + j, so lane 16 g + c ends with the four columns from
// 4 c on of the rows 4 g .. 4 g + 3, and a load or store of y covers whole
// pieces of 64 columns.
template <int RP>
struct Parts {
  static constexpr int OCT = RP / 8, NM = (3 * OCT + 3) / 4;
  static constexpr int NB = RP >= 32 ? RP / 32 : NM;     // different operands of B among the NM
  static constexpr int kT = NM * 1024;                   // bytes of 16 rows of t in LDS
  static constexpr int kB = OCT * 1024;                  // bytes of 64 rows of B in LDS
};

// Where K k .. k + 3 of row i of t lie in LDS: blocks of 1 KB in the order in which
// an operand's lanes read them (rows one after another read at half that rate).
template <int RP>
__device__ __forceinline__ int t_slot(int i, int k) {
  return (i >> 4) * Parts<RP>::kT + 1024 * (k >> 5) + 16 * (16 * (k >> 3 & 3) + (i & 15)) + 2 * (k & 7);
}

// Ranks j .. j + 3 of row i of t, in three parts.
template <int RP>
__device__ __forceinline__ void put_t(char* ts, int i, int j, int r, float scale, f32x4 v) {
  uint32_t part[3][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    // past the rank: not t's, and an infinite x times 0 is NaN
    const float f = j + e < r ? v[e] * scale : 0.f;
    const uint32_t hi = __float_as_uint(f) & 0xffff0000u;
    // an infinite or NaN t has no parts below
    const bool fin = (hi & 0x7f800000u) != 0x7f800000u;
    const float rest = fin ? f - __uint_as_float(hi) : 0.f;
    const uint32_t mid = __float_as_uint(rest) & 0xffff0000u;
    part[0][e] = hi;
    part[1][e] = mid;
    part[2][e] = __float_as_uint(rest - __uint_as_float(mid));
  }
#pragma unroll
  for (int s = 0; s < 3; ++s)
    *reinterpret_cast<uint2*>(ts + t_slot<RP>(i, s * RP + j)) =
        make_uint2(part[s][0] >> 16 | (part[s][1] & 0xffff0000u), part[s][2] >> 16 | (part[s][3] & 0xffff0000u));
}

// the rest of a row of t, up to the instruction's K
template <int RP, int MS>
__device__ __forceinline__ void clear_tail(char* ts, int tid, int threads) {
  constexpr int kTail = (32 * Parts<RP>::NM - 3 * RP) / 4;
  if constexpr (kTail > 0)
    for (int i = tid; i < MS * 16 * kTail; i += threads)
      *reinterpret_cast<uint2*>(ts + t_slot<RP>(i / kTail, 3 * RP + 4 * (i % kTail))) = make_uint2(0, 0);
}

// 64 rows of B (columns of y) go through LDS as x and A do: memory holds them in
// one piece, and an operand's lane wants an octet of every fourth row.  Octet o
// of row n lies at 16 (64 o + 16 (n & 3) + (n >> 2 ^ s)), s = (n & 3) << 2 ^ f(o),
// so that sixteen neighbours in memory are sixteen different bank groups.  All
// terms are disjoint bits or combined by ^, so the places of one lane differ by ^
// of constants.
__device__ __forceinline__ constexpr int b_swizzle(int oct, int o) {
  return oct == 2 ? o << 1 : (o & 3) ^ (o & 4) << 1 ^ (o & 8) >> 1;
}
template <int OCT>
__device__ __forceinline__ int b_slot(int n, int o) {
  return 16 * (64 * o + 16 * (n & 3) + ((n >> 2) ^ ((n & 3) << 2) ^ b_swizzle(OCT, o)));
}

// In flight: 16-byte units, or nothing where rows of B are no whole units.
template <int RP, bool VECB>
using RawB = std::conditional_t<VECB, u32x4[RP / 8], u32x4[1]>;

template <int RP, bool VECB>
__device__ __forceinline__ void load_b(const LoraProblem& p, const Tile& t, int n0,
                                       RawB<RP, VECB>& v) {
  if constexpr (VECB) {
    constexpr int OCT = RP / 8;
    const int ro = p.r / 8, lane = lane_id(), n = lane / OCT, o = min(lane % OCT, ro - 1);
    const uint16_t* b = p.b + (size_t(t.e) * p.N + n0) * p.r;
    if (n0 + 64 <= p.N) {
      const uint16_t* at = b + 8 * (n * ro + o);
#pragma unroll
      for (int i = 0; i < OCT; ++i)
        v[i] = *reinterpret_cast<const u32x4*>(at + i * (64 / OCT) * p.r);
    } else {
#pragma unroll
      for (int i = 0; i < OCT; ++i)
        v[i] = *reinterpret_cast<const u32x4*>(b + 8 * (min(64 / OCT * i + n, p.N - 1 - n0) * ro + o));
    }
  }
}

// past the rank 0
template <int RP, bool VECB>
__device__ __forceinline__ void put_b(const LoraProblem& p, const Tile& t, int n0, char* bs,
                                      const RawB<RP, VECB>& v) {
  constexpr int OCT = RP / 8;
  const int lane = lane_id();
  if constexpr (VECB) {
    const int o = lane % OCT, at = b_slot<OCT>(lane / OCT, o);
#pragma unroll
    for (int i = 0; i < OCT; ++i)
      *reinterpret_cast<u32x4*>(bs + (at ^ 256 / OCT * i)) = 8 * o < p.r ? v[i] : u32x4{0, 0, 0, 0};
  } else {
    const uint16_t* b = p.b + (size_t(t.e) * p.N + n0) * p.r;
#pragma unroll 1
    for (int i0 = 0; i0 < RP; i0 += 8) {
      uint16_t h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int x = 64 * (i0 + i) + lane;
        h[i] = b[min(x / RP, p.N - 1 - n0) * p.r + min(x % RP, p.r - 1)];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int x = 64 * (i0 + i) + lane, j = x % RP;
        *reinterpret_cast<uint16_t*>(bs + b_slot<OCT>(x / RP, j >> 3) + 2 * (j & 7)) = j < p.r ? h[i] : uint16_t(0);
      }
    }
  }
}

// The operand of product j: octet 4 q + g (of OCT) of K, row 4 c + j.  Octets past
// the three parts meet zeros of t.
template <int RP>
__device__ __forceinline__ uint4 get_b(const char* bs, int q, int j) {
  constexpr int OCT = RP / 8;
  const int lane = lane_id(), c = lane & 15, g = lane >> 4;
  const int first = b_slot<OCT>(4 * c, g % OCT);
  const int step = OCT < 4 ? 0 : 4096 * q ^ 16 * b_swizzle(OCT, 4 * q);
  return *reinterpret_cast<const uint4*>(bs + (first ^ step ^ 320 * j));
}

// y at the columns n0 .. n0 + 63 of the tile
template <int MS, bool BF16, bool VECY>
__device__ __forceinline__ void load_cols(const LoraProblem& p, int n0, const int64_t* rows,
                                          RawY<BF16> (&yv)[MS][4]) {
  const int lane = lane_id(), n = n0 + 4 * (lane & 15);
#pragma unroll
  for (int m = 0; m < MS; ++m)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t at = rows[16 * m + 4 * (lane >> 4) + q];
      yv[m][q] = load_y<BF16, VECY>(p.y, size_t(at < 0 ? ~at : at), n, p.N);
    }
}

// and their sums with B_s t
template <int RP, int MS, bool BF16, bool VECY>
__device__ __forceinline__ void expand_cols(const LoraProblem& p, const char* ts, const char* bs,
                                            int n0, const int64_t* rows,
                                            const RawY<BF16> (&yv)[MS][4]) {
  using P = Parts<RP>;
  const int lane = lane_id(), c = lane & 15, g = lane >> 4;
  const int n = n0 + 4 * c;
  f32x4 acc[MS][4];
#pragma unroll
  for (int m = 0; m < MS; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int b = 0; b < P::NB; ++b) {
    uint4 bv[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) bv[j] = get_b<RP>(bs, b, j);
#pragma unroll
    for (int q = b; q < P::NM; q += P::NB)       // the parts that meet this piece of B
#pragma unroll
      for (int m = 0; m < MS; ++m) {
        const uint4 tv = *reinterpret_cast<const uint4*>(ts + m * P::kT + 1024 * q + 16 * lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][j] = mfma(tv, bv[j], acc[m][j]);
      }
    if (MS * RP > 64) __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int m = 0; m < MS; ++m)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t at = rows[16 * m + 4 * g + q];
      const f32x4 d = {acc[m][0][q], acc[m][1][q], acc[m][2][q], acc[m][3][q]};
      if (at >= 0) store_y<BF16, VECY>(p.y, size_t(at) + n, n, p.N, as_f32(yv[m][q]) + d);
    }
}

// Where the rows of a tile begin in y, in elements; for a place without a row, whose
// values are loaded and not used, ~ that of the tile's last row.  In LDS: in registers
// they and the addresses made of them take the 40 that a workgroup of 16 waves does
// not have.
template <int MS>
__device__ __forceinline__ void put_rows(const LoraProblem& p, const Tile& t, int64_t* rows) {
  const int i = threadIdx.x;
  if (i < MS * 16) {
    const int row = row_at(p, t, min(i, t.rows - 1));
    const int64_t at = int64_t(max(row, 0)) * p.N;
    rows[i] = row < 0 || i >= t.rows ? ~at : at;
  }
}

template <int RP, int MS, bool BF16, bool VECB, bool VECY>
__global__ __launch_bounds__(kWaves * kWave) void k_lora_expand(LoraProblem p, int splits) {
  using P = Parts<RP>;
  constexpr int kThreads = kWaves * kWave;
  constexpr int kItems = MS * 16 * RP / 4;               // four ranks of a row
  constexpr int kEach = (kItems + kThreads - 1) / kThreads;
  __shared__ __attribute__((aligned(16))) char ts[MS * P::kT];
  __shared__ __attribute__((aligned(16))) char bstage[kWaves * P::kB];
  __shared__ __attribute__((aligned(16))) int64_t rows[MS * 16];
  Tile t{};
  if (!place_tile<kWaves, 1>(p, 16 * MS, 0, false, t)) return;
  const int wave = threadIdx.x >> 6;
  const int step = gridDim.y * kWaves * kCols;
  int n0 = (blockIdx.y * kWaves + wave) * kCols;
  char* bs = bstage + wave * P::kB;
  RawB<RP, VECB> bv;
  if (n0 < p.N) load_b<RP, VECB>(p, t, n0, bv);
  const float scale = p.scale ? p.scale[t.e] : 1.f;
  const float* src[kEach];
  f32x4 sum[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int it = threadIdx.x + kThreads * i, row = it / (RP / 4), pos = t.row0 + row;
    const bool ok = row < t.rows && unsigned(pos) < unsigned(p.M);
    src[i] = p.part + size_t(ok ? pos : 0) * RP + 4 * (it % (RP / 4));
    sum[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  for (int s0 = 0; s0 < splits; s0 += 4) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool in = s0 + u < splits;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const f32x4 w = *reinterpret_cast<const f32x4*>(src[i] + size_t(in ? s0 + u : 0) * p.M * RP);
        sum[i] += in ? w : f32x4{0.f, 0.f, 0.f, 0.f};
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int it = threadIdx.x + kThreads * i;
    if (it < kItems) put_t<RP>(ts, it / (RP / 4), 4 * (it % (RP / 4)), p.r, scale, sum[i]);
  }
  clear_tail<RP, MS>(ts, threadIdx.x, kThreads);
  put_rows<MS>(p, t, rows);
  __syncthreads();
  while (n0 < p.N) {
    put_b<RP, VECB>(p, t, n0, bs, bv);
    RawY<BF16> yv[MS][4];
    load_cols<MS, BF16, VECY>(p, n0, rows, yv);
    const int n = n0;
    n0 += step;
    if (n0 < p.N) load_b<RP, VECB>(p, t, n0, bv);
    expand_cols<RP, MS, BF16, VECY>(p, ts, bs, n, rows, yv);
  }
}

// Both steps of a tile in one workgroup, which computes t for itself: one launch, no
// workspace, and t once for each of gridDim.y column ranges.  16 waves; for three
// row tiles, whose sums of 16 waves LDS does not hold, eight of twice the registers.
template <int MS>
constexpr int kFusedWaves = MS > 2 ? 8 : 16;

template <int RP, int MS, int W>
struct FusedLds {
  static constexpr int NR = (RP + 15) / 16;
  static constexpr int kStage = (MS + NR) * 1024, kRed = MS * NR * 1024;
  static constexpr int kB = Parts<RP>::kB;
  static constexpr int kMost = kStage > kRed ? kStage : kRed;
  static constexpr int kWork = W * (kMost > kB ? kMost : kB);
  static constexpr int kRows = kWork + MS * Parts<RP>::kT;
  static constexpr int kBytes = kRows + MS * 16 * 8;
};

template <int RP, int MS, int W, bool BF16, bool VECB, bool VECY>
__device__ __forceinline__ void fused_tile(const LoraProblem& p, const Tile& t, int chunks, char* smem) {
  using P = Parts<RP>;
  using L = FusedLds<RP, MS, W>;
  constexpr int NR = L::NR;
  char* ts = smem + L::kWork;
  int64_t* rows = reinterpret_cast<int64_t*>(smem + L::kRows);
  const int lane = lane_id(), wave = threadIdx.x >> 6;
  // column pieces blockIdx.y * chunks + wave, + 16, ...
  const int n1 = min(p.N, int(blockIdx.y + 1) * chunks * kCols);
  int n0 = (blockIdx.y * chunks + wave) * kCols;
  RawB<RP, VECB> bv;
  constexpr bool kEarly = RP <= 16;              // registers for B throughout
  if (kEarly && n0 < n1) load_b<RP, VECB>(p, t, n0, bv);
  const float scale = p.scale ? p.scale[t.e] : 1.f;
  f32x4 acc[MS][NR];
  clear(acc);
  shrink_part<NR, MS, W < 16>(p, t, 32 * wave, p.K, 32 * W, smem + wave * L::kStage, acc);
  constexpr bool kAhead = W < 16 || RP * MS < 64;          // registers for the next of B meanwhile
  if (kAhead && !kEarly && n0 < n1) load_b<RP, VECB>(p, t, n0, bv);
  __syncthreads();                               // `red` lies where the stages were
  f32x4* red = reinterpret_cast<f32x4*>(smem);
#pragma unroll
  for (int m = 0; m < MS; ++m)
#pragma unroll
    for (int j = 0; j < NR; ++j) red[(wave * MS * NR + m * NR + j) * kWave + lane] = acc[m][j];
  clear_tail<RP, MS>(ts, threadIdx.x, W * kWave);
  put_rows<MS>(p, t, rows);
  __syncthreads();
  // The first of y meanwhile, and the next where there are registers for it: 8192 rows
  // of rank 32, K = 2048, N = 6144 61 us without, 58 with.
  constexpr bool kAheadY = VECY && W < 16 && RP * MS < (BF16 ? 192 : 128);
  RawY<BF16> yv[MS][4];
  if (VECY && n0 < n1) load_cols<MS, BF16, VECY>(p, n0, rows, yv);
  // item (m, j, lane) as the waves hold it: ranks 16 j + 4 g .. + 3 of row 16 m + c
  for (int it = threadIdx.x; it < MS * NR * kWave; it += W * kWave) {
    f32x4 v = red[it];
#pragma unroll
    for (int w = 1; w < W; ++w) v += red[w * MS * NR * kWave + it];
    const int mj = it / kWave, l = it % kWave;
    const int j = 16 * (mj % NR) + 4 * (l >> 4);
    if (j < RP) put_t<RP>(ts, 16 * (mj / NR) + (l & 15), j, p.r, scale, v);
  }
  __syncthreads();
  char* bs = smem + wave * P::kB;                // and B's rows after that
  while (n0 < n1) {
    if (!kAhead) load_b<RP, VECB>(p, t, n0, bv);
    if (!VECY) load_cols<MS, BF16, VECY>(p, n0, rows, yv);
    __builtin_amdgcn_sched_barrier(0);           // the steps as they stand: 128 registers
    put_b<RP, VECB>(p, t, n0, bs, bv);
    __builtin_amdgcn_sched_barrier(0);
    const int n = n0;
    n0 += W * kCols;
    if (kAhead && n0 < n1) load_b<RP, VECB>(p, t, n0, bv);
    if constexpr (kAheadY) {
      RawY<BF16> next[MS][4];
      if (n0 < n1) load_cols<MS, BF16, VECY>(p, n0, rows, next);
      __builtin_amdgcn_sched_barrier(0);
      expand_cols<RP, MS, BF16, VECY>(p, ts, bs, n, rows, yv);
#pragma unroll
      for (int m = 0; m < MS; ++m)
#pragma unroll
        for (int q = 0; q < 4; ++q) yv[m][q] = next[m][q];
    } else {
      expand_cols<RP, MS, BF16, VECY>(p, ts, bs, n, rows, yv);
      if (VECY && n0 < n1) load_cols<MS, BF16, VECY>(p, n0, rows, yv);
    }
  }
}

template <int RP, int MS, bool BF16, bool VECB, bool VECY>
__global__ __launch_bounds__(kFusedWaves<MS> * kWave) void k_lora_fused(LoraProblem p, int rows, int places,
                                                                       int chunks) {
  constexpr int W = kFusedWaves<MS>;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  Tile t{};
  if (!place_tile<W, MS>(p, rows, places, gridDim.y == 1, t)) return;
  if constexpr (MS > 1) {
    if (t.rows <= 16 * (MS - 1)) {
      fused_tile<RP, MS - 1, W, BF16, VECB, VECY>(p, t, chunks, smem);
      return;
    }
  }
  fused_tile<RP, MS, W, BF16, VECB, VECY>(p, t, chunks, smem);
}

// f(bf16, vector loads of B, vector accesses of y), as types
template <class F>
void by_form(const LoraProblem& p, F f) {
  const int es = p.bf16 ? 2 : 4;
  const bool vb = p.r % 8 == 0;
  const bool vy = p.N % 4 == 0 && reinterpret_cast<uintptr_t>(p.y) % (4 * es) == 0;
  const std::true_type yes;
  const std::false_type no;
  if (p.bf16) {
    if (vb) { if (vy) f(yes, yes, yes); else f(yes, yes, no); }
    else { if (vy) f(yes, no, yes); else f(yes, no, no); }
  } else {
    if (vb) { if (vy) f(no, yes, yes); else f(no, yes, no); }
    else { if (vy) f(no, no, yes); else f(no, no, no); }
  }
}

template <int RP, int MS>
hipError_t launch_two(const LoraProblem& p, hipStream_t s) {
  const unsigned tiles = unsigned(most_tiles(p, 16 * MS));
  const int splits = k_splits(p);
  const int unit = 32 * kWaves;
  const int piece = ((p.K + splits - 1) / splits + unit - 1) / unit * unit;
  k_lora_shrink<RP, MS><<<dim3(tiles, splits), kWaves * kWave, 0, s>>>(p, piece);
  // enough workgroups for the chip, and no more: each sums its rows' pieces first
  const unsigned cols = unsigned((p.N + kWaves * kCols - 1) / (kWaves * kCols));
  const unsigned most = 512 / tiles + 1;
  const dim3 grid(tiles, cols < most ? cols : most);
  by_form(p, [&](auto bf, auto vecb, auto vecy) {
    k_lora_expand<RP, MS, decltype(bf)::value, decltype(vecb)::value, decltype(vecy)::value>
        <<<grid, kWaves * kWave, 0, s>>>(p, splits);
  });
  return hipGetLastError();
}

template <int RP, int MS>
hipError_t launch_fused(const LoraProblem& p, int rows, int places, hipStream_t s) {
  // or as many of a row tile less as `places` hold
  const int64_t most = most_tiles(p, rows);
  const unsigned tiles = unsigned(MS > 1 && most < places ? places : most);
  const unsigned cols = unsigned((p.N + kCols - 1) / kCols);
  const unsigned ranges = unsigned(col_ranges(p, rows));
  const int chunks = int((cols + ranges - 1) / ranges);
  const dim3 grid(tiles, (cols + chunks - 1) / chunks);
  hipError_t e = hipSuccess;
  by_form(p, [&](auto bf, auto vecb, auto vecy) {
    const auto fn = &k_lora_fused<RP, MS, decltype(bf)::value, decltype(vecb)::value, decltype(vecy)::value>;
    constexpr int threads = kFusedWaves<MS> * kWave, lds = FusedLds<RP, MS, kFusedWaves<MS>>::kBytes;
    if (lds > 64 * 1024) {
      static std::atomic<bool> set[kMaxDevices];
      e = lds_limit_once(reinterpret_cast<const void*>(fn), lds, set);
      if (e != hipSuccess) return;
    }
    fn<<<grid, threads, lds, s>>>(p, rows, places, chunks);
  });
  return e != hipSuccess ? e : hipGetLastError();
}

// One launch wherever it is not much slower: a workgroup reads (ms + nr) 32 K bytes
// for its t, at 60 to 80 GB/s, and every range of columns reads them again.  With
// a workgroup for nearly every CU from the row tiles alone there is one range.  In
// us, one launch and two, of which the second costs a caller 3 more that does not
// replay a graph (who does would have two be the faster for few rows): 8 rows of K =
// 6144, N = 4096, rank 16 9.1 and 7.3; of N = 6144, rank 64 18 and 8.7; 8192 rows of
// rank 64 50 and 59.
bool fused(const LoraProblem& p) {
  const int rows = fused_rows(p), ms = (rows + 15) / 16, nr = padded_tiles(p.r);
  if (nr > 4) return false;
  return int64_t(ms + nr) * 32 * p.K <= 512 * 1024 || p.M / rows + (p.M < p.S ? p.M : p.S) / 2 >= 192;
}

template <int RP>
hipError_t launch(const LoraProblem& p, hipStream_t s) {
  if constexpr (RP <= 64) {
    if (fused(p)) {
      int places = 0;
      const int rows = fused_rows(p, &places);
      return rows <= 16 ? launch_fused<RP, 1>(p, rows, places, s)
             : rows <= 32 ? launch_fused<RP, 2>(p, rows, places, s)
                          : launch_fused<RP, 3>(p, rows, places, s);
    }
  }
  return step_rows(p) == 16 ? launch_two<RP, 1>(p, s) : launch_two<RP, 2>(p, s);
}

}  // namespace

size_t lora_workspace_bytes(int M, int K, int N, int S, int r) {
  LoraProblem p{};
  p.M = M; p.K = K; p.N = N; p.S = S; p.r = r;
  return fused(p) ? 0 : size_t(k_splits(p)) * M * padded(r) * sizeof(float);
}

hipError_t launch_lora(const LoraProblem& p, hipStream_t s) {
  switch (padded(p.r)) {
    case 8: return launch<8>(p, s);
    case 16: return launch<16>(p, s);
    case 32: return launch<32>(p, s);
    case 64: return launch<64>(p, s);
    default: return launch<128>(p, s);
  }
}

}  // namespace mxm
