// Contractions of two MXFP4 factors through LDS: a persistent kernel on the
// scaled matrix instructions.
//
// Work items: (expert, n-tile of 64 AS weight rows, m-tile of at most 192
// rows), expert by expert; within one, blocks of eight m-tiles run through
// the n-tiles.  The list is cut into eight contiguous ranges, one per XCD
// (workgroup b runs on XCD b % 8), whose workgroups, one per CU, take its
// items in rounds, ascending and descending in turn.  Neighbouring items run
// side by side and share weight or activation rows in that XCD's L2; an
// expert of up to 192 rows has its weights read once.
//
// The loads are one endless stream: a workgroup's items are laid out in a
// table first, and the loaders run up to three stages ahead of the matrix
// instructions, across item boundaries, so a new item starts with its first
// stages already in LDS.
//
// A stage is 256 of K: one 128-byte line of codes per row, loaded by eight
// adjacent lanes (whole lines read 15% faster from HBM than half lines: 7.1
// against 6.1 TB/s in a copy of the weight stream alone).  16-byte piece p of
// row r lies at slot p ^ (r % 8) of the row's 128 bytes, which reads without
// bank conflicts at the full rate (measured: 256 bytes per clock, as linear
// reads; r % 4 or r / 2 in its place 160).  Weights go through a ring of
// kRingW stages, activations through two, scale bytes 16 at a time (two
// stages' worth) through two buffers.
//
// Eight waves, 4 x 2, two per SIMD: wave (wn, wm) computes AS 16-row weight
// subtiles x the 16-row subtiles wm, wm + 2, ... of the tile's rows.  A stage
// is two steps of 128; the operands of a step are read from LDS while the
// step before it multiplies.  One barrier per stage, between its steps: past
// it every wave has read all of stage t (its slots are free) and stage t + 1
// has landed.
//
// Matrix rows past a tile's end are not loaded and not stored; blocks past
// the end of K load as zero codes under scale 1.
#include "a4.hpp"
#include "mx_pack.hpp"

namespace mxm {
namespace a4 {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * kWave;
constexpr int kWN = 4, kWM = 2;               // waves along weight rows, along rows
constexpr int kBatch = 32;                    // items laid out at a time
constexpr int kRingX = 2;
constexpr int kMaxE = 1024;
constexpr uint32_t kDead = 0x80000000u;       // a buffer offset out of every range

template <int AS, int MS>
struct Lds {
  static constexpr int kNT = 64 * AS;                        // weight rows per n-tile
  static constexpr int kMT = 16 * kWM * MS;                  // rows per m-tile, at most
  static constexpr int kWSlot = kNT * 128;
  static constexpr int kXSlot = kMT * 128;
  static constexpr int kRingW = AS == 4 ? (MS == 1 ? 4 : 3) : 5;
  static constexpr int kXLoads = (kXSlot / 1024 + kWaves - 1) / kWaves;
  static constexpr int kWLoads = kWSlot / 1024 / kWaves;     // per wave and stage
  static constexpr int kMTw = (kMT + kWave - 1) / kWave * kWave;   // whole waves of rows
  static constexpr int kSRows = kNT + kMTw;
  static constexpr int kX = kRingW * kWSlot;
  static constexpr int kS = kX + kRingX * kXSlot;
  static constexpr int kTok = kS + 2 * kSRows * 16;
  static constexpr int kItems = kTok + 2 * kMTw * 4;
  static constexpr int kBytes = kItems + kBatch * 16;
  static_assert(kBytes <= 160 * 1024, "LDS per CU");
  static_assert((kMaxE + 1) * 4 <= kX, "the tile prefix borrows the weight ring");
};

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((ext_vector_type(4))) int int4v;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

__device__ __forceinline__ lds_void* lds_at(uint8_t* base, int off) {
  return (lds_void*)(base + off);
}

// s_waitcnt immediates (gfx9 layout): vmcnt <= n alone, and lgkmcnt 0 alone
#define MXM_VMCNT(n) ((((n) & 15) | (((n) >> 4) << 14)) | (7 << 4) | (15 << 8))
#define MXM_LGKM0 (15 | (3 << 14) | (7 << 4))

// At most n of this wave's loads and stores outstanding (n is rounded down to
// a count that has an instruction here, which only waits longer).
__device__ __forceinline__ void vmcnt_le(int n) {
  if (n >= 28) __builtin_amdgcn_s_waitcnt(MXM_VMCNT(28));
  else if (n >= 16) __builtin_amdgcn_s_waitcnt(MXM_VMCNT(16));
  else if (n >= 12) __builtin_amdgcn_s_waitcnt(MXM_VMCNT(12));
  else if (n >= 8) __builtin_amdgcn_s_waitcnt(MXM_VMCNT(8));
  else if (n >= 4) __builtin_amdgcn_s_waitcnt(MXM_VMCNT(4));
  else if (n >= 2) __builtin_amdgcn_s_waitcnt(MXM_VMCNT(2));
  else if (n >= 1) __builtin_amdgcn_s_waitcnt(MXM_VMCNT(1));
  else __builtin_amdgcn_s_waitcnt(MXM_VMCNT(0));
}

// LDS reads of the loaders' tables, with their wait inside: the compiler
// would guard them with a wait for every asynchronous load in flight.
__device__ __forceinline__ uint32_t lds_addr(const uint8_t* p) {
  return uint32_t(reinterpret_cast<uintptr_t>((const lds_void*)p));
}
__device__ __forceinline__ int lds_read_i32(const uint8_t* p) {
  int v;
  asm volatile("ds_read_b32 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=v"(v) : "v"(lds_addr(p)) : "memory");
  return v;
}
__device__ __forceinline__ int4v lds_read_i32x4(const uint8_t* p) {
  int4v v;
  asm volatile("ds_read_b128 %0, %1\n\ts_waitcnt lgkmcnt(0)" : "=v"(v) : "v"(lds_addr(p)) : "memory");
  return v;
}

struct Item {
  int e, n, row0, rows;
};

// The scale bytes of block g of a stage's two steps, in bytes 0 and 1.
__device__ __forceinline__ uint32_t pick(u32x2 v, uint32_t sel) {
  return __builtin_amdgcn_perm(v.y, v.x, sel);
}

// acc += W X for byte B of the packed scales
template <int B>
__device__ __forceinline__ f32x4 mfma_step(u32x4 w, uint32_t sw, u32x4 x, uint32_t sx, f32x4 acc) {
  const i32x8 a = {int(w.x), int(w.y), int(w.z), int(w.w), 0, 0, 0, 0};
  const i32x8 b = {int(x.x), int(x.y), int(x.z), int(x.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, kFp4, kFp4, B, int(sw), B,
                                                          int(sx));
}

// KIND, OUT as in a4.hpp; AS: weight subtiles per wave; WHOLE: K is a
// multiple of 512 and scale rows are 16-byte aligned.
template <Kind KIND, Out OUT, int AS, int MS, bool WHOLE>
struct Tiled {
  using L = Lds<AS, MS>;
  static constexpr bool kGU = KIND == kGateUp;
  static constexpr int kCols = kGU ? L::kNT / 2 : L::kNT;    // output columns per n-tile
  static constexpr int kAux = KIND == kGemm ? 0 : 2;         // grouped weights: non-temporal

  const Problem& p;
  uint8_t* lds;
  int wave, lane, r16, g, wn, wm;
  int nst, nblk, rowb;
  int cnt;                          // items of the batch

  // loaders: activations and scales (two stages ahead), weights (kRingW ahead)
  int xi = 0, xs = 0, xt = 0;       // item, stage in it, stage overall
  int xchunk = 0;                   // scale chunks issued
  int nx = 0;                       // activation loads of this wave per stage
  uint32_t xoff[L::kXLoads];
  const uint8_t* sptr = nullptr;    // this lane's scale row
  bool srow = false;                // the wave loads scales for this item
  int wi = 0, wst = 0, wt = 0;
  uint32_t woff[L::kWLoads];
  const uint8_t* wbase = nullptr;
  int young = 0;                    // loads and stores issued since the last one waited for
  // without WHOLE: scale bytes on their way from memory to LDS
  uint32_t spend[4];
  int spend_slot = -1;

  // compute: weights of the step at hand (each subtile is replaced by the next
  // step's once it is used), activations of a stage's two steps, scales
  u32x4 w[AS], xa[MS], xb[MS];
  uint32_t sw[AS], sx[MS], sxn[MS];
  f32x4 acc[AS][MS];

  __device__ __forceinline__ Tiled(const Problem& q, uint8_t* l) : p(q), lds(l) {
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    lane = lane_id();
    r16 = lane & 15;
    g = lane >> 4;
    wn = wave % kWN;
    wm = wave / kWN;
    nblk = p.K / 32;
    nst = (nblk + 7) / 8;
    rowb = p.K / 2;
  }

  __device__ __forceinline__ Item item(int i) const {
    const int4v v = lds_read_i32x4(lds + L::kItems + 16 * i);
    return Item{__builtin_amdgcn_readfirstlane(v.x), __builtin_amdgcn_readfirstlane(v.y),
                __builtin_amdgcn_readfirstlane(v.z), __builtin_amdgcn_readfirstlane(v.w)};
  }

  // Local weight row lr (0 .. kNT-1) of n-tile n, as a row of its expert:
  // gate/up tiles are kCols gate columns, then the same up columns.  Rows
  // past the last column repeat it.
  __device__ __forceinline__ int wrow(int n, int lr) const {
    if constexpr (kGU) {
      const int up = lr >= kCols;
      return up * p.N + min(n * kCols + lr - up * kCols, p.N - 1);
    } else {
      return min(n * kCols + lr, p.N - 1);
    }
  }
  __device__ __forceinline__ int64_t erow(int e) const {     // first weight row of expert e
    return int64_t(e) * (kGU ? 2 : 1) * p.N;
  }

  // Row of X of tile row j (< rows) of the item whose tokens are in slot `par`.
  __device__ __forceinline__ int64_t xrow(const Item& it, int par, int j) const {
    if constexpr (kGU) return lds_read_i32(lds + L::kTok + par * L::kMTw * 4 + 4 * j) / p.k;
    else return int64_t(it.row0) + j;
  }

  // pair ids of an item's rows -> token slot (waves 0 .. 2, one load each)
  __device__ __forceinline__ void issue_tokens(int i) {
    if constexpr (kGU) {
      if (wave < L::kMTw / kWave && i < cnt) {
        const Item it = item(i);
        const int32_t* src = p.pairs + it.row0 + min(wave * kWave + lane, it.rows - 1);
        __builtin_amdgcn_global_load_lds(
            src, lds_at(lds, L::kTok + (i & 1) * L::kMTw * 4 + wave * kWave * 4), 4, 0, 0);
      }
    }
  }

  __device__ __forceinline__ void x_item() {
    const Item it = item(xi);
    const int rl = lane >> 3;
    nx = 0;
#pragma unroll
    for (int q = 0; q < L::kXLoads; ++q) {
      const int j0 = 8 * (wave + kWaves * q);
      if (j0 < it.rows) ++nx;
      const int j = min(j0 + rl, it.rows - 1);
      xoff[q] = uint32_t(xrow(it, xi & 1, j)) * uint32_t(rowb) + 16u * ((lane & 7) ^ rl) +
                (j0 + rl >= it.rows ? kDead : 0u);
    }
    const int sr = (wave & 3) * kWave + lane;
    if (wave < kWN) {
      srow = sr < L::kNT;
      sptr = p.ws + (erow(it.e) + wrow(it.n, sr)) * nblk;
    } else {
      srow = (wave & 3) * kWave < it.rows;
      sptr = p.xs + xrow(it, xi & 1, min(sr, it.rows - 1)) * nblk;
    }
  }

  __device__ __forceinline__ int sslot(int chunk) const { return L::kS + (chunk & 1) * L::kSRows * 16; }
  __device__ __forceinline__ int srow_off() const {
    return ((wave < kWN ? 0 : L::kNT) + (wave & 3) * kWave) * 16;
  }

  // activations (and, for a new pair of stages, scales) of the next stage of
  // the activation stream
  __device__ __forceinline__ void issue_x(const __amdgpu_buffer_rsrc_t& rx) {
    if (xi >= cnt) return;
    if (xs == 0) x_item();
    if ((xs & 1) == 0) {
      if (srow) {
        if constexpr (WHOLE) {
          __builtin_amdgcn_global_load_lds(sptr + 8 * xs, lds_at(lds, sslot(xchunk) + srow_off()), 16,
                                           0, 0);
        } else {
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            uint32_t v = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const int blk = 8 * xs + 4 * d + b;
              v |= (blk < nblk ? uint32_t(sptr[blk]) : 127u) << (8 * b);
            }
            spend[d] = v;
          }
          spend_slot = sslot(xchunk);
        }
      }
      ++xchunk;
    }
    const uint32_t tail =
        !WHOLE && 8 * xs + int((lane & 7) ^ (lane >> 3)) >= nblk ? kDead : 0u;
#pragma unroll
    for (int q = 0; q < L::kXLoads; ++q)
      if (q < nx)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rx, lds_at(lds, L::kX + (xt & 1) * L::kXSlot + 1024 * (wave + kWaves * q)), 16,
            (xoff[q] + 128u * xs) | tail, 0, 0, 0);
    ++xt;
    if (++xs == nst) {
      xs = 0;
      ++xi;
    }
  }

  // scale bytes that came through registers go to LDS before the barrier
  // after which they are read
  __device__ __forceinline__ void flush_scales() {
    if constexpr (!WHOLE) {
      if (spend_slot >= 0)
        *reinterpret_cast<u32x4*>(lds + spend_slot + srow_off() + 16 * lane) =
            u32x4{spend[0], spend[1], spend[2], spend[3]};
      spend_slot = -1;
    }
  }

  __device__ __forceinline__ void w_item() {
    const Item it = item(wi);
    const int rl = lane >> 3;
    const int r0 = kGU ? 0 : it.n * kCols;               // the first row the base stands for
    wbase = p.wc + (erow(it.e) + r0) * rowb;
#pragma unroll
    for (int q = 0; q < L::kWLoads; ++q)
      woff[q] = uint32_t(wrow(it.n, 8 * (wave + kWaves * q) + rl) - r0) * uint32_t(rowb) +
                16u * ((lane & 7) ^ rl);
  }

  __device__ __forceinline__ int issue_w() {
    if (wi >= cnt) return 0;
    if (wst == 0) w_item();
    const __amdgpu_buffer_rsrc_t rw =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(wbase), 0, 0x7fffffff, 0x00020000);
    // a piece past the row's end meets zero activations; it reads the row's first
    const bool past = !WHOLE && 8 * wst + int((lane & 7) ^ (lane >> 3)) >= nblk;
    const uint32_t back = past ? 128u * wst + 16u * ((lane & 7) ^ (lane >> 3)) : 0u;
    const int slot = (wt % L::kRingW) * L::kWSlot;
#pragma unroll
    for (int q = 0; q < L::kWLoads; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, lds_at(lds, slot + 1024 * (wave + kWaves * q)), 16,
                                               woff[q] + 128u * wst - back, 0, 0, kAux);
    ++wt;
    if (++wst == nst) {
      wst = 0;
      ++wi;
    }
    return L::kWLoads;
  }

  // this wave's weight subtile a as a local weight row
  __device__ __forceinline__ int sub_row(int a) const {
    if constexpr (kGU) return (a < AS / 2 ? 0 : kCols) + 16 * (AS / 2) * wn + 16 * (a % (AS / 2));
    else return 16 * AS * wn + 16 * a;
  }

  // where this lane's pieces of step kk lie, from the start of a 16-row subtile
  __device__ __forceinline__ int piece(int kk) const {
    return 16 * ((4 * kk + g) ^ (r16 & 7)) + 128 * r16;
  }
  // weight subtile a of step kk of stage t
  __device__ __forceinline__ void read_w(int t, int kk, int a) {
    w[a] = *reinterpret_cast<const u32x4*>(lds + (t % L::kRingW) * L::kWSlot + piece(kk) +
                                           128 * sub_row(a));
  }
  __device__ __forceinline__ void read_x(int t, int kk, u32x4 (&x)[MS]) const {
    const uint8_t* b = lds + L::kX + (t & 1) * L::kXSlot + 128 * 16 * wm + piece(kk);
#pragma unroll
    for (int i = 0; i < MS; ++i) x[i] = *reinterpret_cast<const u32x4*>(b + 128 * 16 * kWM * i);
  }

  // scales of stage s of an item whose first scale chunk is c
  __device__ __forceinline__ const uint8_t* scales_at(int c, int s) const {
    return lds + sslot(c + (s >> 1)) + 16 * r16 + 8 * (s & 1);
  }
  __device__ __forceinline__ uint32_t scale_pair(const uint8_t* s) const {
    return pick(*reinterpret_cast<const u32x2*>(s), 0x0c0c0400u + 0x0101u * g);   // bytes g
  }
  __device__ __forceinline__ void read_sw(const uint8_t* sc, int a) {
    sw[a] = scale_pair(sc + 16 * sub_row(a));
  }
  __device__ __forceinline__ void read_sx(const uint8_t* sc, uint32_t (&x)[MS]) const {
#pragma unroll
    for (int i = 0; i < MS; ++i) x[i] = scale_pair(sc + 16 * (L::kNT + 16 * (wm + kWM * i)));
  }

  // a step's products; then(a) runs once weight subtile a is used
  template <int B, class F>
  __device__ __forceinline__ void step(const u32x4 (&x)[MS], F&& then) {
#pragma unroll
    for (int a = 0; a < AS; ++a) {
#pragma unroll
      for (int i = 0; i < MS; ++i) acc[a][i] = mfma_step<B>(w[a], sw[a], x[i], sx[i], acc[a][i]);
      then(a);
    }
  }

  __device__ __forceinline__ int epilogue(const Item& it) {
    int stores = 0;
    const int64_t row0 = it.row0;
    if constexpr (OUT == kMx) {
      // a wave's two gate subtiles are one MX block: h rounded to bf16, then
      // packed; the block is this lane's eight and those of lanes +-16, +-32
      static_assert(OUT != kMx || AS == 4, "two 16-column groups per wave");
      const int blk = it.n * (kCols / 32) + wn;
      const bool inside = 32 * blk < p.N;
      const __amdgpu_buffer_rsrc_t rc = __builtin_amdgcn_make_buffer_rsrc(
          p.oc + row0 * (p.N / 2), 0, 0x7fffffff, 0x00020000);
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          p.os + row0 * (p.N / 32), 0, 0x7fffffff, 0x00020000);
#pragma unroll
      for (int i = 0; i < MS; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        uint32_t v[2][4];
        uint32_t amax = 0;
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            v[a][c] = f32_to_bf16_rne(silu_mul(acc[a][i][c], acc[a + AS / 2][i][c])) << 16;
            amax = max(amax, v[a][c] & 0x7fffffffu);
          }
        amax = max(amax, uint32_t(__shfl_xor(int(amax), 16)));
        amax = max(amax, uint32_t(__shfl_xor(int(amax), 32)));
        const bool bad = amax >= 0x7f800000u;              // Inf or NaN in the block
        const uint32_t e = bad ? 255u : mx_scale_byte(amax);
        const MxThresholds th(bad ? 0u : e);
        uint32_t c16[2];
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          uint32_t c = 0;
#pragma unroll
          for (int d = 0; d < 4; ++d) c |= th.code(v[a][d]) << (4 * d);
          c16[a] = bad ? 0u : c;
        }
        // bytes 2g, 2g + 1 of subtile a lie in lane group g: even groups take
        // subtile 0's two pairs, odd ones subtile 1's, four bytes a lane
        const uint32_t give = g & 1 ? c16[0] : c16[1];
        const uint32_t got = uint32_t(__shfl_xor(int(give), 16));
        const uint32_t word = g & 1 ? got | (c16[1] << 16) : c16[0] | (got << 16);
        const int j = 16 * (wm + kWM * i) + r16;
        const bool live = inside && j < it.rows;
        __builtin_amdgcn_raw_buffer_store_b32(
            word, rc, live ? uint32_t(j) * (p.N / 2) + 16 * blk + 8 * (g & 1) + 4 * (g >> 1) : kDead,
            0, 0);
        __builtin_amdgcn_raw_buffer_store_b8(
            uint8_t(e), rs, live && g == 0 ? uint32_t(j) * (p.N / 32) + blk : kDead, 0, 0);
        stores += 2;
      }
    } else {
      constexpr int kSize = OUT == kF32 ? 4 : 2;
      constexpr int kSubs = kGU ? AS / 2 : AS;
      const int col0 = it.n * kCols + 16 * kSubs * wn + 4 * g;
      uint8_t* base = static_cast<uint8_t*>(p.out) + row0 * p.N * kSize;
      const __amdgpu_buffer_rsrc_t ro =
          __builtin_amdgcn_make_buffer_rsrc(base, 0, 0x7fffffff, 0x00020000);
      // rows of whole vectors, or elements one by one
      const bool vec = p.N % 4 == 0 && (reinterpret_cast<uintptr_t>(p.out) & (4 * kSize - 1)) == 0;
#pragma unroll
      for (int i = 0; i < MS; ++i) {
        const int j = 16 * (wm + kWM * i) + r16;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int a = 0; a < kSubs; ++a) {
          f32x4 v = acc[a][i];
          if constexpr (kGU) {
            const f32x4 u = acc[a + AS / 2][i];
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = silu_mul(v[c], u[c]);
          }
          const int col = col0 + 16 * a;
          const uint32_t at = (uint32_t(j) * uint32_t(p.N) + uint32_t(col)) * kSize;
          const bool live = j < it.rows;
          if constexpr (OUT == kF32) {
            const u32x4 b = __builtin_bit_cast(u32x4, v);
            if (vec) {
              __builtin_amdgcn_raw_buffer_store_b128(b, ro, live && col < p.N ? at : kDead, 0, 0);
            } else {
#pragma unroll
              for (int c = 0; c < 4; ++c)
                __builtin_amdgcn_raw_buffer_store_b32(b[c], ro, live && col + c < p.N ? at + 4 * c : kDead,
                                                      0, 0);
            }
          } else {
            uint32_t b[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) b[c] = f32_to_bf16_rne(v[c]);
            if (vec) {
              __builtin_amdgcn_raw_buffer_store_b64(u32x2{b[0] | (b[1] << 16), b[2] | (b[3] << 16)}, ro,
                                                        live && col < p.N ? at : kDead, 0, 0);
            } else {
#pragma unroll
              for (int c = 0; c < 4; ++c)
                __builtin_amdgcn_raw_buffer_store_b16(uint16_t(b[c]), ro,
                                                          live && col + c < p.N ? at + 2 * c : kDead, 0, 0);
            }
          }
          stores += 1;                       // at least
        }
      }
    }
    return stores;
  }

  // One item: its stages and the epilogue.  t: the item's first stage in the
  // stream; c: its first scale chunk.  A stage's operands are read ahead
  // within the item; an item's first ones at its start, after the epilogue
  // before it, whose registers they need.
  __device__ __forceinline__ void run_item(const Item& it, int i, int t, int c,
                                           const __amdgpu_buffer_rsrc_t& rx) {
#pragma unroll
    for (int a = 0; a < AS; ++a)
#pragma unroll
      for (int m = 0; m < MS; ++m) acc[a][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    {
      const uint8_t* sc = scales_at(c, 0);
      read_x(t, 0, xa);
      read_sx(sc, sx);
#pragma unroll
      for (int a = 0; a < AS; ++a) {
        read_w(t, 0, a);
        read_sw(sc, a);
      }
    }
    for (int s = 0; s + 1 < nst; ++s, ++t) {
      first_step(t, s, i, rx);
      const uint8_t* sc = scales_at(c, s + 1);
      read_x(t + 1, 0, xa);
      read_sx(sc, sxn);
      step<1>(xb, [&](int a) {
        read_w(t + 1, 0, a);
        read_sw(sc, a);
      });
#pragma unroll
      for (int m = 0; m < MS; ++m) sx[m] = sxn[m];
    }
    first_step(t, nst - 1, i, rx);
    step<1>(xb, [](int) {});
    __builtin_amdgcn_sched_barrier(0);
    young += epilogue(it);
    __builtin_amdgcn_sched_barrier(0);
  }

  // The first step of stage s (t in the stream), the barrier behind which its
  // slots are free, and the loads that go there.
  __device__ __forceinline__ void first_step(int t, int s, int i, const __amdgpu_buffer_rsrc_t& rx) {
    read_x(t, 1, xb);
    step<0>(xa, [&](int a) { read_w(t, 1, a); });
    flush_scales();
    __builtin_amdgcn_s_waitcnt(MXM_LGKM0);
    vmcnt_le(young);
    wg_barrier();
    if (s == 0) issue_tokens(i + 1);
    issue_x(rx);
    __builtin_amdgcn_sched_barrier(0);      // the count below is of the loads after these
    young = issue_w();
    __builtin_amdgcn_sched_barrier(0);
  }

  __device__ __forceinline__ void run(int items) {
    cnt = items;
    const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(p.xc), 0, int(int64_t(p.M) * rowb), 0x00020000);
    issue_tokens(0);
    if constexpr (kGU) {
      __builtin_amdgcn_s_waitcnt(MXM_VMCNT(0));
      wg_barrier();
    }
    issue_x(rx);
    flush_scales();
#pragma unroll
    for (int q = 0; q < L::kRingW - 1; ++q) issue_w();
    issue_x(rx);
    young = issue_w();
    flush_scales();
    __builtin_amdgcn_s_waitcnt(MXM_LGKM0);
    __builtin_amdgcn_s_waitcnt(MXM_VMCNT(0));
    wg_barrier();
    int t = 0, c = 0;
    for (int i = 0; i < cnt; ++i) {
      run_item(item(i), i, t, c, rx);
      t += nst;
      c += (nst + 1) >> 1;
    }
  }
};

// Number of m-tiles of a segment, and the rows of each (a multiple of 16).
__device__ __forceinline__ int m_tiles(int rows, int bm) { return (rows + bm - 1) / bm; }
__device__ __forceinline__ int tile_rows(int rows, int mt) { return ((rows + mt - 1) / mt + 15) & ~15; }

template <Kind KIND, Out OUT, int AS, int MS, bool WHOLE>
__global__ __launch_bounds__(kThreads, 2) void k_tiled(Problem p) {
  using L = Lds<AS, MS>;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = lane_id();
  constexpr int kCols = KIND == kGateUp ? L::kNT / 2 : L::kNT;
  const int ntn = (p.N + kCols - 1) / kCols;
  const int E = KIND == kGemm ? 1 : p.E;
  int* mpre = reinterpret_cast<int*>(lds);
  auto seg = [&](int e, int& off) {
    if constexpr (KIND == kGemm) {
      off = 0;
      return p.M;
    } else {
      off = p.offsets[e];
      const int n = p.offsets[e + 1] - off;
      return n >= p.lo && n < p.hi ? n : 0;
    }
  };
  const int gx = int(gridDim.x >> 3);              // workgroups per XCD
  const int wi = int(blockIdx.x >> 3), xcd = int(blockIdx.x & 7);
  for (int r0 = 0;; r0 += kBatch) {
    // m-tiles before each expert
    if (wave == 0) {
      int base = 0;
      for (int c0 = 0; c0 < E; c0 += kWave) {
        const int e = c0 + lane;
        int off;
        const int rows = e < E ? seg(e, off) : 0;
        const int mt = m_tiles(rows, L::kMT);
        const int incl = wave_incl_scan(mt);
        if (e < E) mpre[e] = base + incl - mt;
        base += __shfl(incl, kWave - 1);
      }
      if (lane == 0) mpre[E] = base;
    }
    __syncthreads();
    const int64_t nitems = int64_t(mpre[E]) * ntn;
    const int64_t v0 = nitems * xcd / 8, v1 = nitems * (xcd + 1) / 8;
    // round r's item of this workgroup: ascending when r is even
    auto at = [&](int r) { return v0 + int64_t(r) * gx + ((r & 1) ? gx - 1 - wi : wi); };
    int cnt = 0;
    for (int r = r0; r < r0 + kBatch && v0 + int64_t(r) * gx < v1; ++r) cnt += at(r) < v1;
    if (int(threadIdx.x) < cnt) {
      const int64_t v = at(r0 + int(threadIdx.x));
      const int tau = int(v / ntn);
      int lo = 0, hi = E;                          // mpre[lo] <= tau < mpre[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (mpre[mid] <= tau) lo = mid;
        else hi = mid;
      }
      const int mt = mpre[lo + 1] - mpre[lo];
      const int64_t local = v - int64_t(mpre[lo]) * ntn;
      const int sr = int(local / (8 * int64_t(ntn)));
      const int rem = int(local - int64_t(sr) * 8 * ntn);
      const int mw = min(8, mt - 8 * sr);
      const int m = 8 * sr + rem % mw;
      int off;
      const int rows = seg(lo, off);
      const int tr = tile_rows(rows, mt);
      *reinterpret_cast<int4v*>(lds + L::kItems + 16 * threadIdx.x) =
          int4v{lo, rem / mw, off + m * tr, min(tr, rows - m * tr)};
    }
    __syncthreads();
    if (cnt == 0) break;
    Tiled<KIND, OUT, AS, MS, WHOLE> w(p, lds);
    w.run(cnt);
    __syncthreads();
    if (v0 + int64_t(r0 + kBatch) * gx >= v1) break;
  }
}

template <Kind KIND, Out OUT, int AS, int MS, bool WHOLE>
hipError_t launch(const Problem& p, hipStream_t s) {
  static std::atomic<bool> lds_set[kMaxDevices];
  auto* fn = &k_tiled<KIND, OUT, AS, MS, WHOLE>;
  const hipError_t e = lds_limit_once(reinterpret_cast<const void*>(fn), Lds<AS, MS>::kBytes, lds_set);
  if (e != hipSuccess) return e;
  const int grid = (device_cus() + 7) / 8 * 8;     // one per CU, a multiple of 8
  fn<<<dim3(unsigned(grid)), kThreads, Lds<AS, MS>::kBytes, s>>>(p);
  return hipGetLastError();
}

template <Kind KIND, Out OUT, int AS, int MS>
hipError_t launch_k(const Problem& p, hipStream_t s) {
  const bool whole = p.K % 512 == 0 && reinterpret_cast<uintptr_t>(p.xs) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(p.ws) % 16 == 0;
  return whole ? launch<KIND, OUT, AS, MS, true>(p, s) : launch<KIND, OUT, AS, MS, false>(p, s);
}

}  // namespace

// The kernel addresses activations and one item's weights and outputs by
// 31-bit byte offsets.  The pair ids of a gate/up item are fetched while the
// item before it runs its first stage and used two stages before its last:
// four stages.
bool tiled_supported(Kind kind, const Problem& p) {
  const int64_t lim = (int64_t(1) << 31) - 1;
  const int64_t rowb = p.K / 2;
  if (p.E > kMaxE || int64_t(p.M) * rowb > lim) return false;
  if (int64_t(kind == kGateUp ? p.N + 256 : 256) * rowb > lim) return false;
  if (int64_t(192) * p.N * 4 > lim) return false;
  return kind != kGateUp || p.K > 768;
}

hipError_t launch_tiled(Kind kind, Out out, const Problem& p, hipStream_t s) {
  const int groups = kind == kGemm || p.R < p.E ? (kind == kGemm ? 1 : p.R) : p.E;
  const int mean = p.R / groups;
  if (mean <= 24) {
    if (kind == kGemm)
      return out == kBf16 ? launch_k<kGemm, kBf16, 4, 1>(p, s) : launch_k<kGemm, kF32, 4, 1>(p, s);
    if (kind == kDown) return launch_k<kDown, kF32, 4, 1>(p, s);
    return out == kMx ? launch_k<kGateUp, kMx, 4, 1>(p, s) : launch_k<kGateUp, kBf16, 4, 1>(p, s);
  }
  if (kind == kGemm)
    return out == kBf16 ? launch_k<kGemm, kBf16, 4, 6>(p, s) : launch_k<kGemm, kF32, 4, 6>(p, s);
  if (kind == kDown) return launch_k<kDown, kF32, 4, 6>(p, s);
  return out == kMx ? launch_k<kGateUp, kMx, 4, 6>(p, s) : launch_k<kGateUp, kBf16, 4, 6>(p, s);
}

}  // namespace a4
}  // namespace mxm
