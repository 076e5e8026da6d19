// Contractions of two MXFP4 factors through LDS: a persistent kernel on the
// scaled matrix instructions.
//
// Work items: (expert, n-tile of 64 AS weight rows, m-tile of at most 32 MS
// rows), expert by expert; within one, blocks of eight m-tiles run through
// the n-tiles.  The list is cut into eight contiguous ranges, one per XCD
// (workgroup b runs on XCD b % 8), whose workgroups, one per CU, take its
// items in rounds, ascending and descending in turn.  Neighbouring items run
// side by side and share weight or activation rows in that XCD's L2; an
// expert whose rows fit one tile has its weights read once.
//
// The loads are one endless stream: a workgroup's items are laid out in a
// table first, and the loaders run two stages (weights three to five) ahead of
// the matrix instructions, across item boundaries, so a new item starts with
// its first stages already in LDS.
//
// A stage is 256 of K: one 128-byte line of codes per row, loaded by eight
// adjacent lanes (whole lines read 15% faster from HBM than half lines: 7.1
// against 6.1 TB/s in a copy of the weight stream alone).  16-byte piece p of
// row r lies at slot p ^ (r % 8) of the row's 128 bytes, which reads as fast as
// linear addresses do (p ^ (r % 4) and p ^ (r / 2 % 8) at 0.6 of that).  Weights
// go through a ring of kRingW stages, activations through two.  Scales are
// loaded 32 bytes of a row at a time (four stages' worth) into registers and
// written to one LDS buffer a stage later, transposed, so that a lane finds its
// four steps' bytes in one dword.
//
// Eight waves, 4 x 2, two per SIMD: wave (wn, wm) computes AS 16-row weight
// subtiles x the 16-row subtiles wm, wm + 2, ... of the tile's rows.  A stage
// is two steps of 128; the operands of a step are read from LDS while the
// step before it multiplies, and the stage's loads are spread over its
// products.  One barrier per stage, between its steps: past it every wave has
// read all of stage t (its slots are free) and stage t + 1 has landed.
//
// Matrix rows past a tile's end are not loaded and not stored; pieces past the
// end of K load as zero codes.  A row's blocks past its end have scales of that
// row's own, so a NaN among them is one that the row's result holds anyway.
//
// What bounds it.  8192 x 4096 x 6144 takes 131-144 us, 2.9-3.1 PFLOP/s.  The
// matrix pipes are busy a third of its cycles, at 2.1 GHz, and LDS reads a
// quarter at most, so neither bounds it: what is left are the waits of one
// workgroup a CU (a barrier a stage, a tile's start and epilogue), and 2.7 rounds
// of tiles being three.  The page-shaped gate/up (384 experts, 6144 x 2 2048)
// takes 1.3-1.37 ms at 8192 tokens (1.10 at a large copy's rate; there the clock
// falls to 1.7 GHz, the pipes busy 39%) and 135 us at 8 (5.9 TB/s; reads alone
// reach 7.1); down 0.87-0.91 ms at 8192 (0.86 at a copy's rate) and 300 us at 64
// (6.3 TB/s).  An activation ring of three stages was no faster at any size.
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

// Stages of an item: 256 of K each, in pairs
__host__ __device__ __forceinline__ int stages(int K) { return 2 * ((K / 32 + 15) / 16); }

template <int AS, int MS>
struct Lds {
  static constexpr int kNT = 16 * kWN * AS;                 // weight rows per n-tile
  static constexpr int kMT = 16 * kWM * MS;                  // rows per m-tile, at most
  static constexpr int kWSlot = kNT * 128;
  static constexpr int kXSlot = kMT * 128;
  static constexpr int kRingW = AS == 4 ? (MS == 1 ? 4 : 3) : 5;
  static constexpr int kXLoads = (kXSlot / 1024 + kWaves - 1) / kWaves;
  static constexpr int kWLoads = kWSlot / 1024 / kWaves;     // per wave and stage
  static constexpr int kSRows = kNT + kMT;                   // rows of scales, 32 bytes each
  static constexpr int kSLoads = (kSRows / 32 + kWaves - 1) / kWaves;
  static constexpr int kMTw = (kMT + kWave - 1) / kWave * kWave;   // whole waves of rows
  static constexpr int kX = kRingW * kWSlot;
  static constexpr int kS = kX + kRingX * kXSlot;
  static constexpr int kTok = kS + kSRows * 32;
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

// The lane id, as a value of its own: what the rarely run parts derive from it
// is computed there and holds no register in between.
__device__ __forceinline__ int lane_here() {
  int l = lane_id();
  asm volatile("" : "+v"(l));
  return l;
}

// 32-bit product in one register (a multiply-add would hold two)
__device__ __forceinline__ uint32_t times(int a, int b) {
  uint32_t v = uint32_t(a) * uint32_t(b);
  asm("" : "+v"(v));
  return v;
}

// The 4 x 4 bytes of four dwords transposed: dword g gets their bytes g.
__device__ __forceinline__ u32x4 transpose4(u32x4 v) {
  const uint32_t a = __builtin_amdgcn_perm(v.y, v.x, 0x05010400u);   // x0 y0 x1 y1
  const uint32_t b = __builtin_amdgcn_perm(v.y, v.x, 0x07030602u);   // x2 y2 x3 y3
  const uint32_t c = __builtin_amdgcn_perm(v.w, v.z, 0x05010400u);
  const uint32_t d = __builtin_amdgcn_perm(v.w, v.z, 0x07030602u);
  return u32x4{__builtin_amdgcn_perm(c, a, 0x05040100u), __builtin_amdgcn_perm(c, a, 0x07060302u),
               __builtin_amdgcn_perm(d, b, 0x05040100u), __builtin_amdgcn_perm(d, b, 0x07060302u)};
}

// acc += W X for byte B of the packed scales
template <int B>
__device__ __forceinline__ f32x4 mfma_step(u32x4 w, uint32_t sw, u32x4 x, uint32_t sx, f32x4 acc) {
  const i32x8 a = {int(w.x), int(w.y), int(w.z), int(w.w), 0, 0, 0, 0};
  const i32x8 b = {int(x.x), int(x.y), int(x.z), int(x.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, kFp4, kFp4, B, int(sw), B,
                                                          int(sx));
}

// KIND, OUT as in a4.hpp; AS, MS: weight and row subtiles per wave; WHOLE: K
// is a multiple of 512 and scale rows are 16-byte aligned.
template <Kind KIND, Out OUT, int AS, int MS, bool WHOLE>
struct Tiled {
  using L = Lds<AS, MS>;
  static constexpr bool kGU = KIND == kGateUp;
  static constexpr int kCols = kGU ? L::kNT / 2 : L::kNT;    // output columns per n-tile
  static constexpr int kAux = KIND == kGemm ? 0 : 2;         // grouped weights: non-temporal

  const Problem& p;
  uint8_t* lds;
  int wave, lane, r16, g, wn, wm;
  int nst, nblk, rowb;              // stages per item (an even number), blocks and bytes per row
  int cnt;                          // items of the batch

  // the activation (and scale) stream, two stages ahead
  int xi = 0, xs = 0, xt = 0;       // item, stage in it, stage overall
  int xdst = 0, xso = 0;            // LDS slot and offset in the rows of the stage at hand
  uint32_t xtail = 0;
  uint32_t xoff[L::kXLoads];
  uint32_t soff[L::kSLoads];        // this lane's scale rows
  const uint8_t* swbase = nullptr;
  u32x4 spend[L::kSLoads];          // scales on their way from memory to LDS
  bool sfull = false;
  // the weight stream, kRingW stages ahead
  int wi = 0, wst = 0, wt = 0;
  int wdst = 0, wso = 0, wbytes = 0;
  uint32_t wlane;                   // this lane's piece of a load's first row
  const uint8_t* wbase = nullptr;
  int stores = 0;                   // of the epilogue before
  // where this lane's pieces of step kk and its scales lie in a subtile
  int wat[2], xat[2], swat, sxat;

  // compute: weights of the step at hand (each subtile is replaced by the next
  // step's once it is used), activations of a stage's two steps, the scales of
  // a pair of stages (a byte per step)
  u32x4 w[AS], xa[MS], xb[MS];
  uint32_t sw[AS], sx[MS];
  f32x4 acc[AS][MS];

  __device__ __forceinline__ Tiled(const Problem& q, uint8_t* l) : p(q), lds(l) {
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    lane = lane_id();
    r16 = lane & 15;
    g = lane >> 4;
    wn = wave % kWN;
    wm = wave / kWN;
    nblk = p.K / 32;
    nst = stages(p.K);
    rowb = p.K / 2;
    wlane = uint32_t(8 * wave + (lane >> 3)) * uint32_t(rowb) + 16u * ((lane & 7) ^ (lane >> 3));
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int at = 16 * ((4 * kk + g) ^ (r16 & 7)) + 128 * r16;
      wat[kk] = at + 128 * sub_row(0);
      xat[kk] = at + 128 * 16 * wm + L::kX;
    }
    swat = L::kS + 32 * (sub_row(0) + r16) + 16 * (r16 >> 3) + 4 * g;
    sxat = L::kS + 32 * (L::kNT + 16 * wm + r16) + 16 * (r16 >> 3) + 4 * g;
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
  __device__ __forceinline__ int xrow(const Item& it, int par, int j) const {
    if constexpr (kGU) return lds_read_i32(lds + L::kTok + par * L::kMTw * 4 + 4 * j) / p.k;
    else return it.row0 + j;
  }

  // pair ids of an item's rows -> token slot, one load per 64 rows
  __device__ __forceinline__ void issue_tokens(int i) {
    if constexpr (kGU) {
      if (wave < L::kMTw / kWave && i < cnt) {
        const Item it = item(i);
        const int lane = lane_here();
        const int32_t* src = p.pairs + it.row0 + min(wave * kWave + lane, it.rows - 1);
        __builtin_amdgcn_global_load_lds(
            src, lds_at(lds, L::kTok + (i & 1) * L::kMTw * 4 + wave * kWave * 4), 4, 0, 0);
      }
    }
  }

  // Scale load h of this wave: 32 rows, two lanes each; weight rows first.
  // A lane's 16 bytes are the blocks 4 j + g of four steps j of 128; they go to
  // LDS transposed, so that lane group g finds its bytes of the four steps in
  // one dword.  Row r keeps its half b at slot b ^ (r / 8 % 2): the 16 rows of
  // a subtile are read without bank conflicts.
  __device__ __forceinline__ int sload(int h) const { return wave + kWaves * h; }
  __device__ __forceinline__ bool sload_w(int h) const { return sload(h) < L::kNT / 32; }
  __device__ __forceinline__ bool sload_any(int h) const { return sload(h) < L::kSRows / 32; }

  __device__ __forceinline__ void x_item() {
    const Item it = item(xi);
    const int lane = lane_here();
    const int rl = lane >> 3;
#pragma unroll
    for (int q = 0; q < L::kXLoads; ++q) {
      const int j = 8 * (wave + kWaves * q) + rl;
      xoff[q] = times(xrow(it, xi & 1, min(j, it.rows - 1)), rowb) + 16u * ((lane & 7) ^ rl) +
                (j >= it.rows ? kDead : 0u);
    }
    swbase = p.ws + erow(it.e) * nblk;
#pragma unroll
    for (int h = 0; h < L::kSLoads; ++h) {
      const int r = 32 * sload(h) + (lane >> 1);
      soff[h] = times(sload_w(h) ? wrow(it.n, r)
                                 : xrow(it, xi & 1, max(0, min(r - L::kNT, it.rows - 1))), nblk);
    }
  }

  // Scales of stages 4 c .. 4 c + 3 of the activation stream's item, at its
  // stage 4 c: into registers here, to LDS before the next barrier.  One
  // buffer does: a pair of stages' scales are read in the stage before it, so
  // past this point the last of the four before are in registers, and the
  // first of these are read behind the next barrier.
  __device__ __forceinline__ void load_scales() {
    const int lane = lane_here();
    const int half = (lane & 1) ^ ((lane >> 4) & 1);
#pragma unroll
    for (int h = 0; h < L::kSLoads; ++h) {
      if (!sload_any(h)) continue;
      const int b0 = 8 * xs + 16 * half;                // first block of this lane's half
      const uint8_t* src = (sload_w(h) ? swbase : p.xs) + soff[h];
      if constexpr (WHOLE) {
        // a half past the row's end is not used; it reads the row's first
        spend[h] = *reinterpret_cast<const u32x4*>(src + (b0 < nblk ? b0 : 0));
      } else {
        // sixteen bytes from any address, the row's last at the latest
        struct __attribute__((packed, aligned(1))) U {
          u32x4 v;
        };
        spend[h] = reinterpret_cast<const U*>(src + min(b0, nblk - 16))->v;
      }
    }
    sfull = true;
  }
  __device__ __forceinline__ void flush_scales() {
    if (sfull) {
#pragma unroll
      for (int h = 0; h < L::kSLoads; ++h)
        if (sload_any(h)) {
          *reinterpret_cast<u32x4*>(lds + L::kS + 1024 * sload(h) + 16 * lane) =
              transpose4(WHOLE ? spend[h] : trim_scales(spend[h]));
        }
    }
    sfull = false;
  }
  // Scales loaded from the row's last sixteen blocks move to their places.
  // (xs is one past the stage of the load.)
  __device__ __forceinline__ u32x4 trim_scales(u32x4 v) {
    const int lane = lane_here();
    const int by = max(8 * ((xs - 1) & ~3) + 16 * ((lane & 1) ^ ((lane >> 4) & 1)) + 16 - nblk, 0);
    if (by & 8) v.x = v.z, v.y = v.w;
    if (by & 4) v.x = v.y, v.y = v.z, v.z = v.w;
#pragma unroll
    for (int d = 0; d < 4; ++d)
      v[d] = __builtin_amdgcn_alignbyte(d < 3 ? v[d + 1] : 0u, v[d], uint32_t(by) & 3u);
    return v;
  }

  // Next stage of the activation stream: where it goes; a new item's rows; new
  // scales.  Past the stream's end the loads are dead: they move nothing, and
  // keep the count of loads the same in every stage.
  //
  // The scalar offset stays below a row's bytes.  A buffer load's range check
  // compares the vector offset with the buffer's size less the scalar one,
  // unsigned: past the end of a buffer of one row (K = 544: 272 bytes, the
  // fourth stage at 384) that would wrap, and dead offsets be inside.  Stages that
  // the bound changes have dead pieces alone.  (Written as a select it costs the
  // 256 x 192 product up to 17 registers more in scratch.)
  __device__ __forceinline__ void next_x() {
    xdst = L::kX + (xt & 1) * L::kXSlot;
    xso = WHOLE ? 128 * xs : min(128 * xs, rowb - 16);
    xtail = 0;
    ++xt;
    if (xi >= cnt) {
      xtail = kDead;
      return;
    }
    if (xs == 0) x_item();
    if ((xs & 3) == 0) load_scales();
    if (!WHOLE && 8 * xs + 8 > nblk) {
      // an item's last stages: pieces past the row's end are dead from here on
      const int lane = lane_here();
      const uint32_t dead = 8 * xs + ((lane & 7) ^ (lane >> 3)) >= nblk ? kDead : 0u;
#pragma unroll
      for (int q = 0; q < L::kXLoads; ++q) xoff[q] |= dead;
    }
    if (++xs == nst) {
      xs = 0;
      ++xi;
    }
  }
  __device__ __forceinline__ void load_x(const __amdgpu_buffer_rsrc_t& rx, int q) {
    if (L::kXSlot / 1024 % kWaves && wave + kWaves * q >= L::kXSlot / 1024) return;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, lds_at(lds, xdst + 1024 * (wave + kWaves * q)), 16,
                                             xoff[q] | xtail, xso, 0, 0);
  }

  // A tile's weight rows are those of the expert from its first on (gate/up:
  // and N further on, the up rows).  Rows past the last column are other
  // rows, or zeros past the expert's end; so are pieces past a row's end, which
  // meet zero activations.  None of their sums is stored.
  __device__ __forceinline__ void w_item() {
    const Item it = item(wi);
    const int64_t rows = int64_t(kGU ? 2 : 1) * p.N - it.n * kCols;
    wbase = p.wc + (erow(it.e) + it.n * kCols) * rowb;
    wbytes = int(rows * rowb < 0x7fffffff ? rows * rowb : 0x7fffffff);
  }
  __device__ __forceinline__ void next_w() {
    wdst = (wt % L::kRingW) * L::kWSlot;
    wso = 128 * wst;
    ++wt;
    if (wi >= cnt) {
      wbytes = 0;                            // dead loads: out of range
      return;
    }
    if (wst == 0) w_item();
    if (++wst == nst) {
      wst = 0;
      ++wi;
    }
  }
  __device__ __forceinline__ void load_w(int q) {
    const __amdgpu_buffer_rsrc_t rw =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(wbase), 0, wbytes, 0x00020000);
    const int lr0 = 8 * kWaves * q;          // first local row of the load
    const int row0 = kGU && lr0 >= kCols ? p.N + lr0 - kCols : lr0;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, lds_at(lds, wdst + 1024 * (wave + kWaves * q)), 16,
                                             wlane + uint32_t(row0) * uint32_t(rowb) + uint32_t(wso), 0,
                                             0, kAux);
  }

  // this wave's weight subtile a as a local weight row
  __device__ __forceinline__ int sub_row(int a) const {
    if constexpr (kGU) return (a < AS / 2 ? 0 : kCols) + 16 * (AS / 2) * wn + 16 * (a % (AS / 2));
    else return 16 * AS * wn + 16 * a;
  }
  // weight subtile a of step kk of stage t; a's distance from subtile 0 is a
  // constant, so it goes into the read's offset
  __device__ __forceinline__ void read_w(int t, int kk, int a) {
    w[a] = *reinterpret_cast<const u32x4*>(lds + ((t % L::kRingW) * L::kWSlot + wat[kk]) +
                                           128 * (sub_row(a) - sub_row(0)));
  }
  __device__ __forceinline__ void read_x(int t, int kk, u32x4 (&x)[MS]) const {
    const uint8_t* b = lds + ((t & 1) * L::kXSlot + xat[kk]);
#pragma unroll
    for (int i = 0; i < MS; ++i) x[i] = *reinterpret_cast<const u32x4*>(b + 128 * 16 * kWM * i);
  }
  // this lane's scales of stages 2 pr and 2 pr + 1 of an item, a byte per step
  __device__ __forceinline__ void read_sw(int pr, int a) {
    sw[a] = *reinterpret_cast<const uint32_t*>(lds + (swat ^ (16 * (pr & 1))) +
                                               32 * (sub_row(a) - sub_row(0)));
  }
  __device__ __forceinline__ void read_sx(int pr) {
    const uint8_t* b = lds + (sxat ^ (16 * (pr & 1)));
#pragma unroll
    for (int i = 0; i < MS; ++i) sx[i] = *reinterpret_cast<const uint32_t*>(b + 32 * 16 * kWM * i);
  }

  // a step's products; then(a) runs once weight subtile a is used
  template <int B, class F>
  __device__ __forceinline__ void step(const u32x4 (&x)[MS], F&& then) {
#pragma unroll
    for (int a = 0; a < AS; ++a) {
#pragma unroll
      for (int i = 0; i < MS; ++i) acc[a][i] = mfma_step<B>(w[a], sw[a], x[i], sx[i], acc[a][i]);
      // the products are made here, not wherever their sums are next used
#pragma unroll
      for (int i = 0; i < MS; ++i) asm volatile("" : "+v"(acc[a][i]));
      then(a);
      __builtin_amdgcn_sched_barrier(0);       // keeps loads and reads where they stand
    }
  }
  // A step's share of n loads after subtile a: spread over the step, since a
  // burst of all waves' loads stalls their products.
  template <class F>
  __device__ __forceinline__ void spread(int n, int a, F&& load) {
    const int per = (n + AS - 1) / AS;
#pragma unroll
    for (int q = 0; q < n; ++q)
      if (q / per == a) load(q);
  }

  __device__ __forceinline__ int epilogue(const Item& it) {
    int n = 0;
    const int64_t row0 = it.row0;
    const int lane = lane_here(), r16 = lane & 15, g = lane >> 4;
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
        n += 2;
      }
    } else {
      constexpr int kSize = OUT == kF32 ? 4 : 2;
      constexpr int kSubs = kGU ? AS / 2 : AS;
      const int col0 = it.n * kCols + 16 * kSubs * wn + 4 * g;
      uint8_t* base = static_cast<uint8_t*>(p.out) + row0 * p.N * kSize;
      const __amdgpu_buffer_rsrc_t ro =
          __builtin_amdgcn_make_buffer_rsrc(base, 0, 0x7fffffff, 0x00020000);
      // four columns a store, wherever their row starts (buffer stores need
      // no alignment); the last columns of an N that is no multiple of four
      // one by one
      const bool edge = p.N % 4 != 0 && (it.n + 1) * kCols >= p.N;
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
          const uint32_t to = live && col + 4 <= p.N ? at : kDead;
          if constexpr (OUT == kF32) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), ro, to, 0, 0);
            if (edge) {
#pragma unroll
              for (int c = 0; c < 3; ++c)
                __builtin_amdgcn_raw_buffer_store_b32(
                    __float_as_uint(v[c]), ro,
                    live && col + 4 > p.N && col + c < p.N ? at + 4 * c : kDead, 0, 0);
            }
          } else {
            uint32_t b[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) b[c] = f32_to_bf16_rne(v[c]);
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{b[0] | (b[1] << 16), b[2] | (b[3] << 16)}, ro, to,
                                                  0, 0);
            if (edge) {
#pragma unroll
              for (int c = 0; c < 3; ++c)
                __builtin_amdgcn_raw_buffer_store_b16(
                    uint16_t(b[c]), ro, live && col + 4 > p.N && col + c < p.N ? at + 2 * c : kDead, 0,
                    0);
            }
          }
          n += 1;                            // at least
        }
      }
    }
    return n;
  }

  // Stage t of the stream, an item's first (FIRST), last (LAST) or another
  // one; PAR: its parity.  The loads due behind its barrier are spread over
  // the products: activations in its second step, weights in the next stage's
  // first (in this one's second where an epilogue lies between).  At the
  // barrier everything but the youngest weights (and the stores after them)
  // has to have landed.
  template <int PAR, bool FIRST, bool LAST>
  __device__ __forceinline__ void stage(int t, int pr, int i, const __amdgpu_buffer_rsrc_t& rx) {
    read_x(t, 1, xb);
    step<2 * PAR>(xa, [&](int a) {
      if constexpr (!FIRST) spread(L::kWLoads, a, [&](int q) { load_w(q); });
      read_w(t, 1, a);
    });
    flush_scales();
    __builtin_amdgcn_s_waitcnt(MXM_LGKM0);
    // (the tiles that reload spilled registers at an item's start have waited
    // for the stores by then)
    if constexpr (FIRST) vmcnt_le(L::kWLoads + stores);
    else __builtin_amdgcn_s_waitcnt(MXM_VMCNT(L::kWLoads));
    wg_barrier();
    if constexpr (FIRST) issue_tokens(i + 1);
    next_x();
    next_w();
    if constexpr (LAST) {
      step<2 * PAR + 1>(xb, [&](int a) { spread(L::kXLoads, a, [&](int q) { load_x(rx, q); }); });
      __builtin_amdgcn_sched_barrier(0);       // the weights' loads stay the youngest
#pragma unroll
      for (int q = 0; q < L::kWLoads; ++q) load_w(q);
    } else {
      read_x(t + 1, 0, xa);
      step<2 * PAR + 1>(xb, [&](int a) {
        spread(L::kXLoads, a, [&](int q) { load_x(rx, q); });
        read_w(t + 1, 0, a);
        if constexpr (PAR == 1) read_sw(pr + 1, a);
      });
      if constexpr (PAR == 1) read_sx(pr + 1);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // One item: its stages and the epilogue.  t: the item's first stage in the
  // stream.  A stage's operands are read ahead within the item; an item's
  // first ones at its start, after the epilogue before it, whose registers
  // they need.
  __device__ __forceinline__ void run_item(const Item& it, int i, int t,
                                           const __amdgpu_buffer_rsrc_t& rx) {
#pragma unroll
    for (int a = 0; a < AS; ++a)
#pragma unroll
      for (int m = 0; m < MS; ++m) acc[a][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    {
      read_x(t, 0, xa);
      read_sx(0);
#pragma unroll
      for (int a = 0; a < AS; ++a) {
        read_w(t, 0, a);
        read_sw(0, a);
      }
    }
    stage<0, true, false>(t, 0, i, rx);
    const int pairs = nst / 2;
    for (int pr = 0; pr + 1 < pairs; ++pr) {
      stage<1, false, false>(t + 2 * pr + 1, pr, i, rx);
      stage<0, false, false>(t + 2 * pr + 2, pr + 1, i, rx);
    }
    stage<1, false, true>(t + nst - 1, pairs - 1, i, rx);
    __builtin_amdgcn_sched_barrier(0);
    stores = epilogue(it);
    __builtin_amdgcn_sched_barrier(0);
  }

  __device__ __forceinline__ void run(int items) {
    cnt = items;
    const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(p.xc), 0, int(int64_t(p.M) * rowb), 0x00020000);
    if constexpr (kGU) {
      issue_tokens(0);
      __builtin_amdgcn_s_waitcnt(MXM_VMCNT(0));
      wg_barrier();
    }
#pragma unroll
    for (int h = 0; h < kRingX; ++h) {
      next_x();
#pragma unroll
      for (int q = 0; q < L::kXLoads; ++q) load_x(rx, q);
      flush_scales();
    }
#pragma unroll
    for (int h = 0; h < L::kRingW; ++h) {
      next_w();
#pragma unroll
      for (int q = 0; q < L::kWLoads; ++q) load_w(q);
    }
    __builtin_amdgcn_s_waitcnt(MXM_LGKM0);
    __builtin_amdgcn_s_waitcnt(MXM_VMCNT(0));
    wg_barrier();
    for (int i = 0; i < cnt; ++i) run_item(item(i), i, i * nst, rx);
    __builtin_amdgcn_s_waitcnt(MXM_VMCNT(0));    // the dead loads past the stream's end
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
    const int64_t nitems = int64_t(__builtin_amdgcn_readfirstlane(mpre[E])) * ntn;
    const int64_t v0 = nitems * xcd / 8, v1 = nitems * (xcd + 1) / 8;
    // round r's item of this workgroup: ascending when r is even
    auto at = [&](int r) { return v0 + int64_t(r) * gx + ((r & 1) ? gx - 1 - wi : wi); };
    int cnt = 0;
    for (int r = r0; r < r0 + kBatch && v0 + int64_t(r) * gx < v1; ++r) cnt += at(r) < v1;
    cnt = __builtin_amdgcn_readfirstlane(cnt);
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

// Tiles of 192 rows use every register.  With K whole they spill 18 to 34: gate/up
// and down at the start of an item, the product also in its main loop, the second
// of a wave's two scale loads on its way to LDS, out and back once in four stages.
// A reload waits for every load in flight.  Where K is not whole products and
// down spill at most three, not in the loop; gate/up has none left to bring scales
// to their places, and takes 160 rows, without spills.
template <Kind KIND, Out OUT, int AS, int MS>
hipError_t launch_k(const Problem& p, hipStream_t s) {
  const bool whole = p.K % 512 == 0 && reinterpret_cast<uintptr_t>(p.xs) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(p.ws) % 16 == 0;
  constexpr int kRest = KIND == kGateUp && MS == 6 ? 5 : MS;
  return whole ? launch<KIND, OUT, AS, MS, true>(p, s) : launch<KIND, OUT, AS, kRest, false>(p, s);
}

// Experts of up to 32 LIGHT rows with tiles as tall, the others with tiles of
// 32 HEAVY rows.
template <Kind KIND, Out OUT, int LIGHT, int HEAVY>
hipError_t launch_split(const Problem& p, hipStream_t s) {
  Problem part = p;
  part.lo = 32 * LIGHT + 1;
  const hipError_t e = launch_k<KIND, OUT, 4, HEAVY>(part, s);
  if (e != hipSuccess) return e;
  part.lo = p.lo;
  part.hi = 32 * LIGHT + 1;
  return launch_k<KIND, OUT, 4, LIGHT>(part, s);
}

template <Kind KIND, Out OUT>
hipError_t launch_grouped(const Problem& p, int ms, bool split, hipStream_t s) {
  if (split) {
    if (ms == 1) return launch_split<KIND, OUT, 1, 3>(p, s);
    return ms == 2 ? launch_split<KIND, OUT, 2, 6>(p, s) : launch_split<KIND, OUT, 3, 6>(p, s);
  }
  if (ms == 1) return launch_k<KIND, OUT, 4, 1>(p, s);
  return ms == 2 ? launch_k<KIND, OUT, 4, 2>(p, s) : launch_k<KIND, OUT, 4, 3>(p, s);
}

template <Out OUT>
hipError_t launch_gemm(const Problem& p, int as, int ms, hipStream_t s) {
  if (as == 4) return launch_k<kGemm, OUT, 4, 6>(p, s);
  if (ms == 6) return launch_k<kGemm, OUT, 2, 6>(p, s);
  if (ms == 4) return launch_k<kGemm, OUT, 2, 4>(p, s);
  if (ms == 2) return launch_k<kGemm, OUT, 2, 2>(p, s);
  return launch_k<kGemm, OUT, 2, 1>(p, s);
}

}  // namespace

// The kernel addresses activations and one item's weights and outputs by
// 31-bit byte offsets.  The pair ids of a gate/up item are fetched behind the
// barrier of the first stage of the item before it, have landed at the second's
// and are read behind the last but one's, so an item has to have four stages (K
// of 544 and more).  Scales are loaded 16 blocks of a row at a time: K >= 512.
bool tiled_supported(Kind kind, const Problem& p) {
  const int64_t lim = (int64_t(1) << 31) - 1;
  const int64_t rowb = p.K / 2;
  if (p.E > kMaxE || int64_t(p.M) * rowb > lim) return false;
  if (int64_t(kind == kGateUp ? p.N + 256 : 256) * rowb > lim) return false;
  if (int64_t(192) * p.N * 4 > lim || int64_t(p.N) * 2 * (p.K / 32) > lim) return false;
  return p.K >= 512 && (kind != kGateUp || stages(p.K) >= 4);
}

hipError_t launch_tiled(Kind kind, Out out, const Problem& p, int ms, bool split, hipStream_t s) {
  if (kind == kDown) return launch_grouped<kDown, kF32>(p, ms, split, s);
  return out == kMx ? launch_grouped<kGateUp, kMx>(p, ms, split, s)
                    : launch_grouped<kGateUp, kBf16>(p, ms, split, s);
}

hipError_t launch_tiled_gemm(Out out, const Problem& p, int as, int ms, hipStream_t s) {
  return out == kBf16 ? launch_gemm<kBf16>(p, as, ms, s) : launch_gemm<kF32>(p, as, ms, s);
}

}  // namespace a4
}  // namespace mxm
