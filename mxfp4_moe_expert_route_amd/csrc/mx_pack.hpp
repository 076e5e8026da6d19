// The OCP MX v1.0 conversion of one block of 32 values to MXFP4, shared by
// mxfp4_pack and the kernels that write their result in MXFP4.
//
// Values and thresholds are compared as IEEE bit patterns with integer
// arithmetic, so the result is exact (subnormal inputs included) and does not
// depend on the floating-point denormal mode.
#pragma once
#include "common.hpp"

namespace mxm {

// fp32 bits of (1 + mf/2^23) * 2^p * 2^(e-127) for the rounding midpoints;
// exact for every e the conversion can choose (see the caller).
__device__ __forceinline__ uint32_t midpoint_bits(int p, uint32_t mf, int e) {
  const int be = p + e;
  if (be >= 1) return (uint32_t(be) << 23) | mf;
  return (0x800000u | mf) >> (1 - be);               // be >= -2: exact shift
}

// Scale byte of a block whose largest magnitude has the bits `amax` (finite).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  if (amax == 0u) return 0u;
  const int ef = int(amax >> 23);
  const int fl = ef > 0 ? ef - 127 : (31 - __clz(amax)) - 149;     // floor(log2 amax)
  return uint32_t(min(max(fl - 2 + 127, 0), 254));
}

// E2M1 codes under scale byte e (0..254).  The magnitude code is the number
// of midpoints passed; at a midpoint the even code wins: strict '>' below an
// even code, '>=' below an odd one.
struct MxThresholds {
  uint32_t t0, t1, t2, t3, t4, t5, t6;
  __device__ __forceinline__ explicit MxThresholds(uint32_t e) {
    const int ei = int(e);
    t0 = midpoint_bits(-2, 0x000000u, ei);   // 0.25
    t1 = midpoint_bits(-1, 0x400000u, ei);   // 0.75
    t2 = midpoint_bits(0, 0x200000u, ei);    // 1.25
    t3 = midpoint_bits(0, 0x600000u, ei);    // 1.75
    t4 = midpoint_bits(1, 0x200000u, ei);    // 2.5
    t5 = midpoint_bits(1, 0x600000u, ei);    // 3.5
    t6 = midpoint_bits(2, 0x200000u, ei);    // 5
  }
  // code of the finite value with fp32 bits v
  __device__ __forceinline__ uint32_t code(uint32_t v) const {
    const uint32_t a = v & 0x7fffffffu;
    return (uint32_t(a > t0) + uint32_t(a >= t1) + uint32_t(a > t2) + uint32_t(a >= t3) +
            uint32_t(a > t4) + uint32_t(a >= t5) + uint32_t(a > t6)) |
           ((v >> 28) & 8u);                 // sign bit of the input
  }
};

}  // namespace mxm
