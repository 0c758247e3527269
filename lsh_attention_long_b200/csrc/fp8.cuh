// e4m3 with a scale per block, shared by the norm, the quantiser and the
// products.
//
// A block (1 x 128 or 128 x 128 entries) with largest magnitude
// m = max(2^-96, max |v|) is kept as the codes e4m3(448 v / m), rounded to
// nearest even, and the scale m / 448; it stands for code * scale.  448 is
// the largest e4m3 number, so a block's largest entry is held without error;
// the bound 2^-96 keeps both quotients in range and lets a block of zeros be
// an ordinary block.  An infinity or a NaN makes m infinite or NaN, and every
// entry of its block then stands for NaN (0 * inf).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace lsh {

constexpr int kQBlock = 128;
constexpr float kE4m3Max = 448.f;
constexpr float kMinAmax = 1.2621774483536189e-29f;  // 2^-96

// max(|v|) on the bit patterns: as unsigned integers magnitudes compare like
// the numbers, and every NaN is above infinity, so one NaN wins the maximum
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ float block_amax(uint32_t bits) {
  const uint32_t lo = __float_as_uint(kMinAmax);
  return __uint_as_float(bits > lo ? bits : lo);
}

// The quotient 448 v / m of an entry, from inv = 448 / m (rounded): v * inv is
// within 2^-22 of it, which would put one entry in some 10^5 on the wrong side
// of the border between two codes, and bf16 entries far more often, since their
// quotients often are borders.
//
// v and m of 8 significant bits (bf16): the quotient is either one of the 5-bit
// numbers where e4m3 codes border on each other or at least 2^-13 away from all
// of them: 448 v / m = 7 a / b with integers a, b < 256 up to a power of two, a
// border is c < 32 up to one, and |7 a 2^u - c b| >= 1 unless equal, so the
// relative distance is at least 1 / (31 * 255).  Rounding the product to 16
// significant bits first (error 2^-17) therefore puts the former exactly on the
// border, where ties go to even as the definition asks, and leaves the latter
// on their side.
//
// fp32: 448 / m is carried as a sum of two floats, inv + lo, and v * inv as its
// rounded product and the rest, which an fma gives exactly; their sum is the
// quotient to half a unit of its last place or hardly more.
struct BlockScale {
  float inv, lo;
  __device__ __forceinline__ explicit BlockScale(float am) : inv(kE4m3Max / am) {
    lo = fmaf(-inv, am, kE4m3Max) * inv * (1.f / kE4m3Max);
  }
  __device__ __forceinline__ BlockScale(float i, float l) : inv(i), lo(l) {}
};
// Two or four codes, the first in the lowest byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// Codes of eight entries of a block, two at a time.  (A float is rounded to 16
// bits as 257 q - (257 q - q).)
template <bool kFromBf16>
__device__ __forceinline__ uint2 scale_to_e4m3(const float* v, const BlockScale& b) {
  const float2 inv = make_float2(b.inv, b.inv), lo = make_float2(b.lo, b.lo);
  float2 q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = make_float2(v[2 * i], v[2 * i + 1]);
    q[i] = __fmul2_rn(x, inv);
    if (kFromBf16) {
      const float2 c = __fmul2_rn(q[i], make_float2(257.f, 257.f));
      const float2 d = __ffma2_rn(q[i], make_float2(-1.f, -1.f), c);
      q[i] = __ffma2_rn(d, make_float2(-1.f, -1.f), c);
    } else {
      const float2 rest = __ffma2_rn(x, inv, make_float2(-q[i].x, -q[i].y));
      q[i] = __fadd2_rn(q[i], __ffma2_rn(x, lo, rest));
    }
  }
  return make_uint2(e4m3x4(q[0].x, q[0].y, q[1].x, q[1].y),
                    e4m3x4(q[2].x, q[2].y, q[3].x, q[3].y));
}

}  // namespace lsh
