// Product of two e4m3 matrices with a scale per 128 entries of K:
//   C[m, n] = sum_kb sa[m, kb] sb[n, kb] (sum_{k in kb} A[m, k] B[n, k])
//             (+ bias[n]) (max(0, .)).
// The codes of a block are multiplied and added in fp32; each block's sum
// then enters the fp32 total with its two scales.
#pragma once

#include "fp8.cuh"

namespace lsh {

struct Fp8GemmArgs {
  int M, N, K;               // N, K multiples of 16
  const uint8_t* A;          // [M, K]
  const float* sa;           // [M, kb], kb = ceil(K / 128)
  const uint8_t* B;          // [N, K]
  const float* sb;           // [N, kb] (b_rows 1) or [ceil(N / 128), kb] (b_rows 128)
  int b_rows;
  const __nv_bfloat16* bias; // [N] or NULL
  int relu;
  void* C;                   // [M, N]
  int c_f32;                 // fp32, else bf16
};

// max(0, v); a NaN stays one.
__device__ __forceinline__ float relu_nan(float v) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
  return r;
}

// 448 / m as a sum of two floats for the two functions below.  The second is
// above zero, so that an entry of -inf stays one (-inf * 0, or the sum of two
// infinities, would be NaN); the smallest float in place of a zero is far below
// half of the first's last place.
__device__ __forceinline__ BlockScale relu_scale(float am) {
  float inv = kE4m3Max / am, rest = fmaf(-inv, am, kE4m3Max);
  if (rest < 0.f) {  // rounded up: the next smaller float
    inv = __uint_as_float(__float_as_uint(inv) - 1);
    rest = fmaf(-inv, am, kE4m3Max);
  }
  return BlockScale(inv, fmaxf(rest * inv * (1.f / kE4m3Max), __uint_as_float(1u)));
}
// 448 v / m, rounded once.
__device__ __forceinline__ float scaled(float v, const BlockScale& s) {
  return fmaf(v, s.inv, v * s.lo);
}
// The codes of max(0, 448 v[0 .. 3] / m).
__device__ __forceinline__ uint32_t e4m3x4_relu(const float* v, const BlockScale& s) {
  const float2 inv = make_float2(s.inv, s.inv), low = make_float2(s.lo, s.lo);
  const float2 u = make_float2(v[0], v[1]), w = make_float2(v[2], v[3]);
  const float2 a = __ffma2_rn(u, inv, __fmul2_rn(u, low));
  const float2 b = __ffma2_rn(w, inv, __fmul2_rn(w, low));
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.relu.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(a.y), "f"(a.x));
  asm("cvt.rn.satfinite.relu.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(b.y), "f"(b.x));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

}  // namespace lsh
