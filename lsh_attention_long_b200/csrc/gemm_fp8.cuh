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

__device__ __forceinline__ float e4m3_to_f32(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// 64 x 64 outputs per block of 256 threads, 4 x 4 each.
__global__ void __launch_bounds__(256) gemm_fp8_simt_kernel(Fp8GemmArgs g) {
  __shared__ float as[32][65], bs[32][65];
  const int m0 = blockIdx.x * 64, n0 = blockIdx.y * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int kbs = (g.K + 127) >> 7;
  float acc[4][4] = {};
  for (int kb = 0; kb < kbs; ++kb) {
    float p[4][4] = {};
    for (int k0 = kb * 128; k0 < min(g.K, kb * 128 + 128); k0 += 32) {
      for (int i = threadIdx.x; i < 64 * 32; i += 256) {
        const int r = i >> 5, k = i & 31;
        const bool in = k0 + k < g.K;
        as[k][r] = in && m0 + r < g.M ? e4m3_to_f32(g.A[(size_t)(m0 + r) * g.K + k0 + k]) : 0.f;
        bs[k][r] = in && n0 + r < g.N ? e4m3_to_f32(g.B[(size_t)(n0 + r) * g.K + k0 + k]) : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 32; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) p[i][j] = fmaf(as[k][ty + 16 * i], bs[k][tx + 16 * j], p[i][j]);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + ty + 16 * i;
      if (m >= g.M) continue;
      const float sa = g.sa[(size_t)m * kbs + kb];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx + 16 * j;
        if (n < g.N) acc[i][j] = fmaf(p[i][j], sa * g.sb[(size_t)(n / g.b_rows) * kbs + kb], acc[i][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= g.M || n >= g.N) continue;
      float v = acc[i][j];
      if (g.bias) v += __bfloat162float(g.bias[n]);
      if (g.relu) v = v < 0.f ? 0.f : v;  // a NaN stays one
      if (g.c_f32)
        static_cast<float*>(g.C)[(size_t)m * g.N + n] = v;
      else
        static_cast<__nv_bfloat16*>(g.C)[(size_t)m * g.N + n] = __float2bfloat16_rn(v);
    }
}

}  // namespace lsh
