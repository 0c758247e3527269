// Root-mean-square norm with the residual's addition, forward and backward.
//
//   h = x + r (rounded to x's type, and normalised as rounded),
//   rstd = 1 / sqrt(mean(h^2) + eps),   y = h rstd w.
// y leaves as fp32, bf16 or e4m3 with a scale per 128 columns (fp8.cuh).
//
// One pass over the data: a row stays in registers between the sum of its
// squares and the scaling, so each input is read and each output written
// once, and the kernels are bound by memory.  Rows of up to 1024 columns are
// a warp's (no barrier), longer ones a 256-thread block's; a thread holds
// kNV pieces of 8 consecutive columns, piece t + i * threads, so that 16
// neighbouring lanes hold one block of 128 and a warp's loads are contiguous.
#pragma once

#include "fp8.cuh"

namespace lsh {

enum NormOut { kNormF32 = 0, kNormBf16 = 1, kNormE4m3 = 2 };

constexpr int kNormThreads = 256;
constexpr int kNormWarpCols = 1024;   // longest row of the warp kernels
constexpr int kNormMaxCols = 16384;   // 256 threads x 8 pieces x 8 columns

struct NormArgs {
  long long rows;
  int cols;         // multiple of 16
  int r_bf16;       // type of r: bf16, else x's
  int w_bf16;       // type of w: bf16, else fp32
  const void* x;
  const void* r;    // or NULL
  const void* w;
  float eps;
  void* h;          // x's type; NULL when r is
  void* y;
  float* scales;    // kNormE4m3: [rows, ceil(cols / 128)]
  float* rstd;      // [rows] or NULL
};

struct NormBwdArgs {
  long long rows;
  int cols;
  int dy_bf16;      // type of dy: bf16, else fp32
  int w_bf16;
  const void* dy;
  const void* h;
  const void* w;
  const float* rstd;
  const void* dh;   // gradient that reaches h past the norm (x's type), or NULL
  void* dx;         // x's type
  float* dw;        // [blocks, cols] partial sums (one block: dw itself)
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the row's threads: a warp, or the block (two barriers; `red` holds
// one float per warp and may be used again after the next call's first).
template <bool kWarp>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if (kWarp) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kNormThreads / 32; ++i) s += red[i];
  __syncthreads();
  return s;
}

__device__ __forceinline__ void load8_any(const void* p, int is_bf16, size_t at, float* v) {
  if (is_bf16)
    load8(static_cast<const __nv_bfloat16*>(p) + at, v);
  else
    load8(static_cast<const float*>(p) + at, v);
}

template <typename XT, int kOut, int kNV, bool kWarp>
__global__ void __launch_bounds__(kNormThreads) rmsnorm_fwd_kernel(NormArgs a) {
  __shared__ float red[kNormThreads / 32];
  grid_dep_wait();
  grid_dep_launch();
  constexpr int kT = kWarp ? 32 : kNormThreads;  // threads of a row
  const int t = threadIdx.x & (kT - 1);
  const long long row = (long long)blockIdx.x * (kNormThreads / kT) + threadIdx.x / kT;
  if (row >= a.rows) return;  // a whole warp, or nobody (one row per block)
  const size_t base = (size_t)row * a.cols;
  const int pieces = a.cols >> 3;
  const XT* x = static_cast<const XT*>(a.x) + base;
  float h[kNV][8];
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int p = t + i * kT;
    if (p < pieces) {
      load8(x + 8 * p, h[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] = 0.f;
    }
  }
  if (a.r) {
    float r[kNV][8];
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int p = t + i * kT;
      if (p < pieces) load8_any(a.r, a.r_bf16, base + 8 * p, r[i]);
    }
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int p = t + i * kT;
      if (p >= pieces) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] = to_f32(from_f32<XT>(h[i][e] + r[i][e]));
      store8(static_cast<XT*>(a.h) + base + 8 * p, h[i]);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kNV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(h[i][e], h[i][e], ss);
  ss = row_sum<kWarp>(ss, red);
  const float rstd = rsqrtf(ss / (float)a.cols + a.eps);
  if (a.rstd && t == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int p = t + i * kT;
    const bool in = p < pieces;
    float w[8];
    if (in) load8_any(a.w, a.w_bf16, 8 * p, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[i][e] = in ? h[i][e] * rstd * w[e] : 0.f;
    if (kOut == kNormE4m3) {
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, mag_bits(h[i][e]));
#pragma unroll
      for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float am = block_amax(m), inv = kE4m3Max / am;
      if (in) {
        const uint2 q = make_uint2(
            e4m3x4(h[i][0] * inv, h[i][1] * inv, h[i][2] * inv, h[i][3] * inv),
            e4m3x4(h[i][4] * inv, h[i][5] * inv, h[i][6] * inv, h[i][7] * inv));
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + base + 8 * p) = q;
        if ((p & 15) == 0)
          a.scales[(size_t)row * ((a.cols + 127) >> 7) + (p >> 4)] = am / kE4m3Max;
      }
    } else if (in) {
      if (kOut == kNormF32)
        store8(static_cast<float*>(a.y) + base + 8 * p, h[i]);
      else
        store8(static_cast<__nv_bfloat16*>(a.y) + base + 8 * p, h[i]);
    }
  }
}

// Backward.  With n = h rstd and g = w dy,
//   dx = rstd (g - n mean(g n)) + dh,   dw = sum over rows of dy n.
// Blocks are persistent over rows; a thread meets the same columns in every
// row and keeps their dw in registers (fp32).  Blocks leave one partial row
// each, which a second launch adds up in a fixed order: no atomics, so the
// same call gives the same bits.
template <typename XT, int kNV, bool kWarp>
__global__ void __launch_bounds__(kNormThreads) rmsnorm_bwd_kernel(NormBwdArgs a) {
  __shared__ float red[kNormThreads / 32];
  __shared__ float part[kWarp ? kNormThreads / 32 : 1][kWarp ? kNV * 256 : 1];
  grid_dep_wait();
  grid_dep_launch();
  constexpr int kT = kWarp ? 32 : kNormThreads;
  constexpr int kRows = kNormThreads / kT;  // rows in flight per block
  const int t = threadIdx.x & (kT - 1);
  const int pieces = a.cols >> 3;
  const XT* hp = static_cast<const XT*>(a.h);
  const XT* dhp = static_cast<const XT*>(a.dh);
  float dw[kNV][8];
#pragma unroll
  for (int i = 0; i < kNV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
  const float inv_cols = 1.f / (float)a.cols;
  for (long long row = (long long)blockIdx.x * kRows + threadIdx.x / kT; row < a.rows;
       row += (long long)gridDim.x * kRows) {
    const size_t base = (size_t)row * a.cols;
    const float rstd = a.rstd[row];
    float n[kNV][8], g[kNV][8];
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int p = t + i * kT;
      if (p < pieces) {
        load8(hp + base + 8 * p, n[i]);
        load8_any(a.dy, a.dy_bf16, base + 8 * p, g[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) n[i][e] = g[i][e] = 0.f;
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int p = t + i * kT;
      if (p >= pieces) continue;
      float w[8];
      load8_any(a.w, a.w_bf16, 8 * p, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[i][e] *= rstd;
        dw[i][e] = fmaf(g[i][e], n[i][e], dw[i][e]);
        g[i][e] *= w[e];
        dot = fmaf(g[i][e], n[i][e], dot);
      }
    }
    const float mean = row_sum<kWarp>(dot, red) * inv_cols;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int p = t + i * kT;
      if (p >= pieces) continue;
      float v[8];
      if (dhp)
        load8(dhp + base + 8 * p, v);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += rstd * (g[i][e] - n[i][e] * mean);
      store8(static_cast<XT*>(a.dx) + base + 8 * p, v);
    }
  }
  if (kWarp) {  // the warps' sums, added in order of warp
#pragma unroll
    for (int i = 0; i < kNV; ++i) store8(part[threadIdx.x >> 5] + 8 * (t + i * 32), dw[i]);
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += kNormThreads) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kNormThreads / 32; ++i) s += part[kWarp ? i : 0][kWarp ? c : 0];
      a.dw[(size_t)blockIdx.x * a.cols + c] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int p = t + i * kT;
      if (p < pieces) store8(a.dw + (size_t)blockIdx.x * a.cols + 8 * p, dw[i]);
    }
  }
}

// out[c] = sum over b of part[b][c]: a block sums 32 columns, its 8 warps
// every eighth row each, and adds the warps up in a fixed order.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* __restrict__ part,
                                                         int blocks, int cols,
                                                         float* __restrict__ out) {
  __shared__ float red[8][32];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < cols)
    for (int b = warp; b < blocks; b += 8) s += part[(size_t)b * cols + c];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < cols) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += red[i][lane];
    out[c] = v;
  }
}

}  // namespace lsh
