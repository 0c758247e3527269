// Root-mean-square norm with the residual's addition, forward and backward.
//
//   h = x + r (rounded to x's type, and normalised as rounded),
//   rstd = 1 / sqrt(mean(h^2) + eps),   y = h rstd w.
// y leaves as fp32, bf16 or e4m3 with a scale per 128 columns (fp8.cuh).
//
// One pass over the data: a row stays in registers between the sum of its
// squares and the scaling, so each input is read and each output written
// once, and the kernels are bound by memory (in a graph of such calls, 65 536 x
// 512, fp32 stream and bf16 residual to 8 bits: 58 us, 6.4 TB/s; gradients of
// 16 384 x 2048 fp32: 77 us, 6.1 TB/s), but for the gradients of rows of more
// than 8192 columns, whose registers spill (4096 x 16 384: 960 us fp32, 800
// bf16, of 143 and 82 that memory would take).  Rows of up to 1024 columns are
// a warp's (no barrier), longer ones a block's of 256 to 1024 threads (with 256
// threads for all of them, 4096 x 8192 bf16 took 1.3 times as long); a thread
// holds kNV pieces of 8 consecutive columns, piece t + i * kT, so that 16
// neighbouring lanes hold one block of 128 and a warp's loads are contiguous.
#pragma once

#include "fp8.cuh"

namespace lsh {

enum NormOut { kNormF32 = 0, kNormBf16 = 1, kNormE4m3 = 2 };

constexpr int kNormWarpCols = 1024;   // longest row of the warp kernels
constexpr int kNormMaxCols = 16384;   // 1024 threads x 2 pieces x 8 columns
// threads of a block whose rows have kT threads each: eight rows, or one
__host__ __device__ constexpr int norm_block(int kT) { return kT == 32 ? 256 : kT; }

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

// Sum over the row's kT threads: a warp, or the block (two barriers; `red` holds
// one float per warp and may be used again after the next call's first).
template <int kT>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if (kT == 32) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  v = warp_sum(lane < kT / 32 ? red[lane] : 0.f);
  __syncthreads();
  return v;
}

// Eight neighbouring entries as loaded, fp32 or bf16: every load of a row is
// under way before the first is unpacked.
struct Raw8 {
  uint4 a, b;
  __device__ __forceinline__ void load(const void* p, bool bf16, size_t at) {
    if (bf16) {
      a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at);
    } else {
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
      a = q[0];
      b = q[1];
    }
  }
  __device__ __forceinline__ void get(bool bf16, float* v) const {
    if (bf16) {
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    }
  }
};

template <typename XT, int kOut, int kNV, int kT>
__global__ void __launch_bounds__(norm_block(kT), kT == 256 && kNV == 1 ? 8 : 1)  // 8: a full SM
    rmsnorm_fwd_kernel(NormArgs a) {
  __shared__ float red[32];
  grid_dep_wait();
  grid_dep_launch();
  const int t = threadIdx.x & (kT - 1);
  const long long row = (long long)blockIdx.x * (norm_block(kT) / kT) + threadIdx.x / kT;
  if (row >= a.rows) return;  // a whole warp, or nobody (one row per block)
  const size_t base = (size_t)row * a.cols;
  const int pieces = a.cols >> 3;
  constexpr bool kXBf = sizeof(XT) == 2;
  float h[kNV][8];
  {
    Raw8 x[kNV], r[kNV];
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int p = t + i * kT;
      if (p >= pieces) continue;
      x[i].load(a.x, kXBf, base + 8 * p);
      if (a.r) r[i].load(a.r, a.r_bf16, base + 8 * p);
    }
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int p = t + i * kT;
      if (p >= pieces) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = 0.f;
        continue;
      }
      x[i].get(kXBf, h[i]);
      if (a.r) {
        float rv[8];
        r[i].get(a.r_bf16, rv);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = to_f32(from_f32<XT>(h[i][e] + rv[e]));
        store8(static_cast<XT*>(a.h) + base + 8 * p, h[i]);
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kNV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(h[i][e], h[i][e], ss);
  ss = row_sum<kT>(ss, red);
  const float rstd = rsqrtf(ss / (float)a.cols + a.eps);
  if (a.rstd && t == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int p = t + i * kT;
    const bool in = p < pieces;
    float w[8];
    if (in) {
      Raw8 wr;
      wr.load(a.w, a.w_bf16, 8 * p);
      wr.get(a.w_bf16, w);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) h[i][e] = in ? h[i][e] * rstd * w[e] : 0.f;
    if (kOut == kNormE4m3) {
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, mag_bits(h[i][e]));
#pragma unroll
      for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float am = block_amax(m);
      const BlockScale sc(am);
      if (in) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + base + 8 * p) =
            scale_to_e4m3<false>(h[i], sc);
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
template <typename XT, int kNV, int kT>
__global__ void __launch_bounds__(norm_block(kT)) rmsnorm_bwd_kernel(NormBwdArgs a) {
  __shared__ float red[32];
  __shared__ float part[kT == 32 ? 8 : 1][kT == 32 ? kNV * 256 : 1];
  grid_dep_wait();
  grid_dep_launch();
  constexpr int kRows = norm_block(kT) / kT;  // rows in flight per block
  const int t = threadIdx.x & (kT - 1);
  const int pieces = a.cols >> 3;
  constexpr bool kXBf = sizeof(XT) == 2;
  float dw[kNV][8];
#pragma unroll
  for (int i = 0; i < kNV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
  const float inv_cols = 1.f / (float)a.cols;
  // The next row's loads travel while this one is reduced and written (fp32,
  // 65536 x 512: 81 us, 108 without; bf16, 8192 x 4096: 61 us, 93 without).
  Raw8 hr[kNV], gr[kNV], dr[kNV];
  float rstd_next = 0.f;
  const auto load_row = [&](long long row) {
    const size_t base = (size_t)row * a.cols;
    rstd_next = a.rstd[row];
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int p = t + i * kT;
      if (p >= pieces) continue;
      hr[i].load(a.h, kXBf, base + 8 * p);
      gr[i].load(a.dy, a.dy_bf16, base + 8 * p);
      if (a.dh) dr[i].load(a.dh, kXBf, base + 8 * p);
    }
  };
  const long long step = (long long)gridDim.x * kRows;
  long long row = (long long)blockIdx.x * kRows + threadIdx.x / kT;
  if (row < a.rows) load_row(row);
  for (; row < a.rows; row += step) {
    const size_t base = (size_t)row * a.cols;
    const float rstd = rstd_next;
    float n[kNV][8], g[kNV][8];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int p = t + i * kT;
      if (p >= pieces) continue;
      Raw8 wr;
      float w[8];
      wr.load(a.w, a.w_bf16, 8 * p);
      hr[i].get(kXBf, n[i]);
      gr[i].get(a.dy_bf16, g[i]);
      wr.get(a.w_bf16, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[i][e] *= rstd;
        dw[i][e] = fmaf(g[i][e], n[i][e], dw[i][e]);
        g[i][e] *= w[e];
        dot = fmaf(g[i][e], n[i][e], dot);
      }
    }
    float up[kNV][8];  // the gradient past the norm
#pragma unroll
    for (int i = 0; i < kNV; ++i)
      if (a.dh) dr[i].get(kXBf, up[i]);
    if (row + step < a.rows) load_row(row + step);
    const float mean = row_sum<kT>(dot, red) * inv_cols;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int p = t + i * kT;
      if (p >= pieces) continue;
      float* v = up[i];
      if (!a.dh) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += rstd * (g[i][e] - n[i][e] * mean);
      store8(static_cast<XT*>(a.dx) + base + 8 * p, v);
    }
  }
  if (kT == 32) {  // the warps' sums, added in order of warp
#pragma unroll
    for (int i = 0; i < kNV; ++i) store8(part[threadIdx.x >> 5] + 8 * (t + i * 32), dw[i]);
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += 256) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += part[kT == 32 ? i : 0][kT == 32 ? c : 0];
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

// out[c] = sum over b of part[b][c]: a block sums 32 columns, its 32 warps
// every 32nd row each, eight loads under way at a time, and adds the warps up
// in a fixed order.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* part, int blocks, int cols,
                                                          float* out) {
  __shared__ float red[32][33];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < cols)
    for (int b0 = warp; b0 < blocks; b0 += 8 * 32) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = b0 + 32 * i < blocks ? part[(size_t)(b0 + 32 * i) * cols + c] : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
  red[warp][lane] = s;
  __syncthreads();
  // warp w adds up column w
  const float v = warp_sum(red[lane][warp]);
  if (lane == 0 && blockIdx.x * 32 + warp < cols) out[blockIdx.x * 32 + warp] = v;
}

}  // namespace lsh
