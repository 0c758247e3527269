// The product of gemm_fp8.cuh for up to 16 rows of A (single-token serving).
//
// Such a product reads B once and does little else, so it is bound by memory,
// or at small sizes by one trip to memory and back.  A 128-row tcgen05 tile
// would be mostly zeros and starts late (tensor memory, descriptors, a
// pipeline to fill); here B streams from memory into registers, already in the
// fragment layout of mma.sync m16n8k32 (B's rows are its 16 rows, A's rows its
// 8 columns): a lane's 16 bytes of a row serve two MMAs, with the codes of K
// taken in the same permuted order from both operands.  (The same through
// fp16, converted first, m16n8k16: 8.5 us in place of 6.7 at 1 x 8192 x 2048.)
//
// A block of kW warps has kRG groups of 16 rows of B; its warps share out K in
// chunks of 64, scale each chunk's sum (its block of 128 has one scale) into
// fp32 totals, and add the totals up through shared memory in a fixed order.
// To put the result into 8 bits (1 x 128 blocks along B's rows), the blocks of
// a cluster, 128 rows of B together, exchange their largest magnitudes through
// distributed shared memory.
#pragma once

#include "gemm_fp8_tc.cuh"

namespace lsh {

constexpr int kSkMaxM = 16;

struct Fp8SkinnyArgs {
  Fp8GemmArgs g;
  uint8_t* Q;   // kF8Quant, as in Fp8TcArgs
  float* qs;
  // 1: B is not written by the previous grid in the stream, nor by any that
  // may still run: its first loads need not wait for that grid
  int early_b;
};

__device__ __forceinline__ void mma_sync_e4m3(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (Not .nc: the grid may have started before the one that wrote the data ended.)
__device__ __forceinline__ uint4 load16_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// kNT: column tiles of 8 (rows of A); kRG: groups of 16 rows of B per block;
// kW: warps per block.
template <int kNT, int kRG, int kW, int kEpi>
__global__ void __launch_bounds__(32 * kW) gemm_fp8_skinny_kernel(Fp8SkinnyArgs a) {
  constexpr int kSkThreads = 32 * kW;
  constexpr int kDeep = kNT == 1 ? 4 : 2;  // chunks in flight per warp
  constexpr int kRows = 16 * kRG, kTok = 8 * kNT;
  __shared__ float red[kW][kRows][kTok + 1];
  __shared__ float cmax[128 / kRows][kTok];
  const Fp8GemmArgs& g = a.g;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gr = lane >> 2, tc4 = lane & 3;
  const int n0 = blockIdx.x * kRows;
  const int n_c = (g.K + 63) >> 6, kbs = (g.K + 127) >> 7;
  // shared memory of another CTA may be written only once that CTA has started
  if (kEpi == kF8Quant) tc::cluster_arrive_relaxed();
  if (!a.early_b) grid_dep_wait();
  float acc[kRG][kNT][4] = {};
  bool waited = !a.early_b;
  for (int c0 = warp; c0 < n_c; c0 += kW * kDeep) {
    uint4 wv[kDeep][kRG][2];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const int k = (c0 + kW * d) * 64 + 16 * tc4;
#pragma unroll
      for (int r = 0; r < kRG; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = n0 + 16 * r + 8 * h + gr;
          wv[d][r][h] = make_uint4(0, 0, 0, 0);
          if (k < g.K && n < g.N) wv[d][r][h] = load16_stream(g.B + (size_t)n * g.K + k);
        }
    }
    if (!waited) {
      grid_dep_wait();
      waited = true;
    }
    uint4 av[kDeep][kNT];
    float sa[kDeep][kNT][2], sb[kDeep][kRG][2];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      // past the end of K the codes are zero, and any scale will do
      const int c = c0 + kW * d, kb = c < n_c ? c >> 1 : 0;
      const int k = c * 64 + 16 * tc4;
#pragma unroll
      for (int t = 0; t < kNT; ++t) {
        const int m = 8 * t + gr;
        av[d][t] = make_uint4(0, 0, 0, 0);
        if (k < g.K && m < g.M)
          av[d][t] = *reinterpret_cast<const uint4*>(g.A + (size_t)m * g.K + k);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int ms = 8 * t + 2 * tc4 + h;
          sa[d][t][h] = ms < g.M ? g.sa[(size_t)ms * kbs + kb] : 0.f;
        }
      }
#pragma unroll
      for (int r = 0; r < kRG; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = n0 + 16 * r + 8 * h + gr;
          sb[d][r][h] = g.sb[(size_t)(n < g.N ? n / g.b_rows : 0) * kbs + kb];
        }
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      if (c0 + kW * d >= n_c) break;
#pragma unroll
      for (int t = 0; t < kNT; ++t)
#pragma unroll
        for (int r = 0; r < kRG; ++r) {
          float p[4] = {0.f, 0.f, 0.f, 0.f};
          const uint4 lo = wv[d][r][0], hi = wv[d][r][1], x = av[d][t];
          mma_sync_e4m3(p, lo.x, hi.x, lo.y, hi.y, x.x, x.y);
          mma_sync_e4m3(p, lo.z, hi.z, lo.w, hi.w, x.z, x.w);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[r][t][e] = fmaf(p[e], sa[d][t][e & 1] * sb[d][r][e >> 1], acc[r][t][e]);
        }
    }
  }
  if (!waited) grid_dep_wait();
  grid_dep_launch();
#pragma unroll
  for (int r = 0; r < kRG; ++r)
#pragma unroll
    for (int t = 0; t < kNT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        red[warp][16 * r + gr + 8 * (e >> 1)][8 * t + 2 * tc4 + (e & 1)] = acc[r][t][e];
  __syncthreads();
  // thread (token, row): neighbouring lanes have neighbouring rows of B, the
  // output's columns
  constexpr int kOut = kRows * kTok, kPer = (kOut + kSkThreads - 1) / kSkThreads;
  float v[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int o = tid + i * kSkThreads, r = o % kRows, m = o / kRows, n = n0 + r;
    v[i] = 0.f;
    if (o < kOut && n < g.N && m < g.M) {
#pragma unroll
      for (int w = 0; w < kW; ++w) v[i] += red[w][r][m];
      if (g.bias) v[i] += __bfloat162float(g.bias[n]);
      if (kEpi == kF8Quant || g.relu) v[i] = relu_nan(v[i]);
    }
  }
  if (kEpi == kF8Store) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int o = tid + i * kSkThreads, n = n0 + o % kRows, m = o / kRows;
      if (o < kOut && n < g.N && m < g.M) {
        if (g.c_f32)
          static_cast<float*>(g.C)[(size_t)m * g.N + n] = v[i];
        else
          static_cast<__nv_bfloat16*>(g.C)[(size_t)m * g.N + n] = __float2bfloat16_rn(v[i]);
      }
    }
  } else {
    // largest magnitude of this block's rows for each row of A, sent to every
    // block of the cluster
    constexpr int kCluster = 128 / kRows;
    const uint32_t rank = tc::cluster_rank();
    tc::cluster_wait();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int o = tid + i * kSkThreads, m = o / kRows;
      uint32_t b = mag_bits(v[i]);
#pragma unroll
      for (int s = kRows / 2; s; s >>= 1) b = max(b, __shfl_xor_sync(0xffffffffu, b, s));
      if (o < kOut && o % kRows < kCluster) {
        const uint32_t at = tc::cluster_map(tc::smem_u32(&cmax[rank][m]), (uint32_t)(o % kRows));
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(b) : "memory");
      }
    }
    tc::cluster_sync();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int o = tid + i * kSkThreads, n = n0 + o % kRows, m = o / kRows;
      if (o >= kOut || n >= g.N || m >= g.M) continue;
      uint32_t b = 0;
#pragma unroll
      for (int c = 0; c < kCluster; ++c) b = max(b, __float_as_uint(cmax[c][m]));
      const float am = block_amax(b), inv = kE4m3Max / am;
      a.Q[(size_t)m * g.N + n] = (uint8_t)__nv_cvt_float_to_fp8(v[i] * inv, __NV_SATFINITE, __NV_E4M3);
      if ((n & 127) == 0) a.qs[(size_t)m * ((g.N + 127) >> 7) + (n >> 7)] = am / kE4m3Max;
    }
  }
}

}  // namespace lsh
