// The product of gemm_fp8.cuh for up to 16 rows of A (single-token serving).
//
// Such a product reads B once and does little else, so it is bound by memory,
// or at small sizes by one trip to memory and back.  A 128-row tcgen05 tile
// would be mostly zeros and starts late (tensor memory, descriptors, a
// pipeline to fill); here B streams through a ring in shared memory (cp.async:
// what is in flight costs no registers) in pieces of 16 bytes that a lane
// brings for itself, already in the fragment layout of mma.sync m16n8k32 (B's
// rows are its 16 rows, A's rows its 8 columns): a piece serves two MMAs, with
// the codes of K taken in the same permuted order from both operands.  (One row:
// 8192 x 2048 5.9 us, 16 384 x 8192 27 us, 4.9 TB/s; with loads into registers,
// which wait between batches, 6.7 and 39; these and codes converted to fp16
// first, m16n8k16, 8.9 and 53.  16 rows: 7.5 and 36 us, tcgen05 tiles 8.8 and
// 39.)
//
// A block of kW warps has 16 rows of B; its warps share out K in chunks of 128,
// scale each chunk's sum into fp32 totals, and add the totals up through shared
// memory in a fixed order.  To put the result into 8 bits (1 x 128 blocks along
// B's rows), the eight blocks of a cluster, 128 rows of B together, exchange
// their largest magnitudes through distributed shared memory.
#pragma once

#include "gemm_fp8_tc.cuh"

namespace lsh {

constexpr int kSkMaxM = 16;

struct Fp8SkinnyArgs {
  Fp8GemmArgs g;
  uint8_t* Q;   // kF8Quant, as in Fp8TcArgs
  float* qs;
  int prefetch_b;  // 1: B's first pieces go to L2 while the previous grid ends
};

__device__ __forceinline__ void mma_sync_e4m3(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes into shared memory, asynchronously; zeros if !in.  (Through L2, as
// the grid may have started before the one that wrote the data ended.)
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
constexpr int kSkRows = 16;
// Chunks in flight per warp (2 KB each; three or six: no faster), and the
// shared memory for them.
constexpr int kSkDeep = 4;
constexpr size_t sk_smem_bytes(int kW) { return (size_t)kSkDeep * kW * 2048; }

// kNT: column tiles of 8 (rows of A); kW: warps per block.
template <int kNT, int kW, int kEpi>
__global__ void __launch_bounds__(32 * kW) gemm_fp8_skinny_kernel(Fp8SkinnyArgs a) {
  constexpr int kSkThreads = 32 * kW;
  constexpr int kRows = kSkRows, kTok = 8 * kNT;
  __shared__ float red[kW][kRows][kTok + 1];
  __shared__ float cmax[128 / kRows][kTok];
  const Fp8GemmArgs& g = a.g;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gr = lane >> 2, tc4 = lane & 3;
  const int n0 = blockIdx.x * kRows;
  const int n_c = (g.K + 127) >> 7;
  // shared memory of another CTA may be written only once that CTA has started
  if (kEpi == kF8Quant) tc::cluster_arrive_relaxed();
  // a lane's own pieces [chunk in flight][row][half of the chunk]: nobody else
  // reads them, so the warps need no barrier
  extern __shared__ __align__(16) uint8_t ring[];
  constexpr uint32_t kPiece = kSkThreads * 16, kSlot = 4 * kPiece;
  uint8_t* const mine = ring + tid * 16;
  const uint32_t mine_at = tc::smem_u32(mine);
  const uint8_t* pb[2];  // rows n0 + gr and n0 + 8 + gr
  const float* psb[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = n0 + 8 * h + gr;
    pb[h] = n < g.N ? g.B + (size_t)n * g.K + 16 * tc4 : nullptr;
    psb[h] = g.sb + (size_t)(n < g.N ? n / g.b_rows : 0) * n_c;
  }
  const auto fetch = [&](int c, int slot) {
    if (c < n_c) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int k = c * 128 + 64 * half;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool in = pb[h] && k + 16 * tc4 < g.K;
          copy16(mine_at + slot * kSlot + (2 * h + half) * kPiece, in ? pb[h] + k : g.B, in);
        }
      }
    }
    copy_commit();
  };
  // Nothing is read before the grids before this one are done, since B may be
  // theirs; a prefetch to L2, where their writes go too, is no read.
  if (a.prefetch_b) {
#pragma unroll
    for (int d = 0; d < kSkDeep; ++d) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int k = (warp + kW * d) * 128 + 64 * half;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (pb[h] && k + 16 * tc4 < g.K)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(pb[h] + k) : "memory");
      }
    }
  }
  grid_dep_wait();
#pragma unroll
  for (int d = 0; d < kSkDeep; ++d) fetch(warp + kW * d, d);
  struct Side {  // what a chunk needs of A, and the scales, a chunk ahead
    uint4 av[kNT][2];
    float sa[kNT][2], sb[2];
  } next;
  const auto load_side = [&](int c) {
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
      const int m = 8 * t + gr;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int k = c * 128 + 64 * half + 16 * tc4;
        next.av[t][half] = make_uint4(0, 0, 0, 0);
        if (k < g.K && m < g.M)
          next.av[t][half] = *reinterpret_cast<const uint4*>(g.A + (size_t)m * g.K + k);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int ms = 8 * t + 2 * tc4 + h;
        next.sa[t][h] = ms < g.M ? g.sa[(size_t)ms * n_c + c] : 0.f;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) next.sb[h] = psb[h][c];
  };
  float acc[kNT][4] = {};
  if (warp < n_c) load_side(warp);
  int slot = 0;
  for (int c = warp; c < n_c; c += kW) {
    const Side now = next;
    if (c + kW < n_c) load_side(c + kW);
    copy_wait<kSkDeep - 1>();
    uint4 w[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int half = 0; half < 2; ++half)
        w[h][half] =
            *reinterpret_cast<const uint4*>(mine + slot * kSlot + (2 * h + half) * kPiece);
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
      float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint4 lo = w[0][half], hi = w[1][half], x = now.av[t][half];
        mma_sync_e4m3(p, lo.x, hi.x, lo.y, hi.y, x.x, x.y);
        mma_sync_e4m3(p, lo.z, hi.z, lo.w, hi.w, x.z, x.w);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[t][e] = fmaf(p[e], now.sa[t][e & 1] * now.sb[e >> 1], acc[t][e]);
    }
    // the MMAs have read the slot's pieces
    fetch(c + kW * kSkDeep, slot);
    slot = slot + 1 == kSkDeep ? 0 : slot + 1;
  }
  grid_dep_launch();
#pragma unroll
  for (int t = 0; t < kNT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      red[warp][gr + 8 * (e >> 1)][8 * t + 2 * tc4 + (e & 1)] = acc[t][e];
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
        tc::st_cluster(at, b);
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
      const float am = block_amax(b);
      a.Q[(size_t)m * g.N + n] =
          (uint8_t)__nv_cvt_float_to_fp8(scaled(v[i], relu_scale(am)), __NV_SATFINITE, __NV_E4M3);
      if ((n & 127) == 0) a.qs[(size_t)m * ((g.N + 127) >> 7) + (n >> 7)] = am / kE4m3Max;
    }
  }
}

}  // namespace lsh
