// The product of gemm_fp8.cuh on the 5th-generation tensor cores.
//
// The tensor cores multiply e4m3 codes and add in fp32, but know no scale per
// 128 entries of K.  So the sum of each block of 128 is an accumulator of its
// own: four tcgen05.mma of K = 32, the first overwriting, go into one of the
// 512 / kBN tensor-memory buffers, and the epilogue warps read it back and
// add it, times sa[m, kb] sb[n, kb], to their fp32 totals in registers.  A
// 128 x 256 tile's block is 512 cycles of tensor-core time; reading it back
// and one FMA per entry are 256 cycles each of what an SM's four schedulers
// can do in that time, so both fit beside it.
//
// Warp roles (320 threads, persistent blocks, one per SM):
//   warp 0     one thread loads A (128 rows) and B (kBN rows) tiles of 128
//              bytes with TMA (128-byte swizzle; zeros past the matrices'
//              ends) into a ring of kStages stages;
//   warp 1     one thread issues the tcgen05.mma;
//   warps 2-9  two warpgroups, one for each half of the tile's columns; a
//              thread has one row (its TMEM lane) and kBN / 2 totals.
#pragma once

#include <cuda.h>

#include "ffn_tc.cuh"
#include "gemm_fp8.cuh"
#include "tc.cuh"

namespace lsh {

constexpr int kF8Threads = 320;
constexpr int kF8BM = 128, kF8BK = 128;

enum Fp8Epi { kF8Store = 0, kF8Quant = 1 };

struct Fp8TcArgs {
  Fp8GemmArgs g;
  uint8_t* Q;      // kF8Quant: codes [M, N] of max(0, A B^T + bias)
  float* qs;       // and their 1 x 128 scales [M, ceil(N / 128)]
  long long wait_limit;
};

template <int kBN, bool kColScale>
struct Fp8Cfg {
  static constexpr int kStages = kBN == 128 ? 6 : kColScale ? 3 : 4;  // what 227 KB hold
  static constexpr int kABytes = kF8BM * kF8BK, kBBytes = kBN * kF8BK;
  static constexpr int kBufs = 512 / kBN;
  static constexpr int kOutBytes = 8 * 32 * 128;  // a staging row of 128 B per epilogue thread
};

template <int kBN, bool kColScale>
struct Fp8Smem {
  using C = Fp8Cfg<kBN, kColScale>;
  // b_rows 1: a block's column scales, by parity and column
  float sb[2][kColScale ? kBN : 4];
  uint64_t full[C::kStages], empty[C::kStages];
  uint64_t acc_full[C::kBufs], acc_empty[C::kBufs];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};

template <int kBN, bool kColScale>
__host__ __device__ constexpr size_t fp8_tc_smem_bytes() {
  using C = Fp8Cfg<kBN, kColScale>;
  return 1024 + (size_t)C::kStages * (C::kABytes + C::kBBytes) + C::kOutBytes +
         sizeof(Fp8Smem<kBN, kColScale>);
}
static_assert(fp8_tc_smem_bytes<256, false>() <= 232448 && fp8_tc_smem_bytes<256, true>() <= 232448 &&
                  fp8_tc_smem_bytes<128, true>() <= 232448,
              "shared memory of a block");

// OR of pred over the 256 epilogue threads (named barrier 3).
__device__ __forceinline__ bool f8_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 3, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred)
      : "memory");
  return r != 0;
}

template <int kBN, int kEpi, bool kColScale>
__global__ void __launch_bounds__(kF8Threads, 1)
    gemm_fp8_tc_kernel(const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_b, Fp8TcArgs a) {
  using C = Fp8Cfg<kBN, kColScale>;
  using Smem = Fp8Smem<kBN, kColScale>;
  static_assert(kEpi != kF8Quant || kBN == 256, "a thread's columns are one block");
  constexpr int kStages = C::kStages, kBufs = C::kBufs;
  constexpr int kCols = kBN / 2;  // columns of an epilogue thread
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = tc::smem_u32(smem_raw);
  uint8_t* sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* stage_a = sm;
  uint8_t* stage_b = sm + kStages * C::kABytes;
  uint8_t* stage_out = stage_b + kStages * C::kBBytes;
  Smem& S = *reinterpret_cast<Smem*>(stage_out + C::kOutBytes);
  const Fp8GemmArgs& g = a.g;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long limit = a.wait_limit;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&S.full[s], 1);
      tc::mbar_init(&S.empty[s], 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      tc::mbar_init(&S.acc_full[b], 1);
      tc::mbar_init(&S.acc_empty[b], 256);
    }
    tc::mbar_init(&S.mma_done, 1);
    tc::mbar_init_fence();
    S.abort = 0;
  }
  if (warp == 1) {
    tc::tmem_alloc(&S.tmem_base, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t tmem = S.tmem_base;
  const int n_n = (g.N + kBN - 1) / kBN;
  const int n_units = ((g.M + kF8BM - 1) / kF8BM) * n_n;
  const int n_k = (g.K + kF8BK - 1) / kF8BK;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA loads
    if (lane == 0) {
      uint32_t q = 0;  // K blocks loaded
      for (int u = blockIdx.x; u < n_units && !*(volatile int*)&S.abort; u += gridDim.x) {
        const int m0 = (u / n_n) * kF8BM, n0 = (u % n_n) * kBN;
        for (int kb = 0; kb < n_k; ++kb, ++q) {
          const int s = q % kStages;
          if (!gm_wait(&S.empty[s], ((q / kStages) & 1u) ^ 1u, &S.abort, limit)) break;
          tc::mbar_expect_tx(&S.full[s], C::kABytes + C::kBBytes);
          tc::tma_load_2d(tc::smem_u32(stage_a + s * C::kABytes), &map_a, kb * kF8BK, m0, &S.full[s]);
          tc::tma_load_2d(tc::smem_u32(stage_b + s * C::kBBytes), &map_b, kb * kF8BK, n0, &S.full[s]);
        }
      }
      // every load issued has landed before the block leaves
      const uint32_t first = q > (uint32_t)kStages ? q - kStages : 0;
      for (uint32_t p = first; p < q; ++p) {
        const long long t0 = clock64();
        while (!tc::mbar_test(&S.full[p % kStages], (p / kStages) & 1u)) {
          if (clock64() - t0 > limit) {
            record_status(tc::kErrTimeout);
            break;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issue
    if (lane == 0) {
      constexpr uint32_t idesc = tc::idesc_e4m3(kF8BM, kBN);
      uint32_t q = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
        for (int kb = 0; kb < n_k; ++kb, ++q) {
          const int s = q % kStages, b = q % kBufs;
          if (!gm_wait(&S.acc_empty[b], ((q / kBufs) & 1u) ^ 1u, &S.abort, limit) ||
              !gm_wait(&S.full[s], (q / kStages) & 1u, &S.abort, limit)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint64_t da = tc::sdesc_sw128(tc::smem_u32(stage_a + s * C::kABytes), 16, 1024);
          const uint64_t db = tc::sdesc_sw128(tc::smem_u32(stage_b + s * C::kBBytes), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 32 codes = two 16-byte units along K
            tc::mma_e4m3(tmem + b * kBN, da + 2 * kk, db + 2 * kk, idesc, kk > 0 ? 1u : 0u);
          tc::mma_commit(&S.empty[s]);
          tc::mma_commit(&S.acc_full[b]);
        }
      }
      // every MMA issued has finished before tensor memory is freed
      tc::mma_commit(&S.mma_done);
      const long long t0 = clock64();
      while (!tc::mbar_test(&S.mma_done, 0)) {
        if (clock64() - t0 > limit) {
          record_status(tc::kErrTimeout);
          break;
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int sub = warp & 3;          // TMEM lanes 32 * sub .. 32 * sub + 31
    const int half = (warp - 2) >> 2;  // which half of the tile's columns
    const int et = (sub << 5) | lane;  // row in the tile
    uint8_t* stg = stage_out + (warp - 2) * (32 * 128);
    uint8_t* my_row = stg + lane * 128;
    const uint32_t lane_base = tmem + ((uint32_t)(sub * 32) << 16) + half * kCols;
    uint32_t q = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < n_units; u += gridDim.x) {
      const int m0 = (u / n_n) * kF8BM, c0 = (u % n_n) * kBN + half * kCols;
      const int row = m0 + et;
      const float* sa = g.sa + (size_t)(row < g.M ? row : 0) * n_k;
      // past N every code is zero, and any finite scale will do
      const int nb = kColScale ? 0 : (c0 < g.N ? c0 : 0) / g.b_rows;
      const float* sb = g.sb + (size_t)nb * n_k;
      float acc[kCols];
#pragma unroll
      for (int e = 0; e < kCols; ++e) acc[e] = 0.f;
      float s_next = sa[0] * (kColScale ? 1.f : sb[0]);
      for (int kb = 0; kb < n_k; ++kb, ++q) {
        const int b = q % kBufs;
        const float s = s_next;
        if (kb + 1 < n_k) s_next = sa[kb + 1] * (kColScale ? 1.f : sb[kb + 1]);
        float* cs = S.sb[kb & 1] + half * kCols;
        if (kColScale) {
          // this block's column scales: written while the other parity may
          // still be read; the barrier orders both
          if (et < kCols) cs[et] = c0 + et < g.N ? g.sb[(size_t)(c0 + et) * n_k + kb] : 0.f;
          asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory");
        }
        // after an abort every wait returns at once; the loop runs on to its
        // end (reading stale totals), since the warps share its barriers
        ok &= gm_wait(&S.acc_full[b], (q / kBufs) & 1u, &S.abort, limit);
        tc::fence_after_sync();
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) {
          float v[32];
          tc::tmem_ld32(lane_base + b * kBN + 32 * c, v);
          tc::tmem_ld_wait();
          tc::tmem_pin<32>(v);
          if (c == kCols / 32 - 1) {  // the buffer is read: free it
            tc::fence_before_sync();
            tc::mbar_arrive(&S.acc_empty[b]);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e)
            acc[32 * c + e] = fmaf(v[e], kColScale ? s * cs[32 * c + e] : s, acc[32 * c + e]);
        }
      }
      if (f8_any(!ok)) break;  // all of them, or none
      const bool live = row < g.M;
      if (g.bias) {
#pragma unroll
        for (int e = 0; e < kCols; e += 8) {
          if (c0 + e < g.N) {
            float bv[8];
            load8(g.bias + c0 + e, bv);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[e + i] += bv[i];
          }
        }
      }
      if (kEpi == kF8Quant || g.relu) {
#pragma unroll
        for (int e = 0; e < kCols; ++e) acc[e] = acc[e] < 0.f ? 0.f : acc[e];  // a NaN stays one
      }
      if (kEpi == kF8Quant) {
        // the thread's 128 columns are one block of its row (kBN = 256)
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < kCols; ++e) m = max(m, c0 + e < g.N ? mag_bits(acc[e]) : 0u);
        const float am = block_amax(m), inv = kE4m3Max / am;
        if (live && c0 < g.N)
          a.qs[(size_t)row * ((g.N + 127) >> 7) + (c0 >> 7)] = am / kE4m3Max;
#pragma unroll
        for (int p = 0; p < kCols / 16; ++p) {
          const float* v = acc + 16 * p;
          *reinterpret_cast<uint4*>(my_row + ((p ^ (lane & 7)) << 4)) = make_uint4(
              e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
              e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv),
              e4m3x4(v[8] * inv, v[9] * inv, v[10] * inv, v[11] * inv),
              e4m3x4(v[12] * inv, v[13] * inv, v[14] * inv, v[15] * inv));
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int rl = 4 * k + (lane >> 3), p = lane & 7;
          const int r = m0 + sub * 32 + rl, col = c0 + 16 * p;
          const uint4 w = *reinterpret_cast<const uint4*>(stg + rl * 128 + ((p ^ (rl & 7)) << 4));
          if (r < g.M && col < g.N) *reinterpret_cast<uint4*>(a.Q + (size_t)r * g.N + col) = w;
        }
        __syncwarp();
      } else if (!g.c_f32) {
        // 64 columns of bf16 fill a staging row; eight lanes write it out
#pragma unroll
        for (int h = 0; h < kCols / 64; ++h) {
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            const float* v = acc + 64 * h + 8 * p;
            *reinterpret_cast<uint4*>(my_row + ((p ^ (lane & 7)) << 4)) =
                make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                           pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int rl = 4 * k + (lane >> 3), p = lane & 7;
            const int r = m0 + sub * 32 + rl, col = c0 + 64 * h + 8 * p;
            const uint4 w = *reinterpret_cast<const uint4*>(stg + rl * 128 + ((p ^ (rl & 7)) << 4));
            if (r < g.M && col < g.N)
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(g.C) + (size_t)r * g.N + col) = w;
          }
          __syncwarp();
        }
      } else {
#pragma unroll
        for (int h = 0; h < kCols / 32; ++h) {
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            const float* v = acc + 32 * h + 4 * p;
            *reinterpret_cast<float4*>(my_row + ((p ^ (lane & 7)) << 4)) =
                make_float4(v[0], v[1], v[2], v[3]);
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int rl = 4 * k + (lane >> 3), p = lane & 7;
            const int r = m0 + sub * 32 + rl, col = c0 + 32 * h + 4 * p;
            const float4 w =
                *reinterpret_cast<const float4*>(stg + rl * 128 + ((p ^ (rl & 7)) << 4));
            if (r < g.M && col < g.N)
              *reinterpret_cast<float4*>(static_cast<float*>(g.C) + (size_t)r * g.N + col) = w;
          }
          __syncwarp();
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

}  // namespace lsh
