// The product of gemm_fp8.cuh on the 5th-generation tensor cores.
//
// The tensor cores multiply e4m3 codes and add in fp32, but know no scale per
// 128 entries of K.  So the sum of each block of 128 is an accumulator of its
// own: four tcgen05.mma of K = 32, the first overwriting, go into one of the
// 512 / kBN tensor-memory buffers, and the epilogue warps read it back and
// add it, times sa[m, kb] sb[n, kb], to their fp32 totals in registers.  A
// 128 x 256 tile's block is 512 cycles of an SM's tensor core; reading it back
// is 256 cycles of tensor memory and one packed FMA per two entries 128 of
// each scheduler's, so both fit beside it.
//
// kPair 2: two CTAs (a cluster) work on a 256 x 256 tile with pair MMAs.  Each
// loads its own 128 rows of A and half of B's, 32 KB per block of K in place
// of the 48 KB of a 128 x 256 tile alone, which the path from L2 would bound.
// kPair 1 (tiles of 128 x 128) serves products with few tiles; with kParts the
// CTAs of a cluster share out a tile's K and add their totals up through
// distributed shared memory.
//
// Measured: 8192 x 4096 x 4096 in 120 us over twenty warm calls (2 280 TFLOP/s,
// 60% of the tensor cores' cycles; with column scales 169 us), 134 and 190 us
// where the board's power sets the clock.  The busiest pair takes 837 cycles a
// block, of which 512 are its MMAs'; the epilogue with neither loads nor MMAs
// took 795, so it sets the pace.  Its parts measured alone do not add up to
// that: reading and adding 360 at best, and some 370 from commit to the next
// issue, would be 621 a block with two accumulators in turn.  (The forms on
// pairs spill 72 to 88 bytes a thread.)
//
// Warp roles (384 threads, persistent blocks, one per SM):
//   warp 0      one thread loads A and B tiles of 128-byte rows with TMA
//               (128-byte swizzle; zeros past the matrices' ends) into a ring
//               of kStages stages;
//   warps 1, 2  one lane each (of the pair's even rank) issues the tcgen05.mma
//               of every other block: the waits, four MMAs and two commits of
//               a block are some 680 cycles of one thread's time, more than
//               the 512 that the MMAs take;
//   warp 3      brings the scales: rows of sa (and, b_rows 1, of sb) lie n_k
//               apart, so a warp's load of one block's column touches 32 lines;
//               here each is loaded once, some blocks ahead, and reaches the
//               epilogue through a ring in shared memory;
//   warps 4-11  two warpgroups, one for each half of the tile's columns; a
//               thread has one row (its TMEM lane) and kBN / 2 totals.
#pragma once

#include <cuda.h>

#include "ffn_tc.cuh"
#include "gemm_fp8.cuh"
#include "tc.cuh"

namespace lsh {

constexpr int kF8Threads = 384;
// Registers: 168 a thread at launch (what 384 threads can have).  The first
// warpgroup gives some up, which twice as many warps share: most where an
// epilogue thread has 128 totals, fewer where the scales' warp has a tile's
// column scales in its own, fewest with 64 totals.
constexpr int kF8Regs = 168;
__host__ __device__ constexpr int f8_regs_low(int bn, bool col_scale) {
  return bn == 128 ? 104 : col_scale ? 88 : 56;
}
__host__ __device__ constexpr int f8_regs_high(int bn, bool col_scale) {
  return kF8Regs + (kF8Regs - f8_regs_low(bn, col_scale)) / 2;
}
constexpr int kF8BM = 128, kF8BK = 128;

constexpr int kF8Slots = 2;  // ring of scales, in four blocks of K

enum Fp8Epi { kF8Store = 0, kF8Quant = 1 };

struct Fp8TcArgs {
  Fp8GemmArgs g;
  uint8_t* Q;      // kF8Quant: codes [M, N] of max(0, A B^T + bias)
  float* qs;       // and their 1 x 128 scales [M, ceil(N / 128)]
  long long wait_limit;
  int hold_tile;   // test hook: the loads stop before this tile of each CTA (-1: never)
};

template <int kPair, int kBN, int kEpi, bool kColScale>
struct Fp8Cfg {
  static constexpr int kCols = kBN / 2;  // columns of an epilogue thread
  static constexpr int kABytes = kF8BM * kF8BK, kBBytes = kBN / kPair * kF8BK;
  static constexpr int kBufs = 512 / kBN;
  // staging of an epilogue warp: 32 rows of its columns in bf16 or e4m3 (fp32
  // leaves in two parts), as boxes of 32 rows of 128 bytes
  static constexpr int kOutBoxes = kEpi == kF8Quant ? 1 : kCols / 64;
  static constexpr int kOutBytes = 8 * kOutBoxes * 4096;
  static constexpr int kScaleBytes =
      kF8Slots * 4 * 4 * (kColScale ? kF8BM + kBN : 2 * kF8BM) + 4 * kBN * 4;
  static constexpr int kStages =  // what is left of 227 KB, less alignment and barriers
      (232448 - 1024 - 512 - kOutBytes - kScaleBytes) / (kABytes + kBBytes);
};

template <int kPair, int kBN, int kEpi, bool kColScale>
struct Fp8Smem {
  using C = Fp8Cfg<kPair, kBN, kEpi, kColScale>;
  // scales of the blocks to come, four to a slot: per half of the columns and
  // row sa * sb, or (b_rows 1) per row sa and per column sb
  float4 rs[kF8Slots][kColScale ? 1 : 2][kF8BM];
  float cs[kColScale ? kF8Slots : 1][4][kColScale ? kBN : 1];
  // the tile's bias, by tile: the scales' warp is at most two tiles ahead
  float4 bias[4][kBN / 4];
  uint64_t full[C::kStages], empty[C::kStages];
  uint64_t acc_full[C::kBufs], acc_empty[C::kBufs];
  uint64_t sc_full[kF8Slots], sc_empty[kF8Slots];
  uint64_t mma_done[2];
  uint32_t issued[2];  // by MMA warp: its first block of K that was not issued (in both CTAs)
  uint32_t amax[2][kEpi == kF8Quant && kBN == 128 ? kF8BM : 1];
  uint32_t tmem_base;
  int abort;
};

template <int kPair, int kBN, int kEpi, bool kColScale>
__host__ __device__ constexpr size_t fp8_tc_smem_bytes() {
  using C = Fp8Cfg<kPair, kBN, kEpi, kColScale>;
  constexpr size_t bytes = 1024 + (size_t)C::kStages * (C::kABytes + C::kBBytes) + C::kOutBytes +
                           sizeof(Fp8Smem<kPair, kBN, kEpi, kColScale>);
  static_assert(bytes <= 232448 && C::kStages >= 3, "shared memory of a block");
  return bytes;
}

constexpr int kChunk = 16;  // columns read back at a time

// Waits for a phase unless the CTA aborted; false on abort or timeout.  The
// clock is read only where the first look finds nothing.
__device__ __forceinline__ bool f8_wait(uint64_t* bar, uint32_t parity, int* abort,
                                        long long limit) {
  return tc::mbar_test(bar, parity) || gm_wait(bar, parity, abort, limit);
}

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

// About a millisecond.
__device__ __forceinline__ void f8_pause() {
  const long long t0 = clock64();
  while (clock64() - t0 < 2000000) {
  }
}

// The last block of K that went through barrier `at` of a ring of n, of those
// that the MMA warps issued (warp w the blocks w, w + 2, .. before issued[w]); -1: none.
__host__ __device__ inline int f8_last_block(const uint32_t* issued, int n, int at) {
  int last = -1;
  for (int w = 0; w < 2; ++w) {
    int q = (int)issued[w] - 2;
    for (int i = 0; i < n && q >= 0 && q % n != at; ++i) q -= 2;
    if (q >= 0 && q % n == at && q > last) last = q;
  }
  return last;
}

template <int kPair, int kBN, int kEpi, bool kColScale, int kParts>
__global__ void __launch_bounds__(kF8Threads, 1)
    gemm_fp8_tc_kernel(const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_b,
                       const __grid_constant__ CUtensorMap map_c, Fp8TcArgs a) {
  using C = Fp8Cfg<kPair, kBN, kEpi, kColScale>;
  using Smem = Fp8Smem<kPair, kBN, kEpi, kColScale>;
  constexpr bool kSplit = kParts > 1;
  static_assert(!kSplit || (kPair == 1 && kBN == 128 && kEpi == kF8Store), "split of K");
  constexpr int kStages = C::kStages, kBufs = C::kBufs;
  constexpr int kCols = C::kCols;
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
  const int rank = kPair == 2 ? (int)tc::cluster_rank() : 0;
  // kSplit: a cluster shares one tile's blocks of K
  const int part = kSplit ? (int)tc::cluster_rank() : 0;
  const int first_unit = blockIdx.x / (kPair * kParts), unit_step = gridDim.x / (kPair * kParts);

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(&S.full[s], 1);
      tc::mbar_init(&S.empty[s], 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      tc::mbar_init(&S.acc_full[b], 1);
      tc::mbar_init(&S.acc_empty[b], 8 * kPair);  // one arrival per epilogue warp
    }
    for (int b = 0; b < kF8Slots; ++b) {
      tc::mbar_init(&S.sc_full[b], 1);
      tc::mbar_init(&S.sc_empty[b], 8);
    }
    tc::mbar_init(&S.mma_done[0], 1);
    tc::mbar_init(&S.mma_done[1], 1);
    tc::mbar_init_fence();
    S.abort = 0;
  }
  if (warp == 1) {
    if (kPair == 2) {
      tc::tmem_alloc_pair(&S.tmem_base, 512);
      tc::tmem_relinquish_pair();
    } else {
      tc::tmem_alloc(&S.tmem_base, 512);
      tc::tmem_relinquish();
    }
  }
  tc::fence_before_sync();
  if (kPair == 2)
    tc::cluster_sync();  // the peer's barriers are set up too
  else
    __syncthreads();
  tc::fence_after_sync();
  grid_dep_wait();
  grid_dep_launch();
  const uint32_t tmem = S.tmem_base;
  const auto commit = [](uint64_t* bar) { kPair == 2 ? tc::mma_commit_pair(bar) : tc::mma_commit(bar); };
  const int n_n = (g.N + kBN - 1) / kBN;
  const int n_units = ((g.M + kPair * kF8BM - 1) / (kPair * kF8BM)) * n_n;
  const int k_all = (g.K + kF8BK - 1) / kF8BK;  // blocks of K: all, and this CTA's
  const int k_lo = kSplit ? part * k_all / kParts : 0;
  const int n_k = kSplit ? (part + 1) * k_all / kParts - k_lo : k_all;

  if (warp < 4) tc::reg_dec<f8_regs_low(kBN, kColScale)>();
  if (warp == 0) {
    // ------------------------------------------------------------ TMA loads
    if (lane == 0) {
      uint32_t q = 0;  // K blocks loaded
      int tile = 0;
      for (int u = first_unit; u < n_units && !*(volatile int*)&S.abort; u += unit_step, ++tile) {
        if (tile == a.hold_tile) break;
        const int m0 = (u / n_n * kPair + rank) * kF8BM;
        const int n0 = (u % n_n) * kBN + (rank * (kBN / kPair));
        for (int kb = 0; kb < n_k; ++kb, ++q) {
          const int s = q % kStages;
          if (!gm_wait(&S.empty[s], ((q / kStages) & 1u) ^ 1u, &S.abort, limit)) break;
          const uint32_t sa = tc::smem_u32(stage_a + s * C::kABytes);
          const uint32_t sb = tc::smem_u32(stage_b + s * C::kBBytes);
          if (kPair == 2) {
            // both ranks' loads complete on the even rank's barrier, which
            // expects them all
            if (rank == 0) tc::mbar_expect_tx(&S.full[s], 2 * (C::kABytes + C::kBBytes));
            const uint32_t bar = tc::cluster_map(tc::smem_u32(&S.full[s]), 0);
            tc::tma_load_2d_pair(sa, &map_a, (k_lo + kb) * kF8BK, m0, bar);
            tc::tma_load_2d_pair(sb, &map_b, (k_lo + kb) * kF8BK, n0, bar);
          } else {
            tc::mbar_expect_tx(&S.full[s], C::kABytes + C::kBBytes);
            tc::tma_load_2d(sa, &map_a, (k_lo + kb) * kF8BK, m0, &S.full[s]);
            tc::tma_load_2d(sb, &map_b, (k_lo + kb) * kF8BK, n0, &S.full[s]);
          }
        }
      }
      // Every load issued has landed before the block leaves: the even rank
      // (which leaves together with the odd one) waits for the last stages.
      // After an abort one rank may have issued loads that the other's barrier
      // does not expect; then both give them time, far more than a load takes.
      if (kPair == 2 && *(volatile int*)&S.abort) {
        f8_pause();
      } else {
        const uint32_t first = rank ? q : q > (uint32_t)kStages ? q - kStages : 0;
        for (uint32_t p = first; p < q; ++p)
          if (!tc::mbar_wait(&S.full[p % kStages], (p / kStages) & 1u))
            record_status(tc::kErrTimeout);
      }
    }
    __syncwarp();
  } else if (warp <= 2) {
    // ------------------------------------------------------------ MMA issue
    // The whole warp runs the loop, so that its addresses stay uniform; one
    // lane issues.
    if (rank == 0) {
      constexpr uint32_t idesc = tc::idesc_e4m3(kPair * kF8BM, kBN);
      // all the blocks of this CTA's tiles, one after the other
      const uint32_t n_q = (n_units - first_unit + unit_step - 1) / unit_step * (uint32_t)n_k;
      uint32_t q = warp - 1;
      for (; q < n_q; q += 2) {
          const int s = q % kStages, b = q % kBufs;
          bool ok = f8_wait(&S.full[s], (q / kStages) & 1u, &S.abort, limit);
          const uint64_t da = tc::sdesc_sw128(tc::smem_u32(stage_a + s * C::kABytes), 16, 1024);
          ok = ok && f8_wait(&S.acc_empty[b], ((q / kBufs) & 1u) ^ 1u, &S.abort, limit);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc::fence_after_sync();
          const uint64_t db = tc::sdesc_sw128(tc::smem_u32(stage_b + s * C::kBBytes), 16, 1024);
          const uint32_t d = tmem + b * kBN;
          if (tc::elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {  // 32 codes = two 16-byte units along K
              if (kPair == 2)
                tc::mma_e4m3_pair(d, da + 2 * kk, db + 2 * kk, idesc, kk > 0 ? 1u : 0u);
              else
                tc::mma_e4m3(d, da + 2 * kk, db + 2 * kk, idesc, kk > 0 ? 1u : 0u);
            }
            commit(&S.acc_full[b]);
            commit(&S.empty[s]);
          }
          __syncwarp();
      }
      // every MMA issued has finished before tensor memory is freed
      if (tc::elect_one()) {
        commit(&S.mma_done[warp - 1]);
        if (!tc::mbar_wait(&S.mma_done[warp - 1], 0)) record_status(tc::kErrTimeout);
        S.issued[warp - 1] = q;
        if (kPair == 2)
          tc::st_cluster(tc::cluster_map(tc::smem_u32(&S.issued[warp - 1]), 1), q);
      }
    }
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------------------ scales
    // Lane t has rows t, t + 32, .. (and columns t, t + 32, ..); four blocks'
    // scales are in flight at once.
    constexpr int kC = kColScale ? kBN / 32 : 2;
    const bool vec = k_all % 4 == 0 && k_lo % 4 == 0;
    uint32_t q = 0, tile = 0;
    bool ok = true;
    for (int u = first_unit; u < n_units && ok; u += unit_step, ++tile) {
      const int m0 = (u / n_n * kPair + rank) * kF8BM, n0 = (u % n_n) * kBN;
      // past the ends every code is zero, and the last row's scale will do
      const float* pa[4];
      const float* pb[kC];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = m0 + lane + 32 * i;
        pa[i] = g.sa + (size_t)(r < g.M ? r : g.M - 1) * k_all + k_lo;
      }
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        const int n = kColScale ? n0 + lane + 32 * i : n0 + i * kCols;
        pb[i] = g.sb + (size_t)((n < g.N ? n : g.N - 1) / (kColScale ? 1 : g.b_rows)) * k_all + k_lo;
      }
      for (int kb = 0; kb < n_k && ok; kb += 4, ++q) {
        // four blocks' scales of a row: one load where the rows allow it (what
        // lies past this CTA's blocks is not used), else one each
        const auto load4 = [&](const float* row) {
          float4 v;
          if (vec) {
            v = *reinterpret_cast<const float4*>(row + kb);
          } else {
            v.x = row[kb];
            v.y = row[kb + 1 < n_k ? kb + 1 : n_k - 1];
            v.z = row[kb + 2 < n_k ? kb + 2 : n_k - 1];
            v.w = row[kb + 3 < n_k ? kb + 3 : n_k - 1];
          }
          return v;
        };
        float4 va[4], vb[kC];
#pragma unroll
        for (int i = 0; i < 4; ++i) va[i] = load4(pa[i]);
#pragma unroll
        for (int i = 0; i < kC; ++i) vb[i] = load4(pb[i]);
        const int slot = q % kF8Slots;
        float4 bias[kBN / 128];
        if (kb == 0 && g.bias) {
#pragma unroll
          for (int i = 0; i < kBN / 128; ++i) {
            const int n = n0 + 4 * (lane + 32 * i);
            bias[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (n < g.N) {
              const uint2 bv = *reinterpret_cast<const uint2*>(g.bias + n);
              const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&bv.x));
              const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&bv.y));
              bias[i] = make_float4(lo.x, lo.y, hi.x, hi.y);
            }
          }
        }
        ok = f8_wait(&S.sc_empty[slot], ((q / kF8Slots) & 1u) ^ 1u, &S.abort, limit);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (kb == 0 && g.bias) {
#pragma unroll
          for (int i = 0; i < kBN / 128; ++i) S.bias[tile % 4][lane + 32 * i] = bias[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (kColScale) {
            S.rs[slot][0][lane + 32 * i] = va[i];
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              S.rs[slot][h][lane + 32 * i] = make_float4(va[i].x * vb[h].x, va[i].y * vb[h].y,
                                                         va[i].z * vb[h].z, va[i].w * vb[h].w);
          }
        }
        if (kColScale) {
#pragma unroll
          for (int i = 0; i < kC; ++i) {
            S.cs[slot][0][lane + 32 * i] = vb[i].x;
            S.cs[slot][1][lane + 32 * i] = vb[i].y;
            S.cs[slot][2][lane + 32 * i] = vb[i].z;
            S.cs[slot][3][lane + 32 * i] = vb[i].w;
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&S.sc_full[slot]);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    tc::reg_inc<f8_regs_high(kBN, kColScale)>();
    const int sub = warp & 3;          // TMEM lanes 32 * sub .. 32 * sub + 31
    const int half = (warp - 4) >> 2;  // which half of the tile's columns
    const int et = (sub << 5) | lane;  // row in the tile
    uint8_t* stg = stage_out + (warp - 4) * (C::kOutBoxes * 4096);
    uint8_t* my_row = stg + lane * 128;
    const int swz = lane & 7;
    // where this warp's arrivals free a buffer
    uint32_t free_bar = tc::smem_u32(&S.acc_empty[0]);
    if (kPair == 2) free_bar = tc::cluster_map(free_bar, 0);
    const uint32_t lane_base = tmem + ((uint32_t)(sub * 32) << 16) + half * kCols;
    uint32_t q = 0, qs = 0, tile = 0;
    bool ok = true;
    for (int u = first_unit; u < n_units; u += unit_step, ++tile) {
      const int m0 = (u / n_n * kPair + rank) * kF8BM, c0 = (u % n_n) * kBN + half * kCols;
      // the totals start from the bias, which comes with the tile's first scales
      // (with kSplit it is added at the end, once)
      float acc[kCols];
      if (!kSplit && g.bias) {
        ok &= f8_wait(&S.sc_full[qs % kF8Slots], (qs / kF8Slots) & 1u, &S.abort, limit);
        const float4* bias = S.bias[tile % 4] + half * (kCols / 4);
#pragma unroll
        for (int e = 0; e < kCols; e += 4) {
          const float4 t = bias[e / 4];
          acc[e] = t.x; acc[e + 1] = t.y; acc[e + 2] = t.z; acc[e + 3] = t.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < kCols; ++e) acc[e] = 0.f;
      }
      for (int kb4 = 0; kb4 < n_k; kb4 += 4, ++qs) {
        const int slot = qs % kF8Slots;
        // after an abort every wait returns at once; the loop runs on to its
        // end (adding stale sums), since the warps share its barriers
        ok &= f8_wait(&S.sc_full[slot], (qs / kF8Slots) & 1u, &S.abort, limit);
        const float4 s4 = S.rs[slot][kColScale ? 0 : half][et];
        const float sj[4] = {s4.x, s4.y, s4.z, s4.w};
        // (unrolled twice, or not at all: four times costs registers)
#pragma unroll (kColScale || kBN == 128 ? 1 : 2)
        for (int j = 0; j < 4; ++j, ++q) {
          if (kb4 + j >= n_k) break;
          const int b = q % kBufs;
          const float s = j == 0 ? sj[0] : j == 1 ? sj[1] : j == 2 ? sj[2] : sj[3];
          const float* cs = S.cs[kColScale ? slot : 0][j] + (kColScale ? half * kCols : 0);
          ok &= f8_wait(&S.acc_full[b], (q / kBufs) & 1u, &S.abort, limit);
          tc::fence_after_sync();
          // kChunk columns are added while the next kChunk are read
          const uint32_t taddr = lane_base + b * kBN;
          float v[2][kChunk];
#pragma unroll
          for (int e = 0; e < kChunk; e += 16) tc::tmem_ld16(taddr + e, v[0] + e);
#pragma unroll
          for (int c = 0; c < kCols / kChunk; ++c) {
            tc::tmem_ld_wait();
            tc::tmem_pin<kChunk>(v[c & 1]);
            if (c + 1 < kCols / kChunk) {
#pragma unroll
              for (int e = 0; e < kChunk; e += 16)
                tc::tmem_ld16(taddr + (c + 1) * kChunk + e, v[(c + 1) & 1] + e);
            } else {  // the buffer is read: free it
              tc::fence_before_sync();
              __syncwarp();
              if (kPair == 2)
                tc::mbar_arrive_cluster(free_bar + 8 * b, lane == 0);
              else
                tc::mbar_arrive_if(free_bar + 8 * b, lane == 0);
            }
#pragma unroll
            for (int e = 0; e < kChunk; e += 4) {
              float4 k4 = make_float4(s, s, s, s);
              if (kColScale) {
                const float4 t = *reinterpret_cast<const float4*>(cs + c * kChunk + e);
                k4 = make_float4(s * t.x, s * t.y, s * t.z, s * t.w);
              }
              float* t = acc + c * kChunk + e;
              const float* x = v[c & 1] + e;
              const float2 lo = __ffma2_rn(make_float2(x[0], x[1]), make_float2(k4.x, k4.y),
                                           make_float2(t[0], t[1]));
              const float2 hi = __ffma2_rn(make_float2(x[2], x[3]), make_float2(k4.z, k4.w),
                                           make_float2(t[2], t[3]));
              t[0] = lo.x; t[1] = lo.y; t[2] = hi.x; t[3] = hi.y;
            }
          }
        }
        __syncwarp();
        tc::mbar_arrive_if(tc::smem_u32(&S.sc_empty[slot]), lane == 0);  // its scales are read
      }
      // where the warps share barriers below, they all go on or none does
      const bool bad = kSplit || (kEpi == kF8Quant && kCols == 64)
                           ? f8_any(!ok)
                           : !__all_sync(0xffffffffu, ok);
      if (bad && !kSplit) break;
      if (kSplit) {
        // Each CTA of the cluster adds up kCols / kParts columns of every
        // thread's totals, in the order of the parts; they travel through the
        // stages, which all of the tile's MMAs have left.
        constexpr int kW = kCols / kParts, kW4 = kW / 4;
        float4* const inbox = reinterpret_cast<float4*>(sm) + (tid - 128);  // [from][kW4][256]
        tc::cluster_sync();  // every CTA's MMAs are done (warps 0-3 take part below)
        if (!bad) {
#pragma unroll
          for (int to = 0; to < kParts; ++to) {
            const uint32_t at = tc::cluster_map(tc::smem_u32(inbox + part * (kW4 * 256)), to);
#pragma unroll
            for (int j = 0; j < kW4; ++j) tc::st_cluster(at + j * 4096, acc + to * kW + 4 * j);
          }
        }
        tc::cluster_sync();
        const int row = m0 + et, col = c0 + part * kW;
        if (!bad && row < g.M) {
#pragma unroll
          for (int j = 0; j < kW4; ++j) {
            const int c = col + 4 * j;
            if (c >= g.N) break;
            float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int from = 0; from < kParts; ++from) {
              const float4 x = inbox[(from * kW4 + j) * 256];
              o[0] += x.x; o[1] += x.y; o[2] += x.z; o[3] += x.w;
            }
            if (g.bias) {
              const float4 t = S.bias[0][half * (kCols / 4) + part * kW4 + j];
              o[0] += t.x; o[1] += t.y; o[2] += t.z; o[3] += t.w;
            }
            if (g.relu) {
#pragma unroll
              for (int i = 0; i < 4; ++i) o[i] = relu_nan(o[i]);
            }
            if (g.c_f32)
              *reinterpret_cast<float4*>(static_cast<float*>(g.C) + (size_t)row * g.N + c) =
                  make_float4(o[0], o[1], o[2], o[3]);
            else
              *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(g.C) + (size_t)row * g.N + c) =
                  make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
          }
        }
        break;  // a cluster has one tile
      }
      // The output leaves through the warp's staging rows by TMA, which clips
      // it to [M, N], while the next tile is under way: wait_staging() waits
      // for the last tile's, store_boxes() sends this one's.
      const auto wait_staging = [&] {
        if (lane == 0) tc::bulk_wait_read();
        __syncwarp();
      };
      const auto store_boxes = [&](int col, int step, int boxes) {
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          for (int i = 0; i < boxes; ++i)
            if (m0 + sub * 32 < g.M && col + i * step < g.N)
              tc::tma_store_2d(&map_c, col + i * step, m0 + sub * 32, tc::smem_u32(stg) + i * 4096);
          tc::bulk_commit();
        }
        __syncwarp();
      };
      if (kEpi == kF8Store && g.relu) {
#pragma unroll
        for (int e = 0; e < kCols; ++e) acc[e] = relu_nan(acc[e]);
      }
      if (kEpi == kF8Quant) {
        // (columns past N add nothing: they are sums of zeros, or NaN with the
        // rest of their block)
        // a block is the thread's 128 columns, or (kBN = 128) its 64 and those
        // of the other warpgroup's thread of the same row
        // max(0, .) costs nothing here: as signed integers the positive numbers
        // compare like numbers and the negative ones are below zero (a NaN that
        // arithmetic made is the largest), and the conversion has it built in
        int mi = 0;
#pragma unroll
        for (int e = 0; e < kCols; ++e) mi = max(mi, __float_as_int(acc[e]));
        uint32_t m = (uint32_t)mi;
        if (kCols == 64) {
          S.amax[half][et] = m;
          asm volatile("bar.sync 1, 256;" ::: "memory");
          m = max(m, S.amax[half ^ 1][et]);
          asm volatile("bar.sync 1, 256;" ::: "memory");
        }
        const float am = block_amax(m);
        const BlockScale sc = relu_scale(am);
        if (m0 + et < g.M && c0 < g.N && (c0 & 127) == 0)
          a.qs[(size_t)(m0 + et) * ((g.N + 127) >> 7) + (c0 >> 7)] = am / kE4m3Max;
        if (kCols == 128) wait_staging();
#pragma unroll
        for (int p = 0; p < kCols / 16; ++p) {
          const float* v = acc + 16 * p;
          const uint4 w = make_uint4(e4m3x4_relu(v, sc), e4m3x4_relu(v + 4, sc),
                                     e4m3x4_relu(v + 8, sc), e4m3x4_relu(v + 12, sc));
          if (kCols == 128)
            *reinterpret_cast<uint4*>(my_row + ((p ^ swz) << 4)) = w;
          else if (m0 + et < g.M && c0 + 16 * p < g.N)  // two whole sectors of the row
            *reinterpret_cast<uint4*>(a.Q + (size_t)(m0 + et) * g.N + c0 + 16 * p) = w;
        }
        if (kCols == 128) store_boxes(c0, 128, 1);
      } else if (!g.c_f32) {
        wait_staging();
#pragma unroll
        for (int p = 0; p < kCols / 8; ++p) {
          const float* v = acc + 8 * p;
          *reinterpret_cast<uint4*>(my_row + (p >> 3) * 4096 + (((p & 7) ^ swz) << 4)) =
              make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                         pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        }
        store_boxes(c0, 64, kCols / 64);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          wait_staging();
#pragma unroll
          for (int p = 0; p < kCols / 8; ++p) {
            const float* v = acc + h * (kCols / 2) + 4 * p;
            *reinterpret_cast<float4*>(my_row + (p >> 3) * 4096 + (((p & 7) ^ swz) << 4)) =
                make_float4(v[0], v[1], v[2], v[3]);
          }
          store_boxes(c0 + h * (kCols / 2), 32, kCols / 64);
        }
      }
    }
    if (lane == 0) tc::bulk_wait();
    __syncwarp();
  }
  if (kSplit && warp < 4) {  // the epilogue's two
    __syncwarp();
    tc::cluster_sync();
    tc::cluster_sync();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (kPair == 2) tc::cluster_sync();  // neither leaves while the other's threads may reach it
  if (warp == 0) {
    // Nor while a commit's arrival is on its way, which no barrier between
    // threads orders: the last one on each barrier, one to a lane (of a pair in
    // both CTAs, the commits being the even rank's).  A phase of a barrier
    // follows another only once that one was seen in this CTA.  After an abort
    // the epilogue waits for nothing and two may be on their way: then they get
    // time as well, far more than an arrival takes.
    if (*(volatile int*)&S.abort) f8_pause();
    uint64_t* bar = nullptr;
    uint32_t parity = 0;
    const auto wait_for_last = [&](uint64_t* bars, int n, int at) {
      const int last = f8_last_block(S.issued, n, at);
      if (last >= 0) bar = bars + at;
      parity = (uint32_t)(last / n) & 1u;
    };
    if (lane < kStages)
      wait_for_last(S.empty, kStages, lane);
    else if (lane < kStages + kBufs)
      wait_for_last(S.acc_full, kBufs, lane - kStages);
    else if (lane < kStages + kBufs + 2)
      bar = S.mma_done + (lane - kStages - kBufs);
    if (bar && !tc::mbar_wait(bar, parity)) record_status(tc::kErrTimeout);
  }
  if (warp == 1) {
    tc::fence_after_sync();
    if (kPair == 2)
      tc::tmem_dealloc_pair(tmem, 512);
    else
      tc::tmem_dealloc(tmem, 512);
  }
}

}  // namespace lsh
