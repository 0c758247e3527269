// Quantisation of a matrix into e4m3 blocks of 128 (fp8.cuh), and of its
// transpose.
//
//   quant_rows_kernel   blocks of 1 x 128: eight entries per thread, a block
//                       in 16 neighbouring lanes;
//   quant_tile_kernel   a tile of 128 x 128 entries per block of threads, read
//                       once: blocks of 128 x 128, and for either kind of
//                       block the transposed matrix, whose columns (the
//                       positions, the K axis of a weight-gradient product)
//                       become rows of bytes through shared memory.
// Both read the input once and write the codes; neither is bound by that alone.
// 16 000 x 2048 bf16 takes 23 us one way and 28 both in a graph of such calls
// (4.3 and 4.7 TB/s, two thirds of a copy's rate and more).  The first divides
// in 64 bits for its row and once a lane for a block's scale; the second issues
// in 73% of its slots.
#pragma once

#include "fp8.cuh"

namespace lsh {

struct QuantArgs {
  long long rows;
  int cols;           // multiple of 16
  const void* x;      // [rows, cols]
  uint8_t* y;         // [rows, cols] or NULL
  float* scales;      // [rows or row blocks, col blocks]
  uint8_t* yt;        // [cols, pitch_t] or NULL
  float* scales_t;    // [cols or col blocks, row blocks]
  long long pitch_t;  // rows rounded up to a multiple of 16; the rest is zero
  float* colsum;      // [row blocks, cols] sums of the tile's columns, or NULL
};

// Eight neighbouring entries of a row as loaded: bf16 pairs stay packed (half
// the registers, and magnitudes compare two at a time), fp32 as it is.
template <typename XT>
struct QuantPiece;
template <>
struct QuantPiece<__nv_bfloat16> {
  uint32_t w[4];
  static constexpr int kMags = 4;  // words of magnitudes, two columns each
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
  __device__ __forceinline__ float get(int e) const {
    return __uint_as_float((e & 1) ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
  }
  __device__ __forceinline__ uint32_t mag(int i) const { return w[i] & 0x7fff7fffu; }
  // the larger magnitudes of two words (a NaN is the largest)
  __device__ __forceinline__ static uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  // fp32 bits of a column's magnitude in its word
  __device__ __forceinline__ static uint32_t column(uint32_t m, int e) {
    return (e & 1) ? m & 0xffff0000u : m << 16;
  }
  __device__ __forceinline__ uint32_t amax() const {
    const uint32_t m = max2(max2(mag(0), mag(1)), max2(mag(2), mag(3)));
    return max(column(m, 0), column(m, 1));
  }
};
template <>
struct QuantPiece<float> {
  float v[8];
  static constexpr int kMags = 8;
  __device__ __forceinline__ void load(const float* p) { load8(p, v); }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
  }
  __device__ __forceinline__ float get(int e) const { return v[e]; }
  __device__ __forceinline__ uint32_t mag(int i) const { return mag_bits(v[i]); }
  __device__ __forceinline__ static uint32_t max2(uint32_t a, uint32_t b) { return max(a, b); }
  __device__ __forceinline__ static uint32_t column(uint32_t m, int) { return m; }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, mag(e));
    return m;
  }
};

// Pieces of 8 entries under way per thread.
template <typename XT>
constexpr int kQuantRowsPer = sizeof(XT) == 2 ? 4 : 2;

template <typename XT>
__global__ void __launch_bounds__(256) quant_rows_kernel(QuantArgs a) {
  constexpr bool kBf16 = sizeof(XT) == 2;
  constexpr int kPer = kQuantRowsPer<XT>;
  grid_dep_wait();
  grid_dep_launch();
  const int pieces = a.cols >> 3;
  const int padded = (pieces + 15) & ~15;  // a row starts at lane 0 or 16
  QuantPiece<XT> v[kPer];
  long long row[kPer];
  int p[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const long long g = ((long long)blockIdx.x * kPer + i) * 256 + threadIdx.x;
    row[i] = g / padded;
    p[i] = (int)(g - row[i] * padded);
    if (row[i] < a.rows && p[i] < pieces)
      v[i].load(static_cast<const XT*>(a.x) + (size_t)row[i] * a.cols + 8 * p[i]);
    else
      v[i].zero();
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    uint32_t m = v[i].amax();
#pragma unroll
    for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (row[i] >= a.rows || p[i] >= pieces) continue;
    const float am = block_amax(m);
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = v[i].get(e);
    *reinterpret_cast<uint2*>(a.y + (size_t)row[i] * a.cols + 8 * p[i]) =
        scale_to_e4m3<kBf16>(x, BlockScale(am));
    if ((p[i] & 15) == 0)
      a.scales[(size_t)row[i] * (padded >> 4) + (p[i] >> 4)] = am / kE4m3Max;
  }
}

// Magnitudes of 8 rows over 16 lanes, m[i] being the lane's own of row i: the
// largest of row (lane & 14) / 2, which the lane returns.  Each step hands half
// of the rows to the lane across, so 8 shuffles do for 8 rows.
__device__ __forceinline__ uint32_t rows_amax(uint32_t* m, int lane) {
#pragma unroll
  for (int h = 4; h; h >>= 1) {
    const bool up = lane & (2 * h);
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const uint32_t give = up ? m[i] : m[i + h], keep = up ? m[i + h] : m[i];
      m[i] = max(keep, __shfl_xor_sync(0xffffffffu, give, 2 * h));
    }
  }
  return max(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
}

// 256 threads; thread (rg, cg) = (tid / 16, tid % 16) holds rows 8 rg .. 8 rg
// + 7 and columns 8 cg .. 8 cg + 7 of the tile, so a row block (1 x 128) lies
// in 16 neighbouring lanes and a thread's part of the transposed tile is 8
// pieces of 8 consecutive bytes.
//
// The kernel is near the schedulers' limit as well as memory's, so the two
// divisions of a block (its scale and the scale's inverse) are one lane's,
// which hands the inverse on, and bf16 entries stay packed.
template <typename XT, bool kSquare>
__device__ __forceinline__ void quant_tile(const QuantArgs& a, unsigned block) {
  constexpr bool kBf16 = sizeof(XT) == 2;
  using Piece = QuantPiece<XT>;
  constexpr int kMags = Piece::kMags, kPerMag = 8 / kMags;
  __shared__ uint32_t cmax[8][128 / kPerMag];
  __shared__ float csum[8][128];
  __shared__ float cinv[128], clo[128];
  __shared__ __align__(16) uint8_t tile[128 * 128];
  grid_dep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rg = tid >> 4, cg = tid & 15;
  const int cb = (a.cols + 127) >> 7;
  const long long tr = block / cb;   // row block
  const int tc = (int)(block % cb);  // column block
  const long long row0 = tr * 128 + 8 * rg;
  const int col0 = tc * 128 + 8 * cg;
  Piece v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (row0 + i < a.rows && col0 < a.cols)
      v[i].load(static_cast<const XT*>(a.x) + (size_t)(row0 + i) * a.cols + col0);
    else
      v[i].zero();
  }
  grid_dep_launch();
  BlockScale sq(0.f, 0.f);
  if (kSquare) {  // one maximum for the whole tile
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, v[i].amax());
#pragma unroll
    for (int o = 16; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) cmax[warp][0] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, cmax[i][0]);
    const float am = block_amax(m);
    sq = BlockScale(am);
    if (tid == 0) {
      const long long rb = (a.rows + 127) >> 7;
      if (a.y) a.scales[tr * cb + tc] = am / kE4m3Max;
      if (a.yt) a.scales_t[tc * rb + tr] = am / kE4m3Max;
    }
  }
  if (a.y) {
    BlockScale mine(0.f, 0.f);  // of row (cg & 14) / 2
    if (!kSquare) {
      uint32_t m[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = v[i].amax();
      const float am = block_amax(rows_amax(m, lane));
      mine = BlockScale(am);
      const long long r = row0 + (cg >> 1);
      if (!(cg & 1) && r < a.rows) a.scales[(size_t)r * cb + tc] = am / kE4m3Max;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      BlockScale sc = sq;
      if (!kSquare) {
        const int from = (lane & 16) + 2 * i;
        sc.inv = __shfl_sync(0xffffffffu, mine.inv, from);
        if (!kBf16) sc.lo = __shfl_sync(0xffffffffu, mine.lo, from);
      }
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = v[i].get(e);
      if (row0 + i < a.rows && col0 < a.cols)
        *reinterpret_cast<uint2*>(a.y + (size_t)(row0 + i) * a.cols + col0) =
            scale_to_e4m3<kBf16>(x, sc);
    }
  }
  if (a.colsum) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i].get(e);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
      if ((tid & 16) == 0) csum[warp][8 * cg + e] = s;
    }
  }
  if (a.yt && !kSquare) {
#pragma unroll
    for (int e = 0; e < kMags; ++e) {
      uint32_t m = v[0].mag(e);
#pragma unroll
      for (int i = 1; i < 8; ++i) m = Piece::max2(m, v[i].mag(e));
      m = Piece::max2(m, __shfl_xor_sync(0xffffffffu, m, 16));
      if ((tid & 16) == 0) cmax[warp][kMags * cg + e] = m;
    }
  }
  if (a.colsum || (a.yt && !kSquare)) {
    __syncthreads();
    const int c = tc * 128 + (tid & 127);
    if (tid < 128) {
      if (a.yt && !kSquare) {
        uint32_t m = cmax[0][tid / kPerMag];
#pragma unroll
        for (int i = 1; i < 8; ++i) m = Piece::max2(m, cmax[i][tid / kPerMag]);
        const float am = block_amax(Piece::column(m, tid));
        const BlockScale sc(am);
        cinv[tid] = sc.inv;
        clo[tid] = sc.lo;
        if (c < a.cols) a.scales_t[(size_t)c * ((a.rows + 127) >> 7) + tr] = am / kE4m3Max;
      }
    } else if (a.colsum && c < a.cols) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += csum[i][tid & 127];
      a.colsum[(size_t)tr * a.cols + c] = s;
    }
    __syncthreads();
  }
  if (!a.yt) return;
  // row c of the transposed tile: 16 pieces of 8 bytes, in pairs of pieces, so
  // that a store's 16 lanes (one per column group) hit distinct banks
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = 8 * cg + e;
    const BlockScale sc = kSquare ? sq : BlockScale(cinv[c], clo[c]);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[i].get(e);
    *reinterpret_cast<uint2*>(tile + c * 128 + ((((rg >> 1) ^ (cg & 7)) << 4) | ((rg & 1) << 3))) =
        scale_to_e4m3<kBf16>(x, sc);
  }
  __syncthreads();
  // out: 8 lanes write a row's 128 bytes (pitch_t is a multiple of 16, so its
  // end never cuts a piece)
  const long long r = tr * 128 + 16 * (tid & 7);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = 32 * k + (tid >> 3);
    if (tc * 128 + c < a.cols && r < a.pitch_t)
      *reinterpret_cast<uint4*>(a.yt + (size_t)(tc * 128 + c) * a.pitch_t + r) =
          *reinterpret_cast<const uint4*>(tile + c * 128 + (((tid & 7) ^ ((c >> 3) & 7)) << 4));
  }
}

template <typename XT, bool kSquare>
__global__ void __launch_bounds__(256, sizeof(XT) == 2 ? 4 : 2) quant_tile_kernel(QuantArgs a) {
  quant_tile<XT, kSquare>(a, blockIdx.x);
}

// The tiles of two bf16 matrices, `na` of the first.
__global__ void __launch_bounds__(256, 4) quant_two_kernel(QuantArgs a, QuantArgs b, unsigned na) {
  if (blockIdx.x < na)
    quant_tile<__nv_bfloat16, false>(a, blockIdx.x);
  else
    quant_tile<__nv_bfloat16, false>(b, blockIdx.x - na);
}

}  // namespace lsh
