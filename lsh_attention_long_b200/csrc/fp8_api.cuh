// C ABI of the 8-bit feed-forward path: norm, quantiser, products and the
// feed-forward made of them.  Included at the end of lsh_api.cu, whose
// helpers (alignment, launches, tensor maps) it uses.
#pragma once

namespace {

bool any_misaligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (misaligned(p)) return true;
  return false;
}

bool is_f32_or_bf16(int32_t t) { return t == LSH_F32 || t == LSH_BF16; }

inline int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }
inline size_t kblocks(int cols) { return (size_t)((cols + 127) / 128); }
// columns of a transposed 8-bit matrix: its K axis, which a product takes in
// multiples of 16
inline size_t pitch16(int rows) { return ((size_t)rows + 15) & ~(size_t)15; }

// Sizes that a kernel rounds up to whole tiles and indexes with 32 bits.
constexpr int32_t kFp8MaxSize = 0x7fffffff - 255;

lsh_status norm_check(int32_t rows, int32_t cols) {
  if (rows < 0 || cols <= 0) return LSH_ERR_INVALID_ARG;
  if (cols % 16 || cols > lsh::kNormMaxCols) return LSH_ERR_UNSUPPORTED;
  return LSH_OK;
}

template <typename XT, int kOut, int kNV, int kT>
lsh_status norm_fwd_go(const lsh::NormArgs& a, cudaStream_t st) {
  constexpr int kBlock = lsh::norm_block(kT);
  return launch_pdl(lsh::rmsnorm_fwd_kernel<XT, kOut, kNV, kT>,
                    dim3((unsigned)ceil_div(a.rows, kBlock / kT)), dim3(kBlock), 0, st, a);
}
template <typename XT, int kOut>
lsh_status norm_fwd_launch(const lsh::NormArgs& a, cudaStream_t st) {
  if (a.cols <= 256) return norm_fwd_go<XT, kOut, 1, 32>(a, st);
  if (a.cols <= 512) return norm_fwd_go<XT, kOut, 2, 32>(a, st);
  if (a.cols <= 1024) return norm_fwd_go<XT, kOut, 4, 32>(a, st);
  if (a.cols <= 2048) return norm_fwd_go<XT, kOut, 1, 256>(a, st);
  if (a.cols <= 4096) return norm_fwd_go<XT, kOut, 2, 256>(a, st);
  if (a.cols <= 8192) return norm_fwd_go<XT, kOut, 2, 512>(a, st);
  return norm_fwd_go<XT, kOut, 2, 1024>(a, st);
}
template <typename XT>
lsh_status norm_fwd_launch(const lsh::NormArgs& a, int y_dtype, cudaStream_t st) {
  if (y_dtype == LSH_E4M3) return norm_fwd_launch<XT, lsh::kNormE4m3>(a, st);
  if (y_dtype == LSH_BF16) return norm_fwd_launch<XT, lsh::kNormBf16>(a, st);
  return norm_fwd_launch<XT, lsh::kNormF32>(a, st);
}

// Most blocks of the backward, each of which leaves one partial row of dw.
int norm_bwd_most(int32_t rows, int32_t cols) {
  const int n = ceil_div(rows, cols <= lsh::kNormWarpCols ? 8 : 1);
  return n < 592 ? n : 592;
}

// The blocks loop over rows: as many as the SMs hold at once (a few more would
// run alone at the end).
template <typename XT, int kNV, int kT>
lsh_status norm_bwd_go(const lsh::NormBwdArgs& a, int* blocks, cudaStream_t st) {
  const auto kernel = lsh::rmsnorm_bwd_kernel<XT, kNV, kT>;
  static const int per_sm = [&] {
    int n = 0;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, lsh::norm_block(kT), 0) ==
                       cudaSuccess && n > 0
               ? n
               : 1;
  }();
  const int fit = per_sm * num_sms();
  *blocks = *blocks < fit ? *blocks : fit;
  return launch_pdl(kernel, dim3((unsigned)*blocks), dim3(lsh::norm_block(kT)), 0, st, a);
}
template <typename XT>
lsh_status norm_bwd_launch(const lsh::NormBwdArgs& a, int* blocks, cudaStream_t st) {
  if (a.cols <= 256) return norm_bwd_go<XT, 1, 32>(a, blocks, st);
  if (a.cols <= 512) return norm_bwd_go<XT, 2, 32>(a, blocks, st);
  if (a.cols <= 1024) return norm_bwd_go<XT, 4, 32>(a, blocks, st);
  if (a.cols <= 2048) return norm_bwd_go<XT, 1, 256>(a, blocks, st);
  if (a.cols <= 4096) return norm_bwd_go<XT, 1, 512>(a, blocks, st);
  if (a.cols <= 8192) return norm_bwd_go<XT, 1, 1024>(a, blocks, st);
  return norm_bwd_go<XT, 2, 1024>(a, blocks, st);
}

lsh_status column_sum(const float* part, int blocks, int cols, float* out, cudaStream_t st) {
  return launch_pdl(lsh::column_sum_kernel, dim3((unsigned)ceil_div(cols, 32)), dim3(1024), 0, st,
                    part, blocks, cols, out);
}

template <typename XT>
lsh_status quant_launch(const lsh::QuantArgs& a, int block_rows, cudaStream_t st) {
  if (block_rows == 1 && !a.yt && !a.colsum) {
    const long long padded = ((a.cols >> 3) + 15) & ~15;
    constexpr int kPer = 256 * lsh::kQuantRowsPer<XT>;
    const long long grid = (a.rows * padded + kPer - 1) / kPer;
    if (grid > 0x7fffffffLL) return LSH_ERR_UNSUPPORTED;
    return launch_pdl(lsh::quant_rows_kernel<XT>, dim3((unsigned)grid), dim3(256), 0, st, a);
  }
  const long long grid = ((a.rows + 127) / 128) * (long long)kblocks(a.cols);
  if (grid > 0x7fffffffLL) return LSH_ERR_UNSUPPORTED;
  return launch_pdl(block_rows == 1 ? lsh::quant_tile_kernel<XT, false>
                                    : lsh::quant_tile_kernel<XT, true>,
                    dim3((unsigned)grid), dim3(256), 0, st, a);
}

// Two matrices in 1 x 128 blocks (both ways, or transposed alone), one launch.
lsh_status quant_two_launch(const lsh::QuantArgs& a, const lsh::QuantArgs& b, cudaStream_t st) {
  const long long na = ((a.rows + 127) / 128) * (long long)kblocks(a.cols);
  const long long nb = ((b.rows + 127) / 128) * (long long)kblocks(b.cols);
  if (na + nb > 0x7fffffffLL) return LSH_ERR_UNSUPPORTED;
  return launch_pdl(lsh::quant_two_kernel, dim3((unsigned)(na + nb)), dim3(256), 0, st, a, b,
                    (unsigned)na);
}

lsh::QuantArgs quant_args(int32_t rows, int32_t cols, const void* X, void* Y, float* scales,
                          void* Yt, float* scales_t) {
  lsh::QuantArgs a = {};
  a.rows = rows; a.cols = cols; a.x = X;
  a.y = static_cast<uint8_t*>(Y); a.scales = scales;
  a.yt = static_cast<uint8_t*>(Yt); a.scales_t = scales_t;
  a.pitch_t = (long long)pitch16(rows);
  return a;
}

lsh_status fp8_sizes_check(int32_t M, int32_t N, int32_t K) {
  if (M < 0 || N <= 0 || K <= 0) return LSH_ERR_INVALID_ARG;
  if (N % 16 || K % 16 || M > kFp8MaxSize || N > kFp8MaxSize || K > kFp8MaxSize)
    return LSH_ERR_UNSUPPORTED;
  return LSH_OK;
}

// Row-major matrix [rows, cols] read or written in boxes of 128 bytes x
// box_rows rows, 128-byte swizzled; zeros past the ends.
bool map_128b(CUtensorMap* m, CUtensorMapDataType type, uint32_t size, const void* base,
              uint64_t rows, uint64_t cols, uint32_t box_rows) {
  const EncodeTiled f = encode_tiled();
  if (!f) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols * size};
  const cuuint32_t box[2] = {128 / size, box_rows};
  const cuuint32_t elem[2] = {1, 1};
  return f(m, type, 2, const_cast<void*>(base), dims, strides, box, elem,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool u8_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  return map_128b(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, base, rows, cols, box_rows);
}

template <int kPair, int kBN, int kEpi, bool kColScale, int kParts>
lsh_status fp8_tc_launch(const lsh::Fp8TcArgs& a, cudaStream_t st) {
  const lsh::Fp8GemmArgs& g = a.g;
  CUtensorMap ma, mb, mc;
  if (!u8_map(&ma, g.A, (uint64_t)g.M, (uint64_t)g.K, lsh::kF8BM) ||
      !u8_map(&mb, g.B, (uint64_t)g.N, (uint64_t)g.K, kBN / kPair))
    return LSH_ERR_CUDA;
  const uint64_t M = (uint64_t)g.M, N = (uint64_t)g.N;
  if (!(kEpi == lsh::kF8Quant ? u8_map(&mc, a.Q, M, N, 32)
        : g.c_f32 ? map_128b(&mc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, g.C, M, N, 32)
                  : map_128b(&mc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, g.C, M, N, 32)))
    return LSH_ERR_CUDA;
  constexpr size_t smem = lsh::fp8_tc_smem_bytes<kPair, kBN, kEpi, kColScale>();
  const auto kernel = lsh::gemm_fp8_tc_kernel<kPair, kBN, kEpi, kColScale, kParts>;
  // the kernel's register split adds up only if it was built with kF8Regs, which
  // a compiler other than the one it was written with might not give it
  static const bool regs_ok = [&] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, kernel) == cudaSuccess && at.numRegs == lsh::kF8Regs;
  }();
  if (!regs_ok) return LSH_ERR_CUDA;
  const lsh_status s = allow_smem(kernel, smem);
  if (s != LSH_OK) return s;
  const long long units = (long long)ceil_div(g.M, kPair * lsh::kF8BM) * ceil_div(g.N, kBN);
  if (units > 0x3fffffff) return LSH_ERR_UNSUPPORTED;
  const int fit = num_sms() / kPair;
  const int clusters = kParts > 1 || units < fit ? (int)units : fit;
  return launch_pdl_cluster(kernel, dim3((unsigned)(clusters * kPair * kParts)),
                            dim3(lsh::kF8Threads), smem, st, kPair * kParts, ma, mb, mc, a);
}

template <int kNT, int kW, int kEpi>
lsh_status fp8_skinny_launch(const lsh::Fp8SkinnyArgs& a, cudaStream_t st) {
  // a cluster covers 128 rows of B, one block of the 8-bit result
  constexpr int kCluster = kEpi == lsh::kF8Quant ? 128 / lsh::kSkRows : 1;
  const int grid = ceil_div(ceil_div(a.g.N, lsh::kSkRows), kCluster) * kCluster;
  const auto kernel = lsh::gemm_fp8_skinny_kernel<kNT, kW, kEpi>;
  constexpr size_t smem = lsh::sk_smem_bytes(kW);
  const lsh_status s = allow_smem(kernel, smem);
  if (s != LSH_OK) return s;
  return launch_pdl_cluster(kernel, dim3((unsigned)grid), dim3(32 * kW), smem, st, kCluster, a);
}
// Warps per block of 16 rows: eight, which are through K soonest, while blocks
// are few; fewer where several blocks share an SM, so that the last ones to
// start leave less idle (one row, 16 384 x 8192: 28 us with two, 32 with four;
// 8192 x 2048: 6.2 with four, 6.5 with eight).
template <int kNT, int kEpi>
lsh_status fp8_skinny_launch(const lsh::Fp8SkinnyArgs& a, cudaStream_t st) {
  const int per_sm = ceil_div(a.g.N, lsh::kSkRows) / num_sms();
  if (per_sm >= 4) return fp8_skinny_launch<kNT, 2, kEpi>(a, st);
  if (per_sm >= 2) return fp8_skinny_launch<kNT, 4, kEpi>(a, st);
  return fp8_skinny_launch<kNT, 8, kEpi>(a, st);
}
template <int kEpi>
lsh_status fp8_skinny_launch(const lsh::Fp8GemmArgs& g, void* Q, float* qs, cudaStream_t st,
                             int prefetch_b = 0) {
  lsh::Fp8SkinnyArgs a = {};
  a.g = g;
  a.Q = static_cast<uint8_t*>(Q);
  a.qs = qs;
  a.prefetch_b = prefetch_b;
  return g.M <= 8 ? fp8_skinny_launch<1, kEpi>(a, st) : fp8_skinny_launch<2, kEpi>(a, st);
}

// Whether 256 x 256 tiles, on a pair of CTAs each, are enough to occupy half of
// the SMs: they need half the loads per product of 128 x 128 tiles.
bool fp8_pair_tiles(const lsh::Fp8GemmArgs& g) {
  return 4LL * ceil_div(g.M, 256) * ceil_div(g.N, 256) >= num_sms();
}

// CTAs that share a 128 x 128 tile's K, as many as all get an SM at the same
// time (15 clusters of 8 or 33 of 4 fit on a B200).  Meeting at the end costs
// some 2 us, so K has to be long: 64 x 4096 x 4096 takes 9.6 us with four and
// 13.1 with one, 64 x 2048 x 1024 6.0 and 5.2, 1000 x 512 x 2048 8.1 and 7.5.
int fp8_split(const lsh::Fp8GemmArgs& g) {
  const long long tiles = (long long)ceil_div(g.M, 128) * ceil_div(g.N, 128);
  const int k = ceil_div(g.K, 128);
  if (tiles <= 15 && k >= 16) return 8;
  if (tiles <= 33 && k >= 24) return 4;
  if (tiles * 2 <= num_sms() && k >= 32) return 2;
  return 1;
}

template <bool kColScale>
lsh_status fp8_tc_gemm(const lsh::Fp8TcArgs& a, cudaStream_t st) {
  if (fp8_pair_tiles(a.g)) return fp8_tc_launch<2, 256, lsh::kF8Store, kColScale, 1>(a, st);
  const int parts = fp8_split(a.g);
  if (parts == 8) return fp8_tc_launch<1, 128, lsh::kF8Store, kColScale, 8>(a, st);
  if (parts == 4) return fp8_tc_launch<1, 128, lsh::kF8Store, kColScale, 4>(a, st);
  if (parts == 2) return fp8_tc_launch<1, 128, lsh::kF8Store, kColScale, 2>(a, st);
  return fp8_tc_launch<1, 128, lsh::kF8Store, kColScale, 1>(a, st);
}

bool fp8_few_rows(const lsh::Fp8GemmArgs& g) { return g.M <= lsh::kSkMaxM; }

// prefetch_b: see Fp8SkinnyArgs.
lsh_status fp8_gemm_launch(const lsh::Fp8GemmArgs& g, cudaStream_t st, int prefetch_b = 0) {
  if (fp8_few_rows(g)) return fp8_skinny_launch<lsh::kF8Store>(g, nullptr, nullptr, st, prefetch_b);
  lsh::Fp8TcArgs a = {};
  a.g = g;
  a.wait_limit = g_wait_limit;
  a.hold_tile = g_hold_tile;
  return g.b_rows == 1 ? fp8_tc_gemm<true>(a, st) : fp8_tc_gemm<false>(a, st);
}

// The hidden activation of the feed-forward: max(0, A B^T + bias) in 8 bits.
lsh_status fp8_gemm_quant_launch(const lsh::Fp8GemmArgs& g, void* Q, float* qs,
                                 cudaStream_t st) {
  if (fp8_few_rows(g)) return fp8_skinny_launch<lsh::kF8Quant>(g, Q, qs, st);
  lsh::Fp8TcArgs a = {};
  a.g = g;
  a.Q = static_cast<uint8_t*>(Q);
  a.qs = qs;
  a.wait_limit = g_wait_limit;
  a.hold_tile = g_hold_tile;
  return fp8_pair_tiles(g) ? fp8_tc_launch<2, 256, lsh::kF8Quant, false, 1>(a, st)
                           : fp8_tc_launch<1, 128, lsh::kF8Quant, false, 1>(a, st);
}

lsh::Fp8GemmArgs fp8_gemm_args(int M, int N, int K, const void* A, const float* sa, const void* B,
                               const float* sb, int b_rows) {
  lsh::Fp8GemmArgs g = {};
  g.M = M; g.N = N; g.K = K;
  g.A = static_cast<const uint8_t*>(A); g.sa = sa;
  g.B = static_cast<const uint8_t*>(B); g.sb = sb;
  g.b_rows = b_rows;
  return g;
}

// Workspace of lsh_matmul_fp8_backward: dC in 8 bits both ways, A transposed,
// and the column sums of dC's row blocks.
struct Fp8BwdLayout {
  size_t dc, dc_s, dct, dct_s, at, at_s, sums, total;
};
Fp8BwdLayout fp8_bwd_layout(int32_t M, int32_t N, int32_t K) {
  Fp8BwdLayout l;
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t at = off; off += align_up(bytes); return at; };
  const size_t rb = kblocks(M);
  l.dc = take((size_t)M * N);
  l.dc_s = take((size_t)M * kblocks(N) * sizeof(float));
  l.dct = take((size_t)N * pitch16(M));
  l.dct_s = take((size_t)N * rb * sizeof(float));
  l.at = take((size_t)K * pitch16(M));
  l.at_s = take((size_t)K * rb * sizeof(float));
  l.sums = take(rb * (size_t)N * sizeof(float));
  l.total = off;
  return l;
}

// Positions that lsh_ffn_forward_fp8 takes at a time: `chunk`, or more where their
// hidden activation stays within kFfn8Hidden bytes (two chunks' then take half
// of the L2, and every product is a launch: 65 536 positions, 512 -> 2048 ->
// 512, took 227 us by 8192 and 202 by 16 384, 199 now), in parts of nearly equal
// size.
constexpr size_t kFfn8Hidden = (size_t)32 << 20;
int64_t ffn8_step(int32_t tokens, int32_t d_ff, int32_t chunk) {
  const int64_t fit = (int64_t)(kFfn8Hidden / (size_t)d_ff) / 256 * 256;
  int64_t step = chunk > fit ? chunk : fit;
  if (step >= tokens) return tokens;
  const int64_t n = (tokens + step - 1) / step;
  const int64_t even = ((tokens + n - 1) / n + 255) / 256 * 256;
  return even < step ? even : step;
}

// Workspace of lsh_ffn_forward_fp8: the hidden activation of two steps, which
// the steps use in turn (of one, where there is no more).
struct Ffn8Layout {
  size_t h8[2], s[2], total;
};
Ffn8Layout ffn8_layout(int32_t tokens, int32_t d_ff, int32_t chunk) {
  Ffn8Layout l;
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t at = off; off += align_up(bytes); return at; };
  const int64_t rows = ffn8_step(tokens, d_ff, chunk);
  for (int i = 0; i < 2; ++i) {
    if (i && tokens <= rows) {
      l.h8[1] = l.h8[0];
      l.s[1] = l.s[0];
      break;
    }
    l.h8[i] = take((size_t)rows * d_ff);
    l.s[i] = take((size_t)rows * kblocks(d_ff) * sizeof(float));
  }
  l.total = off;
  return l;
}

lsh_status ffn8_check(int32_t tokens, int32_t d_model, int32_t d_ff, int32_t chunk) {
  if (tokens < 0 || d_model <= 0 || d_ff <= 0 || chunk <= 0) return LSH_ERR_INVALID_ARG;
  if (d_model % 16 || d_ff % 16 || chunk % 128 || tokens > kFp8MaxSize ||
      d_model > kFp8MaxSize || d_ff > kFp8MaxSize)
    return LSH_ERR_UNSUPPORTED;
  return LSH_OK;
}

}  // namespace

extern "C" {

lsh_status lsh_rmsnorm_forward(int32_t rows, int32_t cols, int32_t x_dtype, int32_t r_dtype,
                               int32_t w_dtype, int32_t y_dtype, const void* X, const void* R,
                               const void* w, float eps, void* H, void* Y, float* scales,
                               float* rstd, void* stream) {
  if (!is_f32_or_bf16(x_dtype) || !is_f32_or_bf16(w_dtype) ||
      !(is_f32_or_bf16(y_dtype) || y_dtype == LSH_E4M3) || !(eps > 0.f && eps < 1e30f))
    return LSH_ERR_INVALID_ARG;
  if (R && !(r_dtype == LSH_BF16 || r_dtype == x_dtype)) return LSH_ERR_INVALID_ARG;
  const lsh_status s = norm_check(rows, cols);
  if (s != LSH_OK) return s;
  if (rows == 0) return LSH_OK;
  if (!X || !w || !Y || (R && !H) || (!R && H) || (y_dtype == LSH_E4M3 && !scales))
    return LSH_ERR_INVALID_ARG;
  if (any_misaligned({X, R, w, H, Y, scales, rstd})) return LSH_ERR_INVALID_ARG;
  lsh::NormArgs a = {};
  a.rows = rows; a.cols = cols;
  a.r_bf16 = r_dtype == LSH_BF16; a.w_bf16 = w_dtype == LSH_BF16;
  a.x = X; a.r = R; a.w = w; a.eps = eps;
  a.h = H; a.y = Y; a.scales = scales; a.rstd = rstd;
  return x_dtype == LSH_BF16 ? norm_fwd_launch<__nv_bfloat16>(a, y_dtype, as_stream(stream))
                             : norm_fwd_launch<float>(a, y_dtype, as_stream(stream));
}

size_t lsh_rmsnorm_bwd_ws_size(int32_t rows, int32_t cols) {
  if (norm_check(rows, cols) != LSH_OK || rows == 0) return 0;
  const int blocks = norm_bwd_most(rows, cols);
  return blocks > 1 ? align_up((size_t)blocks * cols * sizeof(float)) : 0;
}

lsh_status lsh_rmsnorm_backward(int32_t rows, int32_t cols, int32_t x_dtype, int32_t dy_dtype,
                                int32_t w_dtype, const void* dY, const void* H, const void* w,
                                const float* rstd, const void* dH, void* dX, float* dw, void* ws,
                                size_t ws_bytes, void* stream) {
  if (!is_f32_or_bf16(x_dtype) || !is_f32_or_bf16(dy_dtype) || !is_f32_or_bf16(w_dtype))
    return LSH_ERR_INVALID_ARG;
  lsh_status s = norm_check(rows, cols);
  if (s != LSH_OK) return s;
  if (!dw || misaligned(dw)) return LSH_ERR_INVALID_ARG;
  cudaStream_t st = as_stream(stream);
  if (rows == 0)  // a sum of no rows
    return cudaMemsetAsync(dw, 0, (size_t)cols * sizeof(float), st) == cudaSuccess ? LSH_OK
                                                                                   : LSH_ERR_CUDA;
  if (!dY || !H || !w || !rstd || !dX) return LSH_ERR_INVALID_ARG;
  if (any_misaligned({dY, H, w, rstd, dH, dX, ws})) return LSH_ERR_INVALID_ARG;
  const size_t need = lsh_rmsnorm_bwd_ws_size(rows, cols);
  if (need && (!ws || ws_bytes < need)) return LSH_ERR_WORKSPACE;
  lsh::NormBwdArgs a = {};
  a.rows = rows; a.cols = cols;
  a.dy_bf16 = dy_dtype == LSH_BF16; a.w_bf16 = w_dtype == LSH_BF16;
  a.dy = dY; a.h = H; a.w = w; a.rstd = rstd; a.dh = dH; a.dx = dX;
  a.dw = need ? static_cast<float*>(ws) : dw;
  int blocks = norm_bwd_most(rows, cols);
  s = x_dtype == LSH_BF16 ? norm_bwd_launch<__nv_bfloat16>(a, &blocks, st)
                          : norm_bwd_launch<float>(a, &blocks, st);
  if (s != LSH_OK || !need) return s;
  return column_sum(a.dw, blocks, cols, dw, st);
}

lsh_status lsh_quantize_fp8(int32_t rows, int32_t cols, int32_t x_dtype, int32_t block_rows,
                            const void* X, void* Y, float* scales, void* Yt, float* scales_t,
                            void* stream) {
  if (!is_f32_or_bf16(x_dtype) || rows < 0 || cols <= 0 || (block_rows != 1 && block_rows != 128))
    return LSH_ERR_INVALID_ARG;
  if (cols % 16 || cols > kFp8MaxSize) return LSH_ERR_UNSUPPORTED;
  if (rows == 0) return LSH_OK;
  if (!X || (!Y && !Yt) || (Y && !scales) || (Yt && !scales_t)) return LSH_ERR_INVALID_ARG;
  if (any_misaligned({X, Y, scales, Yt, scales_t})) return LSH_ERR_INVALID_ARG;
  const lsh::QuantArgs a = quant_args(rows, cols, X, Y, scales, Yt, scales_t);
  return x_dtype == LSH_BF16 ? quant_launch<__nv_bfloat16>(a, block_rows, as_stream(stream))
                             : quant_launch<float>(a, block_rows, as_stream(stream));
}

lsh_status lsh_matmul_fp8(int32_t M, int32_t N, int32_t K, const void* A, const float* a_scales,
                          const void* B, const float* b_scales, int32_t b_block_rows,
                          const void* bias, int32_t relu, int32_t c_dtype, void* C,
                          void* stream) {
  if (!is_f32_or_bf16(c_dtype) || (b_block_rows != 1 && b_block_rows != 128))
    return LSH_ERR_INVALID_ARG;
  const lsh_status s = fp8_sizes_check(M, N, K);
  if (s != LSH_OK) return s;
  if (M == 0) return LSH_OK;
  if (!A || !a_scales || !B || !b_scales || !C) return LSH_ERR_INVALID_ARG;
  if (any_misaligned({A, a_scales, B, b_scales, bias, C})) return LSH_ERR_INVALID_ARG;
  lsh::Fp8GemmArgs g = fp8_gemm_args(M, N, K, A, a_scales, B, b_scales, b_block_rows);
  g.bias = static_cast<const __nv_bfloat16*>(bias);
  g.relu = relu ? 1 : 0;
  g.C = C;
  g.c_f32 = c_dtype == LSH_F32;
  return fp8_gemm_launch(g, as_stream(stream));
}

size_t lsh_matmul_fp8_bwd_ws_size(int32_t M, int32_t N, int32_t K) {
  if (fp8_sizes_check(M, N, K) != LSH_OK || M == 0) return 0;
  return fp8_bwd_layout(M, N, K).total;
}

lsh_status lsh_matmul_fp8_backward(int32_t M, int32_t N, int32_t K, const void* dC, const void* A,
                                   const void* Bt, const float* bt_scales, int32_t da_dtype,
                                   void* dA, float* dB, float* db, void* ws, size_t ws_bytes,
                                   void* stream) {
  if (!is_f32_or_bf16(da_dtype)) return LSH_ERR_INVALID_ARG;
  lsh_status s = fp8_sizes_check(M, N, K);
  if (s != LSH_OK) return s;
  if (any_misaligned({dC, A, Bt, bt_scales, dA, dB, db, ws})) return LSH_ERR_INVALID_ARG;
  cudaStream_t st = as_stream(stream);
  if (M == 0) {  // sums of no rows
    if ((dB && cudaMemsetAsync(dB, 0, (size_t)N * K * sizeof(float), st) != cudaSuccess) ||
        (db && cudaMemsetAsync(db, 0, (size_t)N * sizeof(float), st) != cudaSuccess))
      return LSH_ERR_CUDA;
    return LSH_OK;
  }
  if (!dC || (!dA && !dB && !db) || (dA && (!Bt || !bt_scales)) || (dB && !A))
    return LSH_ERR_INVALID_ARG;
  const Fp8BwdLayout l = fp8_bwd_layout(M, N, K);
  if (!ws || ws_bytes < l.total) return LSH_ERR_WORKSPACE;
  char* w = static_cast<char*>(ws);
  auto f = [&](size_t at) { return reinterpret_cast<float*>(w + at); };
  lsh::QuantArgs q = quant_args(M, N, dC, dA ? w + l.dc : nullptr, f(l.dc_s),
                                dB ? w + l.dct : nullptr, f(l.dct_s));
  // one block of 128 rows: its column sums are db
  const bool one = kblocks(M) == 1;
  q.colsum = !db ? nullptr : one ? db : f(l.sums);
  // only what is asked for is put into 8 bits; db alone still reads dC once
  if (dB)
    s = quant_two_launch(q, quant_args(M, K, A, nullptr, nullptr, w + l.at, f(l.at_s)), st);
  else
    s = quant_launch<__nv_bfloat16>(q, 1, st);
  if (s != LSH_OK) return s;
  if (db && !one && (s = column_sum(f(l.sums), (int)kblocks(M), N, db, st)) != LSH_OK) return s;
  if (dA) {
    lsh::Fp8GemmArgs g = fp8_gemm_args(M, K, N, w + l.dc, f(l.dc_s), Bt, bt_scales, 128);
    g.C = dA;
    g.c_f32 = da_dtype == LSH_F32;
    if ((s = fp8_gemm_launch(g, st)) != LSH_OK) return s;
  }
  if (dB) {
    lsh::Fp8GemmArgs g = fp8_gemm_args(N, K, (int)pitch16(M), w + l.dct, f(l.dct_s), w + l.at,
                                       f(l.at_s), 1);
    g.C = dB;
    g.c_f32 = 1;
    if ((s = fp8_gemm_launch(g, st)) != LSH_OK) return s;
  }
  return LSH_OK;
}

size_t lsh_ffn_fp8_ws_size(int32_t tokens, int32_t d_model, int32_t d_ff, int32_t chunk) {
  if (ffn8_check(tokens, d_model, d_ff, chunk) != LSH_OK || tokens == 0) return 0;
  return ffn8_layout(tokens, d_ff, chunk).total;
}

lsh_status lsh_ffn_forward_fp8(int32_t tokens, int32_t d_model, int32_t d_ff, int32_t chunk,
                               const void* X, const float* x_scales, const void* W1,
                               const float* w1_scales, const void* b1, const void* W2,
                               const float* w2_scales, const void* b2, void* Y, void* ws,
                               size_t ws_bytes, void* stream) {
  lsh_status s = ffn8_check(tokens, d_model, d_ff, chunk);
  if (s != LSH_OK) return s;
  if (tokens == 0) return LSH_OK;
  if (!X || !x_scales || !W1 || !w1_scales || !b1 || !W2 || !w2_scales || !b2 || !Y)
    return LSH_ERR_INVALID_ARG;
  if (any_misaligned({X, x_scales, W1, w1_scales, b1, W2, w2_scales, b2, Y, ws}))
    return LSH_ERR_INVALID_ARG;
  const Ffn8Layout l = ffn8_layout(tokens, d_ff, chunk);
  if (!ws || ws_bytes < l.total) return LSH_ERR_WORKSPACE;
  cudaStream_t st = as_stream(stream);
  char* w = static_cast<char*>(ws);
  const int64_t step = ffn8_step(tokens, d_ff, chunk);
  const int64_t n_chunks = (tokens + step - 1) / step;
  const auto rows_of = [&](int64_t c) {
    return (int)(tokens - c * step < step ? tokens - c * step : step);
  };
  const auto hidden = [&](int64_t c) { return w + l.h8[c & 1]; };
  const auto hidden_s = [&](int64_t c) { return reinterpret_cast<float*>(w + l.s[c & 1]); };
  // up(c) makes chunk c's hidden activation, down(c) its output.  Each waits for
  // the launch before it ahead of every load: a grid sees what another wrote
  // only by a wait of its own, however the two are known to follow each other.
  const auto up = [&](int64_t c) {
    const int64_t c0 = c * step;
    lsh::Fp8GemmArgs g = fp8_gemm_args(rows_of(c), d_ff, d_model,
                                       static_cast<const uint8_t*>(X) + c0 * d_model,
                                       x_scales + c0 * kblocks(d_model), W1, w1_scales, 128);
    g.bias = static_cast<const __nv_bfloat16*>(b1);
    g.relu = 1;
    return fp8_gemm_quant_launch(g, hidden(c), hidden_s(c), st);
  };
  const auto down = [&](int64_t c) {
    lsh::Fp8GemmArgs g = fp8_gemm_args(rows_of(c), d_model, d_ff, hidden(c), hidden_s(c), W2,
                                       w2_scales, 128);
    g.bias = static_cast<const __nv_bfloat16*>(b2);
    g.C = static_cast<__nv_bfloat16*>(Y) + c * step * d_model;
    return fp8_gemm_launch(g, st, 1);
  };
  for (int64_t c = 0; c < n_chunks; ++c)
    if ((s = up(c)) != LSH_OK || (s = down(c)) != LSH_OK) return s;
  return LSH_OK;
}

}  // extern "C"
