// 8-bit activation checkpoints for gfx950: a bf16 or fp32 matrix of any size stored as E4M3 codes
// with one fp32 scale per 128 columns of a row, read back, and requantised along its rows for the
// weight-gradient GEMM.
//
// For a group x_1..x_128 with amax = max |x_i| over its finite elements: s = amax/448,
// r = 448/amax, q_i = E4M3(x_i r), and what the checkpoint stands for is value(q_i) s. For sizes
// that are multiples of 128 the bytes are those of the 1x128 quantiser, so an FP8 GEMM operand
// kept from the forward pass is a checkpoint, and a checkpoint is an operand.
//
// All of it is bound by HBM: 3 B per element (bf16) or 5 B (fp32) packed or unpacked, 2 B
// requantised, and 4 B of scale per group.
#include "coltile.hpp"

namespace puro {
namespace {

// ------------------------------------------------------------------ row groups
// Tiles as RowTile lays them out. Lane k of a 16-lane row stores the scale of the row's k-th pass.
constexpr int kPasses = RowTile::kPasses;

template <typename T, bool kShort>
__global__ __launch_bounds__(256) void ckpt_pack_kernel(const T* __restrict__ x, int64_t rows,
                                                        int64_t cols, int64_t ldx, int pow2,
                                                        uint8_t* __restrict__ q,
                                                        float* __restrict__ s) {
  const RowTile t(cols, off_lines(cols));
  const int l16 = threadIdx.x & 15;
  const int64_t c = t.chunk;
  const Span<kShort> sp(t.col, cols, cols % (128 * RowTile::kChunks) != 0);
  typename RawOf<T>::type raw[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p)  // rows past the end read the last one again
    load<true, kShort>(raw[p], x + min(t.row(p), rows - 1) * ldx, sp);
  F8 v[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) values(raw[p], sp, v[p].f);
  const RowGroups<kPasses> g = row_groups<true, kPasses>(&v[0].f, pow2 != 0);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t row = t.row(p);
    if (row < rows) store8<true>(q + row * cols + t.col, sp.n, encode8(v[p].f, g.r[p]));
  }
  if (l16 < kPasses && c * 128 < cols && t.row(l16) < rows) s[c * rows + t.row(l16)] = g.s;
}

template <typename T, bool kShort>
__global__ __launch_bounds__(256) void ckpt_unpack_kernel(const uint8_t* __restrict__ q,
                                                          const float* __restrict__ s,
                                                          int64_t rows, int64_t cols, int64_t ldx,
                                                          T* __restrict__ x) {
  const RowTile t(cols, off_lines(cols));
  const Span<kShort> sp(t.col, cols, cols % (128 * RowTile::kChunks) != 0);
  const int64_t c = min(t.chunk, (cols - 1) >> 7);
  Fp8x8 raw[kPasses];
  float sc[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {  // rows past the end read the last one again
    const int64_t row = min(t.row(p), rows - 1);
    load<true, kShort>(raw[p], q + row * cols, sp);
    sc[p] = s[c * rows + row];
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t row = t.row(p);
    float f[kVec];
    values(raw[p], sp, sc[p], f);
    if (row < rows) store8(x + row * ldx + t.col, sp.n, f);
  }
}

// ------------------------------------------------------------------ along the rows
// Requantisation for the weight gradient: a 512-thread block decodes a 128 x 128 tile into
// registers (4 consecutive rows x 8 columns a thread) and encodes its column groups.
template <bool kShort>
__global__ __launch_bounds__(kTileThreads) void ckpt_transpose_kernel(
    const uint8_t* __restrict__ q, const float* __restrict__ s, int64_t rows, int64_t cols,
    int pow2, uint8_t* __restrict__ qt, float* __restrict__ st) {
  __shared__ ColTile<1> sh;
  const uint32_t bands = static_cast<uint32_t>((rows + 127) >> 7);
  const uint32_t b = off_lines(cols) || off_lines(rows) ? xcd_range(blockIdx.x, gridDim.x)
                                                        : blockIdx.x;
  const int64_t cb = b / bands, mb = b % bands;
  const Span<kShort> sp(cb * 128 + (threadIdx.x & 15) * kVec, cols, off_lines(cols));
  const int64_t r0 = mb * 128 + (threadIdx.x >> 4) * kTileRows;
  Fp8x8 raw[kTileRows];
  float sc[kTileRows];
#pragma unroll
  for (int p = 0; p < kTileRows; ++p) {
    const int64_t row = min(r0 + p, rows - 1);
    load<true, kShort>(raw[p], q + row * cols, sp);
    sc[p] = s[cb * rows + row];
  }
  // A row past the end holds the last one again: it changes no maximum, and its codes are not
  // stored.
  float v[1][kTileRows][kVec];
#pragma unroll
  for (int p = 0; p < kTileRows; ++p) values(raw[p], sp, sc[p], v[0][p]);
  const ColOut out[1] = {{qt, st, cols, cb * 128}};
  col_codes<false>(sh, v, out, rows, mb, pow2 != 0);
}

puro_status check_rows(int64_t rows, int64_t cols, int64_t* blocks) {
  *blocks = row_tiles(rows, cols);
  return grid_ok(*blocks, 256) ? PURO_OK : PURO_ERR_SHAPE;
}

// The 16- or 32-bit side of a checkpoint: any row stride from cols up, element-aligned.
puro_status check_wide(const void* x, int type, int64_t cols, int64_t ldx, bool empty) {
  if (type != PURO_TYPE_BF16 && type != PURO_TYPE_FP32) return PURO_ERR_ARG;
  if (ldx < cols || ldx > (int64_t(1) << 40)) return PURO_ERR_ARG;
  if (empty) return PURO_OK;
  if (x == nullptr) return PURO_ERR_NULL;
  return aligned_to(x, type == PURO_TYPE_BF16 ? 2 : 4) ? PURO_OK : PURO_ERR_ALIGN;
}

}  // namespace
}  // namespace puro

using namespace puro;

extern "C" puro_status puro_ckpt_pack(const void* x, int x_type, int64_t rows, int64_t cols,
                                      int64_t ldx, int pow2, void* q, float* s, void* stream) {
  if (!any_dim_ok(rows) || !any_dim_ok(cols)) return PURO_ERR_SHAPE;
  const bool empty = rows == 0 || cols == 0;
  if (pow2 != 0 && pow2 != 1) return PURO_ERR_ARG;
  PURO_TRY(check_wide(x, x_type, cols, ldx, empty));
  PURO_TRY(check_ptr(q, empty));
  PURO_TRY(check_ptr(s, empty));
  if (empty) return PURO_OK;
  int64_t blocks;
  PURO_TRY(check_rows(rows, cols, &blocks));
  const dim3 grid(static_cast<uint32_t>(blocks));
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (x_type == PURO_TYPE_BF16) {
    const auto k = cols < kVec ? ckpt_pack_kernel<uint16_t, true>
                               : ckpt_pack_kernel<uint16_t, false>;
    hipLaunchKernelGGL(k, grid, dim3(256), 0, st, static_cast<const uint16_t*>(x), rows, cols, ldx,
                       pow2, static_cast<uint8_t*>(q), s);
  } else {
    const auto k = cols < kVec ? ckpt_pack_kernel<float, true> : ckpt_pack_kernel<float, false>;
    hipLaunchKernelGGL(k, grid, dim3(256), 0, st, static_cast<const float*>(x), rows, cols, ldx,
                       pow2, static_cast<uint8_t*>(q), s);
  }
  return launch_status();
}

extern "C" puro_status puro_ckpt_unpack(const void* q, const float* s, int64_t rows, int64_t cols,
                                        void* x, int x_type, int64_t ldx, void* stream) {
  if (!any_dim_ok(rows) || !any_dim_ok(cols)) return PURO_ERR_SHAPE;
  const bool empty = rows == 0 || cols == 0;
  PURO_TRY(check_ptr(q, empty));
  PURO_TRY(check_ptr(s, empty));
  PURO_TRY(check_wide(x, x_type, cols, ldx, empty));
  if (empty) return PURO_OK;
  int64_t blocks;
  PURO_TRY(check_rows(rows, cols, &blocks));
  const dim3 grid(static_cast<uint32_t>(blocks));
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (x_type == PURO_TYPE_BF16) {
    const auto k = cols < kVec ? ckpt_unpack_kernel<uint16_t, true>
                               : ckpt_unpack_kernel<uint16_t, false>;
    hipLaunchKernelGGL(k, grid, dim3(256), 0, st, static_cast<const uint8_t*>(q), s, rows, cols,
                       ldx, static_cast<uint16_t*>(x));
  } else {
    const auto k = cols < kVec ? ckpt_unpack_kernel<float, true>
                               : ckpt_unpack_kernel<float, false>;
    hipLaunchKernelGGL(k, grid, dim3(256), 0, st, static_cast<const uint8_t*>(q), s, rows, cols,
                       ldx, static_cast<float*>(x));
  }
  return launch_status();
}

extern "C" puro_status puro_ckpt_transpose(const void* q, const float* s, int64_t rows,
                                           int64_t cols, int pow2, void* qt, float* st,
                                           void* stream) {
  if (!any_dim_ok(rows) || !any_dim_ok(cols)) return PURO_ERR_SHAPE;
  const bool empty = rows == 0 || cols == 0;
  if (pow2 != 0 && pow2 != 1) return PURO_ERR_ARG;
  PURO_TRY(check_ptr(q, empty));
  PURO_TRY(check_ptr(s, empty));
  PURO_TRY(check_ptr(qt, empty));
  PURO_TRY(check_ptr(st, empty));
  if (empty) return PURO_OK;
  const int64_t blocks = ceil_div(rows, 128) * ceil_div(cols, 128);
  if (!grid_ok(blocks, kTileThreads)) return PURO_ERR_SHAPE;
  const auto k = cols < kVec ? ckpt_transpose_kernel<true> : ckpt_transpose_kernel<false>;
  hipLaunchKernelGGL(k, dim3(static_cast<uint32_t>(blocks)),
                     dim3(kTileThreads), 0, static_cast<hipStream_t>(stream),
                     static_cast<const uint8_t*>(q), s, rows, cols, pow2,
                     static_cast<uint8_t*>(qt), st);
  return launch_status();
}
