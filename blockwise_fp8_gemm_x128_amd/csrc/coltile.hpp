// Column groups of a 128 x 128 tile held in registers: the transposed codes and scales that the
// weight-gradient GEMM reads (groups along the tokens), from fp32 values, for kN tensors at once.
//
// A 512-thread block holds the tile as 4 consecutive rows x 8 consecutive columns per thread
// (16 lanes cover a row, each wave 16 rows). A column's largest magnitude is a register maximum
// over 4 rows, and then 32 words of LDS over the block, which one thread per column reads (lane
// swaps within the wave first cost more instructions than the reads); that thread also does the
// divisions. Only codes are transposed through LDS, one byte per element: four rows of a column
// are one dword, and a column's 128 bytes leave as one line.
//
// Maxima and reciprocal scales of column 8 l + i stand at 64 (i / 4) + 4 l + i mod 4, so that a
// lane's eight are two 16 B accesses, each contiguous over the lanes (as 8 l + i they were half of
// the kernels' bank conflicts).
//
// Dword of column 8 l + i, rows 4 g .. 4 g + 3: codes[(16 i + l) * kPitch + g]. With a pitch of 36
// dwords the 16 lanes of a row start 16 different multiples of 4 banks and the wave's four row
// groups fill the banks between, so the writes are free of conflicts and the reads are 16 B.
//
// Tiles are numbered down the rows first, so that blocks running together write neighbouring lines
// of the transposed codes (across the columns first, 16384 x 6144 of the activation's gradient took
// 199 us instead of 190; 185 since its codes go past the caches).
#pragma once
#include "block.hpp"

namespace puro {

constexpr int kTileThreads = 512;
constexpr int kTileRows = 4;   // rows per thread

template <int kN>
struct ColTile {
  static constexpr int kPitch = 36;
  // The maxima are read for the last time a barrier before the first code is written.
  union __attribute__((aligned(16))) {
    uint32_t codes[kN][128 * kPitch];
    float maxima[kN][32][128];
  };
  alignas(16) float r[kN][128];
  int odd;
};

// Where one tensor's transposed codes go: qt [cols][rows], st [ceil(rows/128)][cols].
struct ColOut {
  uint8_t* qt;
  float* st;
  int64_t cols;   // columns of the tensor
  int64_t c0;     // first column of this tile
};

template <int kN, bool kFinite>
__device__ __forceinline__ void col_maxima(ColTile<kN>& sh, const float (&v)[kN][kTileRows][kVec]) {
  const int l16 = threadIdx.x & 15, seg = threadIdx.x >> 4;
#pragma unroll
  for (int t = 0; t < kN; ++t) {
    float m[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if constexpr (kFinite) {
        uint32_t u = finite_mag(v[t][0][i]);
#pragma unroll
        for (int p = 1; p < kTileRows; ++p) u = umax32(u, finite_mag(v[t][p][i]));
        m[i] = __uint_as_float(u);
      } else {  // computed values: NaN are quiet and passed over, infinities noticed
        m[i] = __builtin_fabsf(v[t][0][i]);
#pragma unroll
        for (int p = 1; p < kTileRows; ++p) m[i] = fmaxf(m[i], __builtin_fabsf(v[t][p][i]));
      }
    }
    float4* dst = reinterpret_cast<float4*>(&sh.maxima[t][seg][4 * l16]);
    dst[0] = make_float4(m[0], m[1], m[2], m[3]);
    dst[16] = make_float4(m[4], m[5], m[6], m[7]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

template <int kN, bool kMark>
__device__ __forceinline__ void col_scales(ColTile<kN>& sh, const ColOut (&out)[kN], int64_t mb,
                                           bool pow2) {
  const int t = threadIdx.x;
  if (t < kN * 128) {
    const int k = __builtin_amdgcn_readfirstlane(t >> 7), pos = t & 127;  // one tensor per wave
    const int c = 2 * (pos & 60) + (pos >> 6) * 4 + (pos & 3);
    float x = sh.maxima[k][0][pos];
#pragma unroll
    for (int w = 1; w < 32; ++w) x = fmaxf(x, sh.maxima[k][w][pos]);
    const uint32_t m = mag(x);
    if (kMark && m >= kInfBits) sh.odd = 1;  // every writer writes the same value
    float s, r;
    ckpt_scale(m, pow2, s, r);
    sh.r[k][pos] = r;
#pragma unroll
    for (int j = 0; j < kN; ++j)
      if (k == j && out[j].c0 + c < out[j].cols)
        out[j].st[mb * out[j].cols + out[j].c0 + c] = s;
  }
}

// All 512 threads call it once; v[t][p][i] is element (row m0 + 4 (thread/16) + p, column
// c0 + 8 (thread mod 16) + i) of tensor t; columns past the end are zero, rows past the end repeat
// the last one (which changes no maximum; their codes are not stored).
template <bool kLater, int kN>
__device__ __forceinline__ void col_codes(ColTile<kN>& sh, const float (&v)[kN][kTileRows][kVec],
                                          const ColOut (&out)[kN], int64_t rows, int64_t mb,
                                          bool pow2) {
  static_assert(kN * 128 <= kTileThreads, "one thread per column of each tensor");
  const int t = threadIdx.x, l16 = t & 15, seg = t >> 4;
  if (t == 0) sh.odd = 0;
  col_maxima<kN, false>(sh, v);
  __syncthreads();
  // An infinite maximum (or NaN: a column of nothing else) marks the tile, which is then gone over
  // again with the finite maxima; the first pass's scales are overwritten by the same threads.
  col_scales<kN, true>(sh, out, mb, pow2);
  __syncthreads();
  if (sh.odd != 0) {
    col_maxima<kN, true>(sh, v);
    __syncthreads();
    col_scales<kN, false>(sh, out, mb, pow2);
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const float4 r0 = *reinterpret_cast<const float4*>(&sh.r[k][4 * l16]);
    const float4 r1 = *reinterpret_cast<const float4*>(&sh.r[k][64 + 4 * l16]);
    const float rs[kVec] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const float r = rs[i];
      const float a = v[k][0][i], b = v[k][1][i], c = v[k][2][i], d = v[k][3][i];
      sh.codes[k][(16 * i + l16) * ColTile<kN>::kPitch + seg] =
          codes4(a * r, b * r, c * r, d * r);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  __syncthreads();
  const int64_t row = mb * 128 + 16 * (t & 7);
  const int64_t left = rows - row;
#pragma unroll
  for (int k = 0; k < kN; ++k)
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      const int pos = pass * 64 + (t >> 3);
      const int64_t col = out[k].c0 + 8 * (pos & 15) + (pos >> 4);
      const uint4 w = *reinterpret_cast<const uint4*>(
          &sh.codes[k][pos * ColTile<kN>::kPitch + 4 * (t & 7)]);
      if (col >= out[k].cols) continue;
      uint8_t* p = out[k].qt + col * rows + row;
      if (left >= 16) {
        put<kLater>(reinterpret_cast<u32x4_el*>(p), u32x4_el{w.x, w.y, w.z, w.w});
      } else {
        const uint32_t b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < left) p[i] = static_cast<uint8_t>(b[i >> 2] >> (8 * (i & 3)));
      }
    }
}

}  // namespace puro
