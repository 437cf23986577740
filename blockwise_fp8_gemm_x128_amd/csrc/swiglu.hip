// The gated activation of the MLP for gfx950, between the gate_up and the down projection:
//
//   gu = [g | u], f columns each;   h = u g sigma(g),   sigma(g) = 1/(1 + exp(-g))
//   dg = dh u sigma(g) (1 + g (1 - sigma(g))),   du = dh g sigma(g)
//
// The forward kernel writes h as the down projection's FP8 operand (and/or as bf16) and g, u as
// an 8-bit checkpoint; the backward kernels read the checkpoint (or bf16) and write dgu as bf16,
// or straight as the FP8 operands of gate_up's data and weight gradients, with h's transposed
// copy for down's weight gradient made from the same read.
//
// All of it is bound by HBM, the forward pass by its vector instructions as well (they issue 91 % of
// the time). All arithmetic is fp32; the exponential and the reciprocal are the hardware's (1 ulp
// each; the argument's own rounding adds |g| 2^-24), far inside the 2^-4 steps of the codes and the
// 2^-9 of bf16. The reciprocal has no subnormal results: for g below -87.3, where 1 + exp(-g)
// reaches 2^126, the sigmoid, less than 2^-126 there, counts as zero.
#include "coltile.hpp"

namespace puro {
namespace {

__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-g));
}

// Eight columns of g and u of one row, from bf16 or from the checkpoint.
struct GuSource {
  const uint16_t* gu;   // bf16 [rows][2f], or NULL
  const uint8_t* q;     // codes [rows][2f]
  const float* s;       // scales [2 ceil(f/128)][rows]
};
template <bool kCodes>
struct GuRaw {
  Bf16x8 g, u;
};
template <>
struct GuRaw<true> {
  Fp8x8 g, u;
  float sg, su;
};
template <bool kCodes, bool kShort>
__device__ __forceinline__ GuRaw<kCodes> load_gu(const GuSource& a, int64_t rows, int64_t f,
                                                 int64_t chunks, int64_t row, int64_t c,
                                                 const Span<kShort>& sp) {
  GuRaw<kCodes> o;
  if constexpr (kCodes) {
    load<true, kShort>(o.g, a.q + row * 2 * f, sp);
    load<true, kShort>(o.u, a.q + row * 2 * f + f, sp);
    o.sg = a.s[c * rows + row];
    o.su = a.s[(chunks + c) * rows + row];
  } else {
    load<true, kShort>(o.g, a.gu + row * 2 * f, sp);
    load<true, kShort>(o.u, a.gu + row * 2 * f + f, sp);
  }
  return o;
}
template <bool kCodes, bool kShort>
__device__ __forceinline__ void gu_values(const GuRaw<kCodes>& w, const Span<kShort>& sp, float* g,
                                          float* u) {
  if constexpr (kCodes) {
    values(w.g, sp, w.sg, g);
    values(w.u, sp, w.su, u);
  } else {
    values(w.g, sp, g);
    values(w.u, sp, u);
  }
}

// ------------------------------------------------------------------ forward
// Tiles of h as RowTile lays them out.
constexpr int kPasses = RowTile::kPasses;

struct FwdArgs {
  const uint16_t* gu;
  int64_t rows, f;
  uint16_t* h;
  uint8_t* hq;
  float* hs;
  uint8_t* guq;
  float* gus;
  int pow2;
};

template <bool kShort>
__global__ __launch_bounds__(256) void swiglu_fwd_kernel(const FwdArgs a) {
  const int64_t chunks = (a.f + 127) >> 7;
  const RowTile t(a.f, off_lines(a.f));
  const int l16 = threadIdx.x & 15;
  const int64_t c = t.chunk, col = t.col;
  const Span<kShort> sp(col, a.f, a.f % (128 * RowTile::kChunks) != 0);
  const int n = sp.n;
  const GuSource src = {a.gu, nullptr, nullptr};
  GuRaw<false> raw[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p)  // rows past the end read the last one again
    raw[p] = load_gu<false, kShort>(src, a.rows, a.f, chunks, min(t.row(p), a.rows - 1), c, sp);
  const bool pow2 = a.pow2 != 0;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t row = t.row(p);
    const bool in = row < a.rows;
    float v[3][kVec];  // g, u, h
    gu_values<false, kShort>(raw[p], sp, v[0], v[1]);
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[2][i] = v[0][i] * sigmoid(v[0][i]) * v[1][i];
    if (a.h != nullptr && in) store8(a.h + row * a.f + col, n, v[2]);
    const RowGroups<3> g = row_groups<true, 3>(v, pow2);
    if (!in || c >= chunks) continue;
    if (a.hq != nullptr) {
      store8(a.hq + row * a.f + col, n, encode8(v[2], g.r[2]));
      if (l16 == 2) a.hs[c * a.rows + row] = g.s;
    }
    if (a.guq != nullptr) {
      uint8_t* q = a.guq + row * 2 * a.f + col;
      store8<true>(q, n, encode8(v[0], g.r[0]));
      store8<true>(q + a.f, n, encode8(v[1], g.r[1]));
      if (l16 < 2) a.gus[(l16 * chunks + c) * a.rows + row] = g.s;
    }
  }
}

// ------------------------------------------------------------------ backward to bf16
struct BwdArgs {
  const uint16_t* dh;
  GuSource src;
  int64_t rows, f;
  uint16_t* dgu;
};

template <bool kCodes, bool kShort>
__global__ __launch_bounds__(256) void swiglu_bwd_kernel(const BwdArgs a) {
  const int64_t chunks = (a.f + 127) >> 7;
  const RowTile t(a.f, off_lines(a.f));
  const int64_t c = min(t.chunk, chunks - 1), col = t.col;
  const Span<kShort> sp(col, a.f, a.f % (128 * RowTile::kChunks) != 0);
  GuRaw<kCodes> raw[kPasses];
  Bf16x8 dhr[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {  // rows past the end read the last one again
    const int64_t row = min(t.row(p), a.rows - 1);
    raw[p] = load_gu<kCodes, kShort>(a.src, a.rows, a.f, chunks, row, c, sp);
    load<true, kShort>(dhr[p], a.dh + row * a.f, sp);
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t row = t.row(p);
    if (row >= a.rows) break;
    float g[kVec], u[kVec], dh[kVec];
    gu_values<kCodes, kShort>(raw[p], sp, g, u);
    values(dhr[p], sp, dh);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const float sg = sigmoid(g[i]);
      const float silu = g[i] * sg;
      g[i] = dh[i] * u[i] * fmaf(silu, 1.0f - sg, sg);
      u[i] = dh[i] * silu;
    }
    uint16_t* o = a.dgu + row * 2 * a.f + col;
    store8(o, sp.n, g);
    store8(o + a.f, sp.n, u);
  }
}

// ------------------------------------------------------------------ backward to FP8 operands
struct BwdFp8Args {
  const uint16_t* dh;
  GuSource src;
  int64_t rows, f;
  uint8_t* dguq;
  float* dgus;
  uint8_t* dgutq;
  float* dguts;
  uint8_t* htq;
  float* hts;
  int pow2;
};

// A thread's part of a 128 x 128 tile: rows r4 .. r4 + 3 and eight columns. Addresses are one
// 32-bit offset per lane (at most 127 (2 f) + 128 < 2^32 for f <= 2^24) on top of a uniform pointer
// per row.
struct TilePart {
  int64_t chunks, c, mb;
  uint32_t r4, at1, at2;   // element offsets in tensors of f and of 2f columns
  int64_t base1, base2;
  __device__ __forceinline__ TilePart(int64_t rows, int64_t f) {
    const uint32_t bands = static_cast<uint32_t>(rows >> 7);
    chunks = f >> 7;
    c = blockIdx.x / bands, mb = blockIdx.x % bands;
    r4 = (threadIdx.x >> 4) * kTileRows;
    at1 = r4 * static_cast<uint32_t>(f) + (threadIdx.x & 15) * kVec;
    at2 = r4 * 2 * static_cast<uint32_t>(f) + (threadIdx.x & 15) * kVec;
    base1 = mb * 128 * f + c * 128;
    base2 = mb * 256 * f + c * 128;
  }
};

template <bool kCodes>
struct TileRaw {
  GuRaw<kCodes> gu[kTileRows];
  Bf16x8 dh[kTileRows];
};
template <bool kCodes>
__device__ __forceinline__ void load_tile(TileRaw<kCodes>& w, const BwdFp8Args& a,
                                          const TilePart& t, const Span<false>& sp) {
  constexpr bool kShort = false;
#pragma unroll
  for (int p = 0; p < kTileRows; ++p) {
    const int64_t g = t.base2 + p * 2 * a.f;
    if constexpr (kCodes) {
      load<true, kShort>(w.gu[p].g, a.src.q + g + t.at2, sp);
      load<true, kShort>(w.gu[p].u, a.src.q + g + a.f + t.at2, sp);
    } else {
      load<true, kShort>(w.gu[p].g, a.src.gu + g + t.at2, sp);
      load<true, kShort>(w.gu[p].u, a.src.gu + g + a.f + t.at2, sp);
    }
    load<true, kShort>(w.dh[p], a.dh + t.base1 + p * a.f + t.at1, sp);
  }
  if constexpr (kCodes) {
    const float* s = a.src.s + t.c * a.rows + t.mb * 128;
    const float4 sg = *reinterpret_cast<const float4*>(s + t.r4);
    const float4 su = *reinterpret_cast<const float4*>(s + t.chunks * a.rows + t.r4);
    w.gu[0].sg = sg.x, w.gu[1].sg = sg.y, w.gu[2].sg = sg.z, w.gu[3].sg = sg.w;
    w.gu[0].su = su.x, w.gu[1].su = su.y, w.gu[2].su = su.z, w.gu[3].su = su.w;
  }
}

// Codes of dg (t = 0) or du (t = 1) in the row orientation.
template <bool kLater>
__device__ __forceinline__ void store_rows(const float (&v)[kTileRows][kVec], const BwdFp8Args& a,
                                           const TilePart& t, int which) {
  const RowGroups<kTileRows> rg = row_groups<false, kTileRows>(v, a.pow2 != 0);
#pragma unroll
  for (int p = 0; p < kTileRows; ++p)
    store8<kLater>(a.dguq + t.base2 + p * 2 * a.f + which * a.f + t.at2, kVec,
                   encode8(v[p], rg.r[p]));
  const uint32_t l16 = threadIdx.x & 15;
  if (l16 < kTileRows)
    a.dgus[(which * t.chunks + t.c) * a.rows + t.mb * 128 + t.r4 + l16] = rg.s;
}

// Four waves per SIMD, two blocks per CU, so that one block's loads and stores run under the
// other's arithmetic: that caps the registers at 128, of which the three tensors' values take 96.
// kLater: the codes go past the caches, for outputs larger than these (see the launch).
template <bool kCodes, bool kLater>
__global__ __launch_bounds__(kTileThreads, 4) void swiglu_bwd_fp8_kernel(const BwdFp8Args a) {
  __shared__ ColTile<3> sh;
  const TilePart t(a.rows, a.f);
  Span<false> sp;  // whole groups: never cut short
  sp.at = 0, sp.n = kVec, sp.cut = false;
  float v[3][kTileRows][kVec];  // dg, du, h
  {
    TileRaw<kCodes> raw;
    load_tile(raw, a, t, sp);
#pragma unroll
    for (int p = 0; p < kTileRows; ++p) {
      float g[kVec], u[kVec], dh[kVec];
      gu_values<kCodes, false>(raw.gu[p], sp, g, u);
      values(raw.dh[p], sp, dh);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const float sg = sigmoid(g[i]);
        const float silu = g[i] * sg;
        v[0][p][i] = dh[i] * u[i] * fmaf(silu, 1.0f - sg, sg);
        v[1][p][i] = dh[i] * silu;
        v[2][p][i] = silu * u[i];
      }
      // The compiler would rather keep the inputs and work the values out where they are used,
      // which takes more registers than there are: the empty statements pin the values here.
#pragma unroll
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < kVec; ++i) asm volatile("" : "+v"(v[k][p][i]));
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    store_rows<kLater>(v[k], a, t, k);
    __builtin_amdgcn_sched_barrier(0);
  }
  const ColOut out[3] = {{a.dgutq, a.dguts, 2 * a.f, t.c * 128},
                         {a.dgutq, a.dguts, 2 * a.f, a.f + t.c * 128},
                         {a.htq, a.hts, a.f, t.c * 128}};
  col_codes<kLater>(sh, v, out, a.rows, t.mb, a.pow2 != 0);
}

// The same with one block per tile and tensor (grid y: dg, du, h), which reads the inputs again and
// works the sigmoid out again but has three times the blocks and a third of the work in each.
template <bool kCodes>
__global__ __launch_bounds__(kTileThreads) void swiglu_bwd_fp8_split_kernel(const BwdFp8Args a) {
  __shared__ ColTile<1> sh;
  const TilePart t(a.rows, a.f);
  const int which = blockIdx.y;
  Span<false> sp;
  sp.at = 0, sp.n = kVec, sp.cut = false;
  float v[1][kTileRows][kVec];
  TileRaw<kCodes> raw;
  load_tile(raw, a, t, sp);
#pragma unroll
  for (int p = 0; p < kTileRows; ++p) {
    float g[kVec], u[kVec], dh[kVec];
    gu_values<kCodes, false>(raw.gu[p], sp, g, u);
    values(raw.dh[p], sp, dh);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const float sg = sigmoid(g[i]);
      const float silu = g[i] * sg;
      v[0][p][i] = which == 0   ? dh[i] * u[i] * fmaf(silu, 1.0f - sg, sg)
                   : which == 1 ? dh[i] * silu
                                : silu * u[i];
    }
  }
  if (which < 2) store_rows<false>(v[0], a, t, which);
  const ColOut out[1] = {{which < 2 ? a.dgutq : a.htq, which < 2 ? a.dguts : a.hts,
                          which < 2 ? 2 * a.f : a.f, (which == 1 ? a.f : 0) + t.c * 128}};
  col_codes<false>(sh, v, out, a.rows, t.mb, a.pow2 != 0);
}

puro_status check_gu(const void* gu, const void* guq, const float* gus, bool empty) {
  if (empty) return PURO_OK;
  if (gu != nullptr) return guq != nullptr || gus != nullptr ? PURO_ERR_ARG : check_ptr(gu, false);
  PURO_TRY(check_ptr(guq, false));
  return check_ptr(gus, false);
}

}  // namespace
}  // namespace puro

using namespace puro;

extern "C" puro_status puro_swiglu_fwd(const void* gu, int64_t rows, int64_t f, void* h, void* hq,
                                       float* hs, void* guq, float* gus, int pow2, void* stream) {
  if (!any_dim_ok(rows) || !any_dim_ok(f)) return PURO_ERR_SHAPE;
  if (pow2 != 0 && pow2 != 1) return PURO_ERR_ARG;
  const bool empty = rows == 0 || f == 0;
  if (empty) return PURO_OK;
  if (h == nullptr && hq == nullptr && guq == nullptr) return PURO_ERR_NULL;
  PURO_TRY(check_ptr(gu, false));
  PURO_TRY(check_optional(h));
  if (hq != nullptr || hs != nullptr) {
    PURO_TRY(check_ptr(hq, false));
    PURO_TRY(check_ptr(hs, false));
  }
  if (guq != nullptr || gus != nullptr) {
    PURO_TRY(check_ptr(guq, false));
    PURO_TRY(check_ptr(gus, false));
  }
  const int64_t blocks = row_tiles(rows, f);
  if (!grid_ok(blocks, 256)) return PURO_ERR_SHAPE;
  const FwdArgs a = {static_cast<const uint16_t*>(gu), rows, f, static_cast<uint16_t*>(h),
                     static_cast<uint8_t*>(hq), hs, static_cast<uint8_t*>(guq), gus, pow2};
  const auto k = f < kVec ? swiglu_fwd_kernel<true> : swiglu_fwd_kernel<false>;
  hipLaunchKernelGGL(k, dim3(static_cast<uint32_t>(blocks)), dim3(256), 0,
                     static_cast<hipStream_t>(stream), a);
  return launch_status();
}

extern "C" puro_status puro_swiglu_bwd(const void* dh, const void* gu, const void* guq,
                                       const float* gus, int64_t rows, int64_t f, void* dgu,
                                       void* stream) {
  if (!any_dim_ok(rows) || !any_dim_ok(f)) return PURO_ERR_SHAPE;
  const bool empty = rows == 0 || f == 0;
  PURO_TRY(check_ptr(dh, empty));
  PURO_TRY(check_gu(gu, guq, gus, empty));
  PURO_TRY(check_ptr(dgu, empty));
  if (empty) return PURO_OK;
  const int64_t blocks = row_tiles(rows, f);
  if (!grid_ok(blocks, 256)) return PURO_ERR_SHAPE;
  const BwdArgs a = {static_cast<const uint16_t*>(dh),
                     {static_cast<const uint16_t*>(gu), static_cast<const uint8_t*>(guq), gus},
                     rows, f, static_cast<uint16_t*>(dgu)};
  const dim3 grid(static_cast<uint32_t>(blocks));
  const auto k = gu != nullptr
                     ? (f < kVec ? swiglu_bwd_kernel<false, true> : swiglu_bwd_kernel<false, false>)
                     : (f < kVec ? swiglu_bwd_kernel<true, true> : swiglu_bwd_kernel<true, false>);
  hipLaunchKernelGGL(k, grid, dim3(256), 0, static_cast<hipStream_t>(stream), a);
  return launch_status();
}

extern "C" puro_status puro_swiglu_bwd_fp8(const void* dh, const void* gu, const void* guq,
                                           const float* gus, int64_t rows, int64_t f, int pow2,
                                           void* dguq, float* dgus, void* dgutq, float* dguts,
                                           void* htq, float* hts, void* stream) {
  if (!dim_ok(rows) || !dim_ok(f)) return PURO_ERR_SHAPE;
  const bool empty = rows == 0 || f == 0;
  if (pow2 != 0 && pow2 != 1) return PURO_ERR_ARG;
  PURO_TRY(check_ptr(dh, empty));
  PURO_TRY(check_gu(gu, guq, gus, empty));
  for (const void* p : {static_cast<const void*>(dguq), static_cast<const void*>(dgus),
                        static_cast<const void*>(dgutq), static_cast<const void*>(dguts),
                        static_cast<const void*>(htq), static_cast<const void*>(hts)})
    PURO_TRY(check_ptr(p, empty));
  if (empty) return PURO_OK;
  const int64_t blocks = (rows / 128) * (f / 128);
  if (!grid_ok(blocks, kTileThreads)) return PURO_ERR_SHAPE;
  const BwdFp8Args a = {static_cast<const uint16_t*>(dh),
                        {static_cast<const uint16_t*>(gu), static_cast<const uint8_t*>(guq), gus},
                        rows, f, static_cast<uint8_t*>(dguq), dgus, static_cast<uint8_t*>(dgutq),
                        dguts, static_cast<uint8_t*>(htq), hts, pow2};
  // Tiles that leave two thirds of the CUs idle are split by tensor: 128 x 6144 (48 tiles) in 7.2
  // us against 8.2, 1024 x 1024 (64) in 7.4 against 8.4; but 1024 x 2048 (128) in 10.3 against 9.4.
  const bool split = 3 * blocks <= 256;
  // Codes of more bytes than the memory-side cache has (5 per element of h, 256 MiB) cannot all
  // wait there for the GEMMs that read them, and go past it: 16384 x 6144 in 186 us against 198.
  // Smaller ones stay: 4096 x 2048 in 17.7 us against 18.3, and their readers find them.
  const bool later = 5 * rows * f > (int64_t(256) << 20);
  const auto k = gu != nullptr ? (split   ? swiglu_bwd_fp8_split_kernel<false>
                                  : later ? swiglu_bwd_fp8_kernel<false, true>
                                          : swiglu_bwd_fp8_kernel<false, false>)
                               : (split   ? swiglu_bwd_fp8_split_kernel<true>
                                  : later ? swiglu_bwd_fp8_kernel<true, true>
                                          : swiglu_bwd_fp8_kernel<true, false>);
  hipLaunchKernelGGL(k, dim3(static_cast<uint32_t>(blocks), split ? 3 : 1), dim3(kTileThreads), 0,
                     static_cast<hipStream_t>(stream), a);
  return launch_status();
}
