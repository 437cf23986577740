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
// All of it is bound by HBM. All arithmetic is fp32; the exponential and the reciprocal are the
// hardware's (1 ulp each; the argument's own rounding adds |g| 2^-24), far inside the 2^-4 steps
// of the codes and the 2^-9 of bf16.
#include "coltile.hpp"

namespace puro {
namespace {

__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-g));
}

// One row of eight: values of g and u, from bf16 or from the checkpoint.
struct GuSource {
  const uint16_t* gu;   // bf16 [rows][2f], or NULL
  const uint8_t* q;     // codes [rows][2f]
  const float* s;       // scales [2 ceil(f/128)][rows]
};
template <bool kCodes>
struct GuRaw {
  u32x4_el g, u;
};
template <>
struct GuRaw<true> {
  u32x2_el g, u;
  float sg, su;
};
template <bool kCodes>
__device__ __forceinline__ GuRaw<kCodes> load_gu(const GuSource& a, int64_t rows, int64_t f,
                                                 int64_t chunks, int64_t row, int64_t c,
                                                 int64_t col, int n) {
  GuRaw<kCodes> o;
  const int64_t at = row * 2 * f + col;
  if constexpr (kCodes) {
    o.g = load_raw<true>(a.q + at, n);
    o.u = load_raw<true>(a.q + at + f, n);
    o.sg = n > 0 ? a.s[c * rows + row] : 0.0f;
    o.su = n > 0 ? a.s[(chunks + c) * rows + row] : 0.0f;
  } else {
    o.g = load_raw<true>(a.gu + at, n);
    o.u = load_raw<true>(a.gu + at + f, n);
  }
  return o;
}
template <bool kCodes>
__device__ __forceinline__ void values(const GuRaw<kCodes>& w, float* g, float* u) {
  if constexpr (kCodes) {
    decode8(w.g, w.sg, g);
    decode8(w.u, w.su, u);
  } else {
    widen8(w.g, g);
    widen8(w.u, u);
  }
}

// ------------------------------------------------------------------ forward
// As the 1x128 quantisers: a 256-thread block covers 64 rows of one 128-column chunk of h.
constexpr int kPasses = 4;
constexpr int kRowsPerBlock = 16 * kPasses;

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

__global__ __launch_bounds__(256) void swiglu_fwd_kernel(const FwdArgs a) {
  const int64_t chunks = (a.f + 127) >> 7;
  const int64_t c = blockIdx.x % chunks;
  const int64_t r0 = blockIdx.x / chunks * kRowsPerBlock + (threadIdx.x >> 4);
  const int l16 = threadIdx.x & 15;
  const int64_t col = c * 128 + l16 * kVec;
  const int n = static_cast<int>(min(a.f - col, int64_t(kVec)));
  const GuSource src = {a.gu, nullptr, nullptr};
  GuRaw<false> raw[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t row = r0 + 16 * p;
    raw[p] = load_gu<false>(src, a.rows, a.f, chunks, row, c, col, row < a.rows ? n : 0);
  }
  const bool pow2 = a.pow2 != 0;
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t row = r0 + 16 * p;
    const bool in = row < a.rows;
    float v[3][kVec];  // g, u, h
    values<false>(raw[p], v[0], v[1]);
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[2][i] = v[0][i] * sigmoid(v[0][i]) * v[1][i];
    if (a.h != nullptr && in) store8(a.h + row * a.f + col, n, v[2]);
    const RowGroups<3> g = row_groups<true, 3>(v, pow2);
    if (!in) continue;
    if (a.hq != nullptr) {
      store8(a.hq + row * a.f + col, n, encode8(v[2], g.r[2]));
      if (l16 == 2) a.hs[c * a.rows + row] = g.s;
    }
    if (a.guq != nullptr) {
      uint8_t* q = a.guq + row * 2 * a.f + col;
      store8(q, n, encode8(v[0], g.r[0]));
      store8(q + a.f, n, encode8(v[1], g.r[1]));
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

template <bool kCodes>
__global__ __launch_bounds__(256) void swiglu_bwd_kernel(const BwdArgs a) {
  const int64_t chunks = (a.f + 127) >> 7;
  const int64_t c = blockIdx.x % chunks;
  const int64_t r0 = blockIdx.x / chunks * kRowsPerBlock + (threadIdx.x >> 4);
  const int64_t col = c * 128 + (threadIdx.x & 15) * kVec;
  const int n = static_cast<int>(min(a.f - col, int64_t(kVec)));
  GuRaw<kCodes> raw[kPasses];
  u32x4_el dhr[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t row = r0 + 16 * p;
    const int k = row < a.rows ? n : 0;
    raw[p] = load_gu<kCodes>(a.src, a.rows, a.f, chunks, row, c, col, k);
    dhr[p] = load_raw<true>(a.dh + row * a.f + col, k);
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t row = r0 + 16 * p;
    if (row >= a.rows) break;
    float g[kVec], u[kVec], dh[kVec];
    values<kCodes>(raw[p], g, u);
    widen8(dhr[p], dh);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const float sg = sigmoid(g[i]);
      const float t = dh[i] * sg;
      const float gi = g[i];
      g[i] = t * u[i] * fmaf(gi, 1.0f - sg, 1.0f);
      u[i] = t * gi;
    }
    uint16_t* o = a.dgu + row * 2 * a.f + col;
    store8(o, n, g);
    store8(o + a.f, n, u);
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

// Four waves per SIMD, two blocks per CU, so that one block's loads and stores run under the
// other's arithmetic: that caps the registers at 128, of which the three tensors' values take 96.
// Addresses are therefore one 32-bit offset per lane on top of a uniform pointer per row.
template <bool kCodes>
__global__ __launch_bounds__(kTileThreads, 4) void swiglu_bwd_fp8_kernel(const BwdFp8Args a) {
  __shared__ ColTile<3> sh;
  const int64_t chunks = a.f >> 7;
  const int64_t c = blockIdx.x % chunks, mb = blockIdx.x / chunks;
  const int l16 = threadIdx.x & 15;
  const uint32_t f = static_cast<uint32_t>(a.f);
  const uint32_t r4 = (threadIdx.x >> 4) * kTileRows;  // first of the thread's rows in the tile
  // at most 127 (2 f) + 128 < 2^32 for f <= 2^24
  const uint32_t at1 = r4 * f + l16 * kVec, at2 = r4 * 2 * f + l16 * kVec;
  const int64_t base1 = mb * 128 * a.f + c * 128, base2 = mb * 256 * a.f + c * 128;
  float v[3][kTileRows][kVec];  // dg, du, h
  {
    GuRaw<kCodes> raw[kTileRows];
    u32x4_el dhr[kTileRows];
#pragma unroll
    for (int p = 0; p < kTileRows; ++p) {
      if constexpr (kCodes) {
        raw[p].g = load_raw<true>(a.src.q + base2 + p * 2 * a.f + at2, kVec);
        raw[p].u = load_raw<true>(a.src.q + base2 + p * 2 * a.f + a.f + at2, kVec);
      } else {
        raw[p].g = load_raw<true>(a.src.gu + base2 + p * 2 * a.f + at2, kVec);
        raw[p].u = load_raw<true>(a.src.gu + base2 + p * 2 * a.f + a.f + at2, kVec);
      }
      dhr[p] = load_raw<true>(a.dh + base1 + p * a.f + at1, kVec);
    }
    if constexpr (kCodes) {
      const float4 sg = *reinterpret_cast<const float4*>(a.src.s + c * a.rows + mb * 128 + r4);
      const float4 su =
          *reinterpret_cast<const float4*>(a.src.s + (chunks + c) * a.rows + mb * 128 + r4);
      raw[0].sg = sg.x, raw[1].sg = sg.y, raw[2].sg = sg.z, raw[3].sg = sg.w;
      raw[0].su = su.x, raw[1].su = su.y, raw[2].su = su.z, raw[3].su = su.w;
    }
#pragma unroll
    for (int p = 0; p < kTileRows; ++p) {
      float g[kVec], u[kVec], dh[kVec];
      values<kCodes>(raw[p], g, u);
      widen8(dhr[p], dh);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const float sg = sigmoid(g[i]);
        const float t = dh[i] * sg;
        v[0][p][i] = t * u[i] * fmaf(g[i], 1.0f - sg, 1.0f);
        v[1][p][i] = t * g[i];
        v[2][p][i] = g[i] * sg * u[i];
      }
      // The compiler would rather keep the inputs and work the values out where they are used,
      // which takes more registers than there are: the empty statements pin the values here.
#pragma unroll
      for (int t = 0; t < 3; ++t)
#pragma unroll
        for (int i = 0; i < kVec; ++i) asm volatile("" : "+v"(v[t][p][i]));
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  const bool pow2 = a.pow2 != 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const RowGroups<kTileRows> rg = row_groups<false, kTileRows>(v[t], pow2);
#pragma unroll
    for (int p = 0; p < kTileRows; ++p)
      store8(a.dguq + base2 + p * 2 * a.f + t * a.f + at2, kVec, encode8(v[t][p], rg.r[p]));
    if (l16 < kTileRows) a.dgus[(t * chunks + c) * a.rows + mb * 128 + r4 + l16] = rg.s;
    __builtin_amdgcn_sched_barrier(0);
  }
  const ColOut out[3] = {{a.dgutq, a.dguts, 2 * a.f, c * 128},
                         {a.dgutq, a.dguts, 2 * a.f, a.f + c * 128},
                         {a.htq, a.hts, a.f, c * 128}};
  col_codes<3>(sh, v, out, a.rows, mb, pow2);
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
  const int64_t blocks = ceil_div(rows, kRowsPerBlock) * ceil_div(f, 128);
  if (blocks > INT32_MAX) return PURO_ERR_SHAPE;
  const FwdArgs a = {static_cast<const uint16_t*>(gu), rows, f, static_cast<uint16_t*>(h),
                     static_cast<uint8_t*>(hq), hs, static_cast<uint8_t*>(guq), gus, pow2};
  hipLaunchKernelGGL(swiglu_fwd_kernel, dim3(static_cast<uint32_t>(blocks)), dim3(256), 0,
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
  const int64_t blocks = ceil_div(rows, kRowsPerBlock) * ceil_div(f, 128);
  if (blocks > INT32_MAX) return PURO_ERR_SHAPE;
  const BwdArgs a = {static_cast<const uint16_t*>(dh),
                     {static_cast<const uint16_t*>(gu), static_cast<const uint8_t*>(guq), gus},
                     rows, f, static_cast<uint16_t*>(dgu)};
  const dim3 grid(static_cast<uint32_t>(blocks));
  if (gu != nullptr)
    hipLaunchKernelGGL(swiglu_bwd_kernel<false>, grid, dim3(256), 0,
                       static_cast<hipStream_t>(stream), a);
  else
    hipLaunchKernelGGL(swiglu_bwd_kernel<true>, grid, dim3(256), 0,
                       static_cast<hipStream_t>(stream), a);
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
  if (blocks > INT32_MAX) return PURO_ERR_SHAPE;
  const BwdFp8Args a = {static_cast<const uint16_t*>(dh),
                        {static_cast<const uint16_t*>(gu), static_cast<const uint8_t*>(guq), gus},
                        rows, f, static_cast<uint8_t*>(dguq), dgus, static_cast<uint8_t*>(dgutq),
                        dguts, static_cast<uint8_t*>(htq), hts, pow2};
  const dim3 grid(static_cast<uint32_t>(blocks));
  if (gu != nullptr)
    hipLaunchKernelGGL(swiglu_bwd_fp8_kernel<false>, grid, dim3(kTileThreads), 0,
                       static_cast<hipStream_t>(stream), a);
  else
    hipLaunchKernelGGL(swiglu_bwd_fp8_kernel<true>, grid, dim3(kTileThreads), 0,
                       static_cast<hipStream_t>(stream), a);
  return launch_status();
}
