// Shared device and host helpers of the operators between the GEMMs (norm.hip, swiglu.hip,
// ckpt.hip): vectors of eight elements at any element alignment and with a ragged end, sums over
// the lanes of a row, and the 8-bit checkpoint's group scale and encoding.
//
// The unit of work everywhere is eight consecutive columns per lane, so that 16 lanes (one DPP
// row) hold one group of 128 columns: the group's largest magnitude is four DPP steps away.
#pragma once
#include "common.hpp"

namespace puro {

constexpr int kVec = 8;
constexpr uint32_t kInfBits = 0x7f800000u;

inline bool aligned_to(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Rows and columns of the operators here: any size up to kMaxDim.
inline bool any_dim_ok(int64_t d) { return d >= 0 && d <= kMaxDim; }

// Checks one tensor pointer that may be NULL to leave its tensor out.
inline puro_status check_optional(const void* p) {
  return p == nullptr || aligned16(p) ? PURO_OK : PURO_ERR_ALIGN;
}

// ---------------------------------------------------------------- vectors of eight
// Rows of any length start at any element, so vectors are only element-aligned; the global
// memory instructions take any address, and an aligned vector costs what it always did.
typedef uint32_t u32x4_el __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_el __attribute__((ext_vector_type(2), aligned(1)));
typedef float f32x4_el __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ void widen8(const u32x4_el v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(v[i]);
    f[2 * i + 1] = bf16_hi(v[i]);
  }
}

// n: elements of the vector that exist (columns left in the row); the others read as zero.
// `kOnce`: the input is read by nobody else soon, keep it out of the caches' way.
template <bool kOnce>
__device__ __forceinline__ u32x4_el load_raw(const uint16_t* p, int n) {
  u32x4_el v = {0, 0, 0, 0};
  if (n >= kVec) {
    const u32x4_el* q = reinterpret_cast<const u32x4_el*>(p);
    v = kOnce ? __builtin_nontemporal_load(q) : *q;
  } else if (n > 0) {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (i < n) v[i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
  }
  return v;
}

struct F8 {
  float f[kVec];
};
template <bool kOnce>
__device__ __forceinline__ F8 load8(const uint16_t* p, int n) {
  F8 o;
  widen8(load_raw<kOnce>(p, n), o.f);
  return o;
}
template <bool kOnce>
__device__ __forceinline__ F8 load8(const float* p, int n) {
  F8 o;
  if (n >= kVec) {
    const f32x4_el* q = reinterpret_cast<const f32x4_el*>(p);
    const f32x4_el a = kOnce ? __builtin_nontemporal_load(q) : q[0];
    const f32x4_el b = kOnce ? __builtin_nontemporal_load(q + 1) : q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o.f[i] = a[i];
      o.f[4 + i] = b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) o.f[i] = i < n ? p[i] : 0.0f;
  }
  return o;
}
// Eight E4M3 codes as eight bytes.
template <bool kOnce>
__device__ __forceinline__ u32x2_el load_raw(const uint8_t* p, int n) {
  u32x2_el v = {0, 0};
  if (n >= kVec) {
    const u32x2_el* q = reinterpret_cast<const u32x2_el*>(p);
    v = kOnce ? __builtin_nontemporal_load(q) : *q;
  } else if (n > 0) {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (i < n) v[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  }
  return v;
}
// Values the codes stand for, times their group's scale (one fp32 product each).
__device__ __forceinline__ void decode8(const u32x2_el v, float s, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(v[i], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(v[i], true);
    f[4 * i] = lo[0] * s;
    f[4 * i + 1] = lo[1] * s;
    f[4 * i + 2] = hi[0] * s;
    f[4 * i + 3] = hi[1] * s;
  }
}

__device__ __forceinline__ void store8(uint16_t* p, int n, const float* f) {
  u32x4_el v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  if (n >= kVec) {
    *reinterpret_cast<u32x4_el*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (i < n) p[i] = static_cast<uint16_t>(v[i >> 1] >> (16 * (i & 1)));
  }
}
__device__ __forceinline__ void store8(float* p, int n, const float* f) {
  if (n >= kVec) {
    f32x4_el* q = reinterpret_cast<f32x4_el*>(p);
    q[0] = f32x4_el{f[0], f[1], f[2], f[3]};
    q[1] = f32x4_el{f[4], f[5], f[6], f[7]};
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (i < n) p[i] = f[i];
  }
}
__device__ __forceinline__ void store8(uint8_t* p, int n, const u32x2_el v) {
  if (n >= kVec) {
    *reinterpret_cast<u32x2_el*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (i < n) p[i] = static_cast<uint8_t>(v[i >> 2] >> (8 * (i & 3)));
  }
}

// ---------------------------------------------------------------- sums over lanes
// A lane permutation within rows of 16 that the compiler can fold into the instruction using it.
template <int kCtrl>
__device__ __forceinline__ uint32_t dppu(uint32_t v) {
  return static_cast<uint32_t>(
      __builtin_amdgcn_mov_dpp(static_cast<int>(v), kCtrl, 0xF, 0xF, true));
}
template <int kCtrl>
__device__ __forceinline__ float dppf(float v) {
  return __uint_as_float(dppu<kCtrl>(__float_as_uint(v)));
}
// Sum over a team of kLanes (16, 32 or 64) consecutive lanes, the same bits in each of them: the
// partners of every step hold mirrored operands of one addition.
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
  v += dppf<0xB1>(v);   // quad_perm [1,0,3,2]
  v += dppf<0x4E>(v);   // quad_perm [2,3,0,1]
  v += dppf<0x141>(v);  // row_half_mirror
  v += dppf<0x140>(v);  // row_mirror
  if constexpr (kLanes >= 32) {
    const uint32_t u = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  if constexpr (kLanes >= 64) {
    const uint32_t u = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  return v;
}

// ---------------------------------------------------------------- 8-bit groups
// Magnitudes as bit patterns: for non-negative floats the order of the patterns is the order of
// the values, with infinity and NaN above every finite value.
__device__ __forceinline__ uint32_t mag(float x) { return __float_as_uint(x) & 0x7fffffffu; }
// Zero for infinities and NaN. For rare paths: the empty statement keeps the compiler from working
// the magnitudes out ahead of the branch that leads here.
__device__ __forceinline__ uint32_t finite_mag(float x) {
  asm volatile("" : "+v"(x));
  const uint32_t m = mag(x);
  return m < kInfBits ? m : 0u;
}
// Largest magnitude of eight values as bits. Of stored values (kRaw) over the bit patterns, where
// an infinity or NaN tops everything and so is noticed. Of computed values, whose NaN are quiet,
// by three-operand maxima with free absolute values, which pass NaN over and notice infinities.
template <bool kRaw>
__device__ __forceinline__ uint32_t max8(const float* f) {
  if constexpr (kRaw) {
    uint32_t m = mag(f[0]);
#pragma unroll
    for (int i = 1; i < kVec; ++i) m = umax32(m, mag(f[i]));
    return m;
  } else {
    float m = __builtin_fabsf(f[0]);
#pragma unroll
    for (int i = 1; i < kVec; ++i) m = fmaxf(m, __builtin_fabsf(f[i]));
    return __float_as_uint(m) & 0x7fffffffu;
  }
}
__device__ __forceinline__ uint32_t finite_max8(const float* f) {
  uint32_t m = finite_mag(f[0]);
#pragma unroll
  for (int i = 1; i < kVec; ++i) m = umax32(m, finite_mag(f[i]));
  return m;
}
// Over the 16 lanes of a DPP row: neighbours, pairs, halves of 8, the row.
__device__ __forceinline__ uint32_t row16_umax(uint32_t u) {
  u = umax32(u, dppu<0xB1>(u));
  u = umax32(u, dppu<0x4E>(u));
  u = umax32(u, dppu<0x141>(u));
  return umax32(u, dppu<0x140>(u));
}

// Scale of a checkpoint group from its largest finite magnitude (bits): the quantisers' rule,
// with a nonzero amax below 2^-119 raised to it, so that 448/amax stays finite for any input.
__device__ __forceinline__ void ckpt_scale(uint32_t amax, bool pow2, float& s, float& r) {
  constexpr uint32_t kLeast = (127u - 119u) << 23;
  const float a = __uint_as_float(umax32(amax, kLeast));
  if (pow2) {
    group_scale_pow2(a, s, r);
  } else {
    s = a / 448.0f;
    r = 448.0f / a;
  }
  if (amax == 0) s = r = 1.0f;
}

// Codes of four scaled values. A finite element of its own group is at most 448 (1 + 2^-22) in
// magnitude, which rounds to 448, so nothing needs clamping; an infinity and a NaN convert to the
// NaN code with their sign.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true));
}
__device__ __forceinline__ u32x2_el encode8(const float* f, float r) {
  u32x2_el v;
  v[0] = codes4(f[0] * r, f[1] * r, f[2] * r, f[3] * r);
  v[1] = codes4(f[4] * r, f[5] * r, f[6] * r, f[7] * r);
  return v;
}

// kN row groups at once, each spread over the 16 lanes of a DPP row: lane k of the row works out
// group k's scale and stores it, and the others take its reciprocal by a row broadcast, so the
// two divisions run once for all the groups instead of once for each. All 64 lanes take part.
template <int kN>
struct RowGroups {
  float r[kN];   // reciprocal scales
  float s;       // in lane k of the row (k < kN): group k's scale
};
template <int kN, int kK = 0>
__device__ __forceinline__ void take_scales(float r, float* out) {
  if constexpr (kK < kN) {
    out[kK] = dppf<0x150 + kK>(r);  // row_newbcast: lane kK of each 16-lane row
    take_scales<kN, kK + 1>(r, out);
  }
}
template <bool kRaw, int kN>
__device__ __forceinline__ RowGroups<kN> row_groups(const float (*f)[kVec], bool pow2) {
  static_assert(kN <= 16, "one lane per group");
  const int l16 = threadIdx.x & 15;
  RowGroups<kN> g;
  uint32_t mine = 0, all = 0;
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const uint32_t m = row16_umax(max8<kRaw>(f[k]));
    all = umax32(all, m);
    mine = l16 == k ? m : mine;
  }
  if (all >= kInfBits) {  // rare: an infinity or NaN, which the scale leaves out
#pragma unroll 1
    for (int k = 0; k < kN; ++k) {
      float v[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = f[0][i];
#pragma unroll
      for (int j = 1; j < kN; ++j)
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = j == k ? f[j][i] : v[i];
      const uint32_t m = row16_umax(finite_max8(v));
      mine = l16 == k ? m : mine;
    }
  }
  float r;
  ckpt_scale(mine, pow2, g.s, r);
  take_scales<kN>(r, g.r);
  return g;
}

}  // namespace puro
