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

// ---------------------------------------------------------------- tiles of rows and chunks
// Consecutive block indices go to the eight XCDs in turn. Where neighbouring tiles share memory
// lines (rows that do not start on one), `b`, of `n`, is renumbered so that each XCD gets a
// contiguous range of tiles and the shared lines meet in one L2.
__device__ __forceinline__ uint32_t xcd_range(uint32_t b, uint32_t n) {
  const uint32_t x = b & 7, rest = n & 7;
  return x * (n >> 3) + min(x, rest) + (b >> 3);
}

// The elementwise kernels' block of 256 threads: 16 lane groups of 16, each on one 128-column chunk
// of a row; two chunks side by side, eight rows a pass, two passes with all their loads issued
// first. Measured on MI355X, all stores through the caches, against 1, 4, 8 and 16 chunks and 1 and
// 4 passes: 16384 x 2048 fp32 packed in 30.3 us (30.8 to 35.2), the activation of 8192 x 6144 in
// 63.9 us (67 to 74.5), 2047 x 4111 unpacked in 7.1 us (7 to 9.8). (Checkpoints' codes now go past
// the caches, which makes the first two 29.7 and 55.3 us.) Ranges per XCD: 4000 x 5003 packed in
// 12.4 us against 14.9, but 8192 x 6144 activated in 67.5 against 63.9, so only rows off the 128 B
// lines take them.
struct RowTile {
  static constexpr int kChunks = 2, kPasses = 2;
  static constexpr int kStep = 16 / kChunks;      // rows between passes
  static constexpr int kRows = kStep * kPasses;   // rows per block
  int64_t chunk, row0, col;
  __device__ __forceinline__ RowTile(int64_t cols, bool ranges) {
    const uint32_t across = static_cast<uint32_t>((cols + 128 * kChunks - 1) / (128 * kChunks));
    const uint32_t b = ranges ? xcd_range(blockIdx.x, gridDim.x) : blockIdx.x;
    const int g = threadIdx.x >> 4;
    chunk = int64_t(b % across) * kChunks + g % kChunks;
    row0 = int64_t(b / across) * kRows + g / kChunks;
    col = chunk * 128 + (threadIdx.x & 15) * 8;
  }
  __device__ __forceinline__ int64_t row(int p) const { return row0 + p * kStep; }
};
inline int64_t row_tiles(int64_t rows, int64_t cols) {
  return ceil_div(rows, RowTile::kRows) * ceil_div(cols, 128 * RowTile::kChunks);
}
// Rows of codes and of bf16 both start on 128 B lines.
__host__ __device__ inline bool off_lines(int64_t cols) { return cols % 128 != 0; }

// ---------------------------------------------------------------- vectors of eight
// Rows of any length start at any element, so vectors are only element-aligned; the global
// memory instructions take any address, and an aligned vector costs what it always did.
typedef uint32_t u32x4_el __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_el __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32_el __attribute__((aligned(1)));
typedef uint16_t u16_el __attribute__((aligned(1)));
typedef float f32x4_el __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ void widen8(const u32x4_el v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(v[i]);
    f[2 * i + 1] = bf16_hi(v[i]);
  }
}

// Where a lane's vector lies in a row of `cols`: columns col .. col + n - 1 exist. A vector that
// the row's end cuts short is read as the row's last eight columns and shifted into place (`shift`
// columns, 8 or more for a lane past the end, whose vector is zero), so that every lane issues the
// same loads and no branch stands between them; `cut`, the same in all lanes, says whether any
// lane of the kernel has such a vector. kShort: rows of fewer than eight columns, which go by
// element.
template <bool kShort>
struct Span {
  uint32_t col, at;
  int n, shift;
  bool cut;
  __device__ __forceinline__ Span() {}
  __device__ __forceinline__ Span(int64_t c, int64_t cols, bool any_cut) {
    cut = any_cut;
    col = static_cast<uint32_t>(c);
    n = static_cast<int>(min(cols - c, int64_t(kVec)));
    at = kShort ? 0 : static_cast<uint32_t>(min(c, cols - kVec));
    shift = static_cast<int>(min(c - int64_t(at), int64_t(kVec)));
  }
};

// A row's address, from a row index that is the same in all lanes of a wave (kUniform): kept in
// scalar registers (the empty statement hides its making, which the compiler would otherwise split
// into a vector base per tensor), so that each access is this plus one 32-bit offset per lane.
template <bool kUniform, typename T>
__device__ __forceinline__ T* row_ptr(T* base, int64_t offset) {
  uint64_t p = reinterpret_cast<uint64_t>(base + offset);
  if constexpr (kUniform) asm("" : "+s"(p));
  return reinterpret_cast<T*>(p);
}

// Raw vectors of eight bf16, E4M3 codes or fp32, and their shift.
struct Bf16x8 {
  u32x4_el v;
};
struct Fp8x8 {
  u32x2_el v;
};
struct F8 {
  float f[kVec];
};
// (The empty statement keeps the compiler from running these ahead of the branch to them.)
__device__ __forceinline__ void shift_in(Bf16x8& r, int shift) {
  asm volatile("" : "+v"(shift));
  if (shift == 0) return;
  uint64_t lo = r.v[0] | uint64_t(r.v[1]) << 32, hi = r.v[2] | uint64_t(r.v[3]) << 32;
  const int k = 16 * shift;
  if (k >= 64) {
    lo = k < 128 ? hi >> (k - 64) : 0;
    hi = 0;
  } else {
    lo = lo >> k | hi << (64 - k);
    hi >>= k;
  }
  r.v = u32x4_el{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32),
                 static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)};
}
__device__ __forceinline__ void shift_in(Fp8x8& r, int shift) {
  asm volatile("" : "+v"(shift));
  if (shift == 0) return;
  const uint64_t w = r.v[0] | uint64_t(r.v[1]) << 32;
  const uint64_t t = shift < kVec ? w >> (8 * shift) : 0;
  r.v = u32x2_el{static_cast<uint32_t>(t), static_cast<uint32_t>(t >> 32)};
}
__device__ __forceinline__ void shift_in(F8& r, int shift) {
  asm volatile("" : "+v"(shift));
  if (shift == 0) return;
#pragma unroll
  for (int s = kVec; s > 0; s >>= 1)
    if (shift & s) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) r.f[i] = i + s < kVec ? r.f[i + s] : 0.0f;
    }
}

// kOnce: nobody else reads the input soon, keep it out of the caches' way.
template <bool kOnce, bool kShort>
__device__ __forceinline__ void load(Bf16x8& r, const uint16_t* row, const Span<kShort>& s) {
  if constexpr (!kShort) {
    const u32x4_el* q = reinterpret_cast<const u32x4_el*>(row + s.at);
    r.v = kOnce ? __builtin_nontemporal_load(q) : *q;
  } else {
    r.v = u32x4_el{0, 0, 0, 0};
    for (int i = 0; i < s.n; ++i) {
      const uint32_t w = static_cast<uint32_t>(row[i]) << (16 * (i & 1));
#pragma unroll
      for (int k = 0; k < 4; ++k) r.v[k] |= (i >> 1) == k ? w : 0u;
    }
  }
}
template <bool kOnce, bool kShort>
__device__ __forceinline__ void load(Fp8x8& r, const uint8_t* row, const Span<kShort>& s) {
  if constexpr (!kShort) {
    const u32x2_el* q = reinterpret_cast<const u32x2_el*>(row + s.at);
    r.v = kOnce ? __builtin_nontemporal_load(q) : *q;
  } else {
    uint64_t w = 0;
    for (int i = 0; i < s.n; ++i) w |= uint64_t(row[i]) << (8 * i);
    r.v = u32x2_el{static_cast<uint32_t>(w), static_cast<uint32_t>(w >> 32)};
  }
}
template <bool kOnce, bool kShort>
__device__ __forceinline__ void load(F8& r, const float* row, const Span<kShort>& s) {
  if constexpr (!kShort) {
    const f32x4_el* q = reinterpret_cast<const f32x4_el*>(row + s.at);
    const f32x4_el a = kOnce ? __builtin_nontemporal_load(q) : q[0];
    const f32x4_el b = kOnce ? __builtin_nontemporal_load(q + 1) : q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.f[i] = a[i];
      r.f[4 + i] = b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) r.f[i] = i < s.n ? row[i] : 0.0f;
  }
}
// The raw vector of an element type.
template <typename T>
struct RawOf;
template <>
struct RawOf<uint16_t> {
  typedef Bf16x8 type;
};
template <>
struct RawOf<float> {
  typedef F8 type;
};

// A raw vector's columns in place, and its values: the first step that waits for the load.
template <typename Raw, bool kShort>
__device__ __forceinline__ void settle(Raw& r, const Span<kShort>& s) {
  if (s.cut) shift_in(r, s.shift);
}
template <bool kShort>
__device__ __forceinline__ void values(Bf16x8 r, const Span<kShort>& s, float* f) {
  settle(r, s);
  widen8(r.v, f);
}
template <bool kShort>
__device__ __forceinline__ void values(F8 r, const Span<kShort>& s, float* f) {
  settle(r, s);
#pragma unroll
  for (int i = 0; i < kVec; ++i) f[i] = r.f[i];
}

// Values that codes stand for, times their group's scale (one fp32 product each).
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

template <bool kShort>
__device__ __forceinline__ void values(Fp8x8 r, const Span<kShort>& s, float scale, float* f) {
  settle(r, s);
  decode8(r.v, scale, f);
}

// Stores of the n <= 8 elements of a vector that exist; a short vector goes in pieces of four, two
// and one element. kLater: nobody reads the output soon (a checkpoint waits for the backward pass,
// the residual stream for the end of the next block): it goes past the caches, which keep what the
// next kernel reads. Measured on MI355X over rotating buffers: the activation of 8192 x 6144 with
// its checkpoint 63.8 -> 55.4 us, the block norm of 4096 x 8192 72 -> 66.5 us forward (63.8 with
// two vectors per lane) and 78 -> 69 backward, of 8192 x 2048 33.3 -> 32.2 and 37.6 -> 38.2.
// (One function per type: a template parameter would lose the pointer's weak alignment.)
template <bool kLater>
__device__ __forceinline__ void put(u32x4_el* p, u32x4_el v) {
  if constexpr (kLater)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}
template <bool kLater>
__device__ __forceinline__ void put(u32x2_el* p, u32x2_el v) {
  if constexpr (kLater)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}
template <bool kLater>
__device__ __forceinline__ void put(f32x4_el* p, f32x4_el v) {
  if constexpr (kLater)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}
template <bool kLater = false>
__device__ __forceinline__ void store8(uint16_t* p, int n, const float* f) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  if (n >= kVec) {
    put<kLater>(reinterpret_cast<u32x4_el*>(p), u32x4_el{v[0], v[1], v[2], v[3]});
  } else if (n > 0) {
    if (n & 4) {
      *reinterpret_cast<u32x2_el*>(p) = u32x2_el{v[0], v[1]};
      p += 4, v[0] = v[2], v[1] = v[3];
    }
    if (n & 2) {
      *reinterpret_cast<u32_el*>(p) = v[0];
      p += 2, v[0] = v[1];
    }
    if (n & 1) *p = static_cast<uint16_t>(v[0]);
  }
}
template <bool kLater = false>
__device__ __forceinline__ void store8(float* p, int n, const float* f) {
  if (n >= kVec) {
    f32x4_el* q = reinterpret_cast<f32x4_el*>(p);
    put<kLater>(q, f32x4_el{f[0], f[1], f[2], f[3]});
    put<kLater>(q + 1, f32x4_el{f[4], f[5], f[6], f[7]});
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (i < n) p[i] = f[i];
  }
}
template <bool kLater = false>
__device__ __forceinline__ void store8(uint8_t* p, int n, const u32x2_el v) {
  if (n >= kVec) {
    put<kLater>(reinterpret_cast<u32x2_el*>(p), v);
  } else if (n > 0) {
    uint32_t w = v[0];
    if (n & 4) {
      *reinterpret_cast<u32_el*>(p) = w;
      p += 4, w = v[1];
    }
    if (n & 2) {
      *reinterpret_cast<u16_el*>(p) = static_cast<uint16_t>(w);
      p += 2, w >>= 16;
    }
    if (n & 1) *p = static_cast<uint8_t>(w);
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
// Of eight stored bf16, two at a time, as the bits of their fp32 values.
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                                __builtin_bit_cast(u16x2_t, b)));
}
__device__ __forceinline__ uint32_t max8(const Bf16x8& r) {
  constexpr uint32_t kMag = 0x7fff7fffu;
  const uint32_t m = pk_max(pk_max(r.v[0] & kMag, r.v[1] & kMag),
                            pk_max(r.v[2] & kMag, r.v[3] & kMag));
  return umax32(m << 16, m & 0xffff0000u);
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

// a/448 and 448/a correctly rounded, for 2^-119 <= a < infinity, in a third of two divisions'
// instructions: with c = fl(1/448), q = a c is within an ulp of a/448, its remainder a - 448 q is
// exact in one fused step, and q + remainder c rounds to the quotient. The other way the reciprocal
// of a/16 (so that neither it nor its argument leaves the normal range) is first refined by one
// Newton step. Both are the quotients' bits for every float in the range and a hardware reciprocal
// off by a unit in the last place either way; tests/test_amax_scale.py runs this function over all
// of them.
__device__ __forceinline__ void amax_scale(float a, float& s, float& r) {
  constexpr float c = 1.0f / 448.0f;
  const float q = a * c;
  s = __builtin_fmaf(__builtin_fmaf(-448.0f, q, a), c, q);
  const float b = a * 0.0625f;
  float y = __builtin_amdgcn_rcpf(b);
  y = __builtin_fmaf(__builtin_fmaf(-b, y, 1.0f), y, y);
  const float t = 28.0f * y;
  r = __builtin_fmaf(__builtin_fmaf(-b, t, 28.0f), y, t);
}

// Scale of a checkpoint group from its largest finite magnitude (bits): the quantisers' rule,
// with a nonzero amax below 2^-119 raised to it, so that 448/amax stays finite for any input.
__device__ __forceinline__ void ckpt_scale(uint32_t amax, bool pow2, float& s, float& r) {
  constexpr uint32_t kLeast = (127u - 119u) << 23;
  const float a = __uint_as_float(umax32(amax, kLeast));
  if (pow2)
    group_scale_pow2(a, s, r);
  else
    amax_scale(a, s, r);
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
  float s;       // in lane k of the row (k < kN): group k's scale (in every lane for kN = 1)
};
template <int kN, int kK = 0>
__device__ __forceinline__ void take_scales(float r, float* out) {
  if constexpr (kK < kN) {
    out[kK] = dppf<0x150 + kK>(r);  // row_newbcast: lane kK of each 16-lane row
    take_scales<kN, kK + 1>(r, out);
  }
}
// m: this lane's maxima of the kN groups; f: its values of them, for the rare path.
template <int kN>
__device__ __forceinline__ RowGroups<kN> row_groups(const uint32_t (&m)[kN],
                                                    const float (*f)[kVec], bool pow2) {
  static_assert(kN <= 16, "one lane per group");
  const int l16 = threadIdx.x & 15;
  RowGroups<kN> g;
  uint32_t mine = 0, all = 0;
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const uint32_t t = row16_umax(m[k]);
    all = umax32(all, t);
    mine = kN == 1 || l16 == k ? t : mine;
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
      const uint32_t t = row16_umax(finite_max8(v));
      mine = kN == 1 || l16 == k ? t : mine;
    }
  }
  float r;
  ckpt_scale(mine, pow2, g.s, r);
  if constexpr (kN == 1)
    g.r[0] = r;
  else
    take_scales<kN>(r, g.r);
  return g;
}
template <bool kRaw, int kN>
__device__ __forceinline__ RowGroups<kN> row_groups(const float (*f)[kVec], bool pow2) {
  uint32_t m[kN];
#pragma unroll
  for (int k = 0; k < kN; ++k) m[k] = max8<kRaw>(f[k]);
  return row_groups<kN>(m, f, pow2);
}

}  // namespace puro
