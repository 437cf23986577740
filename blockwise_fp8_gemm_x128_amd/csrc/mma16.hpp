// 16-bit matrix products (bf16 or fp16, fp32 sums) for gfx950: the tile loop that the output head's
// cross entropy and the orthogonalisation of the optimizer's momentum share.
//
//     C[i][j] = sum_k A(i, k) B(j, k)
//
// Either operand lies row-major with the reduction contiguous, A[i][k], or reduction-major, A[k][i]
// (kTransA, kTransB), so that no operand is ever copied into another orientation: a gradient's
// products read the same matrix once along each of its sides.
//
// Decomposition. A block owns a BM x BN tile of C and WAVES_M x WAVES_N waves, each with a WM x 64
// sub-tile of 16x16 matrix-core tiles (16x16x32 instructions). The reduction runs in chunks of 64
// (128 bytes of a row) through two LDS stages: while one chunk is multiplied out of one stage, the
// next streams into the other with 16-byte loads that write LDS directly. Tiles too few to share a CU
// take a ring of three or four stages instead (multiply_ring).
//
// Measured with 256x256 tiles: 1.32 to 1.40 PFLOP/s at 8192 x 2048 x 8192, matrix cores busy 71 to 75 %
// of the time at 1.8 GHz, where a library product of that size runs them 88 % at 1.5: the power limit
// binds both. Fragments read ahead across the barrier, or four waves of 128x128, gained at most 4 % and
// only with both operands row-major.
//
// LDS layout. A row-major operand keeps its rows of 128 bytes; a reduction-major one is cut into
// slabs of 64 columns, each 64 rows (of the reduction) of 128 bytes. The eight 16-byte pieces of a row are
// XOR-permuted, so that neither the 16-byte fragment reads nor the transposing 8-byte reads of
// reduction-major slabs meet on a bank: rows of a fragment differ in the bits that swz_rows takes,
// the rows of a transposing read in those of swz_slab16.
//
// The order of k inside a chunk is free as long as both operands share it: lane (G, r) of the
// instruction e (of two) holds k = 16 G + 8 e .. + 7 of row (column) r.
#pragma once
#include "common.hpp"

namespace puro {
namespace mma16 {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) v4i lds_v4i;
typedef __attribute__((address_space(3))) v2i lds_v2i;
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(3))) v4f lds_v4f;
typedef __attribute__((address_space(3))) float lds_f32;
typedef __attribute__((address_space(3))) int lds_i32;
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kChunk = 64;             // reduction elements of a chunk
constexpr int kRowBytes = 2 * kChunk;  // bytes of a staged row

template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, bool kTransA_, bool kTransB_, bool kHalf_,
          int kStages_ = 2>
struct Tile {
  static constexpr int BM = BM_, BN = BN_;
  static constexpr int WAVES_M = WAVES_M_, WAVES_N = WAVES_N_;
  static constexpr bool kTransA = kTransA_, kTransB = kTransB_;
  static constexpr bool kHalf = kHalf_;  // fp16 operands, else bf16
  static constexpr int kWaves = WAVES_M * WAVES_N;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;
  static constexpr int MI = WM / 16, NJ = WN / 16;
  static constexpr int kBOff = BM * kRowBytes;
  static constexpr int kStageBytes = (BM + BN) * kRowBytes;
  static constexpr int kStages = kStages_;
  // the two LDS arrays of a block: a stage each, or the whole ring and nothing
  static constexpr bool kRing = kStages > 2;
  static constexpr int kLds0 = kRing ? kStages * kStageBytes : kStageBytes;
  static constexpr int kLds1 = kRing ? 16 : kStageBytes;
  static_assert(WN == 64 && WM % 16 == 0 && BM % 64 == 0 && BN % 64 == 0, "tile shape");
};

__device__ __forceinline__ int swz_rows(int row) { return ((row & 3) << 1) | ((row >> 3) & 1); }
__device__ __forceinline__ int swz_slab16(int row) { return (row & 2) | ((row >> 2) & 4); }

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
}

typedef __amdgpu_buffer_rsrc_t rsrc_t;
// Offsets from here on are outside every resource: a load there reads zeros.
constexpr uint32_t kOutside = 0x80000000u;

// A resource of `bytes` (none or fewer: empty, every load reads zeros), cut at kOutside.
__device__ __forceinline__ rsrc_t make_rsrc(const void* base, int64_t bytes) {
  const int n = bytes > int64_t(0x7fffffff) ? 0x7fffffff : bytes < 0 ? 0 : static_cast<int>(bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, n, 0x00020000);
}

// One matrix operand: `rows` x `cols` elements of 2 bytes with a row stride of ld elements. The
// base is 16-byte aligned and ld a multiple of 8; cols may end inside a chunk of the reduction at a
// multiple of 8 (what lies behind is read as zero).
struct Operand {
  const uint8_t* p;
  int64_t rows, cols, ld;
};
// Largest row stride in elements: the offsets inside a tile (256 rows) stay below 2^30 bytes.
constexpr int64_t kMaxLd = int64_t(1) << 21;

// One operand's share of the loads: BX rows (columns) of C from x0 on, by kIssuers waves. Load n of
// issuing wave w fills staged rows [8q, 8q + 8), q = w + kIssuers n; lane l takes row l / 8 of them
// and slot l % 8, which holds logical piece (l % 8) ^ swizzle(row).
template <bool kTrans, int BX, int kIssuers>
struct Stager {
  static constexpr int kLoads = BX / 8 / kIssuers;
  static_assert(BX / 8 % kIssuers == 0 && kIssuers % 4 == 0, "even split, swizzle fixed per wave");
  rsrc_t r;
  uint32_t voff, voff_tail;
  const uint8_t* p;
  int64_t ld2, rows, x_bytes;
  int w;

  __device__ __forceinline__ void init(const Operand& o, int64_t x0, int w_, int lane) {
    const int r8 = lane >> 3, p8 = lane & 7;
    w = w_;
    ld2 = 2 * o.ld;
    if constexpr (kTrans) {
      p = o.p + 2 * x0;
      rows = o.rows;
      x_bytes = 2 * (o.cols - x0);
      voff = static_cast<uint32_t>(r8 * ld2) + 16 * (p8 ^ swz_slab16(8 * w + r8));
    } else {
      const int piece = p8 ^ swz_rows(8 * w + r8);
      r = make_rsrc(o.p + x0 * ld2, (o.rows - x0 - 1) * ld2 + 2 * o.cols);
      voff = static_cast<uint32_t>(r8 * ld2) + 16 * piece;
      // in the last chunk, the pieces behind the operand's columns
      const int64_t last = (o.cols - 1) / kChunk * kChunk;
      voff_tail = last + 8 * piece < o.cols ? voff : kOutside;
    }
  }

  __device__ __forceinline__ void issue(lds_u8* dst, int64_t c, bool last) const {
    if constexpr (kTrans) {
      const rsrc_t rc = make_rsrc(p + c * kChunk * ld2, (rows - c * kChunk - 1) * ld2 + x_bytes);
#pragma unroll
      for (int n = 0; n < kLoads; ++n) {
        const int q = w + kIssuers * n;
        const uint32_t off = static_cast<uint32_t>((q & 7) * 8 * ld2) + (q >> 3) * kRowBytes;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rc, (lds_void*)(dst + 8 * q * kRowBytes), 16,
                                                 static_cast<int>(voff + off), 0, 0, 0);
      }
    } else {
      uint32_t v = (last ? voff_tail : voff) + static_cast<uint32_t>(c * kRowBytes);
      asm volatile("" : "+v"(v));  // one register plus uniform offsets, not one register per load
#pragma unroll
      for (int n = 0; n < kLoads; ++n) {
        const int q = w + kIssuers * n;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            r, (lds_void*)(dst + 8 * q * kRowBytes), 16,
            static_cast<int>(v + static_cast<uint32_t>(8 * q * ld2)), 0, 0, 0);
      }
    }
  }
};

// The ring's loads (multiply, kStages > 2) are inline assembly: the compiler, which does not see that they
// write LDS, adds no waits of its own before reads of other stages. They have no output registers.
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v4u rsrc_words(const void* base, int64_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint32_t n = bytes > int64_t(0x7fffffff) ? 0x7fffffffu
                     : bytes < 0                 ? 0u
                                                 : static_cast<uint32_t>(bytes);
  v4u r;
  r[0] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b));
  r[1] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32) & 0xffffu);
  r[2] = __builtin_amdgcn_readfirstlane(n);
  r[3] = 0x00020000u;
  return r;
}
// (m0, the LDS address, may be read one wait state after it is written at the earliest)
__device__ __forceinline__ void load_lds16(v4u r, uint32_t voff, uint32_t lds) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"{m0}"(lds), "v"(voff), "s"(r)
               : "memory");
}
template <int n>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(n) : "memory");
}

template <bool kTrans, int BX, int kIssuers>
struct RingStager : Stager<kTrans, BX, kIssuers> {
  using Base = Stager<kTrans, BX, kIssuers>;
  v4u words;
  __device__ __forceinline__ void init(const Operand& o, int64_t x0, int w_, int lane) {
    Base::init(o, x0, w_, lane);
    if constexpr (!kTrans)
      words = rsrc_words(o.p + x0 * Base::ld2, (o.rows - x0 - 1) * Base::ld2 + 2 * o.cols);
  }
  // The chunk to send next, c of nk, and its stage; from nk on zeros are written, so that every wave
  // always has the same number of loads under way.
  v4u aimed;
  uint32_t v, dst;
  __device__ __forceinline__ void aim(uint32_t dst_, int64_t c, int64_t nk) {
    dst = dst_;
    if constexpr (kTrans) {
      aimed = rsrc_words(Base::p + c * kChunk * Base::ld2,
                         c < nk ? (Base::rows - c * kChunk - 1) * Base::ld2 + Base::x_bytes : 0);
      v = Base::voff;
    } else {
      aimed = words;
      v = c < nk ? (c == nk - 1 ? Base::voff_tail : Base::voff) +
                       static_cast<uint32_t>(c * kRowBytes)
                 : kOutside;
      asm volatile("" : "+v"(v));
    }
  }
  // load n of it
  __device__ __forceinline__ void send(int n) const {
    const int q = Base::w + kIssuers * n;
    const uint32_t off =
        kTrans ? static_cast<uint32_t>((q & 7) * 8 * Base::ld2) + (q >> 3) * kRowBytes
               : static_cast<uint32_t>(8 * q * Base::ld2);
    load_lds16(aimed, v + off, dst + 8 * q * kRowBytes);
  }
};

// Lane offsets of a wave's fragment reads of one operand, whose rows (columns) begin at x of the tile.
template <bool kTrans>
struct Frag {
  int o[kTrans ? 4 : 2];
  __device__ __forceinline__ void init(int base, int x, int lane) {
    const int G = lane >> 4, r = lane & 15;
    if constexpr (kTrans) {
      const int row = 16 * G + (r >> 2);
      for (int b = 0; b < 4; ++b)  // 16 columns b of the slab from x on (x is 0 or 32 of its 64)
        o[b] = base + (x >> 6) * 64 * kRowBytes + row * kRowBytes + 8 * (r & 1) +
               (((2 * ((b + (x >> 4)) & 3) + ((r & 3) >> 1)) ^ swz_slab16(row)) << 4);
    } else {
      for (int e = 0; e < 2; ++e)
        o[e] = base + (x + r) * kRowBytes + (((2 * G + e) ^ swz_rows(r)) << 4);
    }
  }
  // the 16 rows (columns) from 16 n on, instruction e of the chunk
  template <int n, int e>
  __device__ __forceinline__ v4i read(const lds_u8* stage) const {
    if constexpr (kTrans) {
      constexpr int kAt = (n >> 2) * 64 * kRowBytes + 8 * e * kRowBytes;
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(stage + o[n & 3] + kAt));
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_v4s*)(stage + o[n & 3] + kAt + 4 * kRowBytes));
      return __builtin_bit_cast(v4i, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      return *reinterpret_cast<const lds_v4i*>(stage + o[e] + 16 * n * kRowBytes);
    }
  }
};

template <bool kHalf>
__device__ __forceinline__ v4f mfma(v4i a, v4i b, v4f c) {
  if constexpr (kHalf)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a),
                                                  __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                   __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

template <class C>
struct Fragments {
  Frag<C::kTransA> fa;
  Frag<C::kTransB> fb;
  v4i b[C::NJ][2];
  v4i a[2][2];  // the row block at hand and the next
};

template <class C, int nj>
__device__ __forceinline__ void load_b(const lds_u8* stage, Fragments<C>& f) {
  if constexpr (nj < C::NJ) {
    f.b[nj][0] = f.fb.template read<nj, 0>(stage);
    f.b[nj][1] = f.fb.template read<nj, 1>(stage);
    __builtin_amdgcn_sched_barrier(0);
    load_b<C, nj + 1>(stage, f);
  }
}

// Step k = mi * NJ + nj of a chunk; the next row block's fragment is fetched at the start of each
// row block. `mid` runs before the second row block (the second half of the next chunk's loads).
template <class C, int k, class Mid>
__device__ __forceinline__ void chunk_step(const lds_u8* stage, Fragments<C>& f,
                                           v4f (&acc)[C::MI][C::NJ], const Mid& mid) {
  if constexpr (k < C::MI * C::NJ) {
    constexpr int mi = k / C::NJ, nj = k % C::NJ;
    if constexpr (nj == 0 && mi + 1 < C::MI) {
      f.a[(mi + 1) & 1][0] = f.fa.template read<mi + 1, 0>(stage);
      f.a[(mi + 1) & 1][1] = f.fa.template read<mi + 1, 1>(stage);
    }
    if constexpr (k == C::NJ || (C::MI == 1 && k == 0)) mid();
    acc[mi][nj] = mfma<C::kHalf>(f.b[nj][0], f.a[mi & 1][0], acc[mi][nj]);
    acc[mi][nj] = mfma<C::kHalf>(f.b[nj][1], f.a[mi & 1][1], acc[mi][nj]);
    __builtin_amdgcn_sched_barrier(0);
    chunk_step<C, k + 1>(stage, f, acc, mid);
  }
}

// The fragments of a half chunk: one matrix instruction per 16x16 tile.
template <class C>
struct HalfChunk {
  v4i a[C::MI], b[C::NJ];
};

// Step k of a half chunk's MI NJ: a fragment of the next half (e) is read from its stage, `send` may send
// loads, and one instruction runs on this half's fragments.
template <class C, int k, int e, class Send>
__device__ __forceinline__ void half_step(const Fragments<C>& f, const lds_u8* stage,
                                          HalfChunk<C>& next, const HalfChunk<C>& now,
                                          v4f (&acc)[C::MI][C::NJ], const Send& send) {
  if constexpr (k < C::MI * C::NJ) {
    static_assert(C::MI + C::NJ <= C::MI * C::NJ, "a fragment a step");
    // in the order of their use: the first row block, all columns, the other row blocks
    if constexpr (k == 0)
      next.a[0] = f.fa.template read<0, e>(stage);
    else if constexpr (k <= C::NJ)
      next.b[k - 1] = f.fb.template read<k - 1, e>(stage);
    else if constexpr (k < C::MI + C::NJ)
      next.a[k - C::NJ] = f.fa.template read<k - C::NJ, e>(stage);
    send(k);
    constexpr int mi = k / C::NJ, nj = k % C::NJ;
    acc[mi][nj] = mfma<C::kHalf>(now.b[nj], now.a[mi], acc[mi][nj]);
    __builtin_amdgcn_sched_barrier(0);
    half_step<C, k + 1, e>(f, stage, next, now, acc, send);
  }
}

// the first half of the first chunk
template <class C, int k>
__device__ __forceinline__ void read_half(const Fragments<C>& f, const lds_u8* stage,
                                          HalfChunk<C>& h) {
  if constexpr (k < C::MI) h.a[k] = f.fa.template read<k, 0>(stage);
  if constexpr (k < C::NJ) h.b[k] = f.fb.template read<k, 0>(stage);
  if constexpr (k + 1 < C::MI || k + 1 < C::NJ) read_half<C, k + 1>(f, stage, h);
}

// multiply below with a ring of kStages stages, chunk c in stage c % kStages, for tiles too few to share
// a CU: their loads come from far (another XCD wrote them) and a SIMD has one wave, so nothing else
// hides a wait. A half chunk's fragments are read while the half before it is multiplied, across
// the barrier too; behind the barrier in a chunk's middle every wave has read the chunk and its
// stage is sent the one kStages later, a load every few instructions.
template <class C, bool kMore>
__device__ __forceinline__ void multiply_ring(const Operand& A, const Operand& B, int64_t i0,
                                              int64_t j0, int64_t c0, int64_t c1, int64_t nk,
                                              lds_u8* ring, v4f (&acc)[C::MI][C::NJ]) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  RingStager<C::kTransA, C::BM, C::kWaves> sa;
  RingStager<C::kTransB, C::BN, C::kWaves> sb;
  sa.init(A, i0, wave, lane);
  sb.init(B, j0, wave, lane);
  Fragments<C> f;
  f.fa.init(0, wm * C::WM, lane);
  f.fb.init(C::kBOff, wn * C::WN, lane);
  if constexpr (!kMore) {
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi)
#pragma unroll
      for (int nj = 0; nj < C::NJ; ++nj) acc[mi][nj] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }
  constexpr int kSteps = C::MI * C::NJ;
  constexpr int kLoads = decltype(sa)::kLoads + decltype(sb)::kLoads;
  const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(ring));
  auto aim = [&](int64_t c, int stage) {
    const int64_t end = c < c1 ? nk : 0;
    sa.aim(base + stage * C::kStageBytes, c, end);
    sb.aim(base + stage * C::kStageBytes + C::kBOff, c, end);
  };
  auto send = [&](int n) {
    if (n < decltype(sa)::kLoads)
      sa.send(n);
    else
      sb.send(n - decltype(sa)::kLoads);
  };
#pragma unroll
  for (int k = 0; k < C::kStages; ++k) {
    aim(c0 + k, k);
#pragma unroll
    for (int n = 0; n < kLoads; ++n) send(n);
  }
  // The next chunk has landed when at most the later chunks' loads are under way, here and, behind the
  // barrier, in every wave.
  wait_loads<(C::kStages - 1) * kLoads>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  HalfChunk<C> first, second;
  read_half<C, 0>(f, ring, first);
  int stage = 0;
  for (int64_t c = c0; c < c1; ++c) {
    half_step<C, 0, 1>(f, ring + stage * C::kStageBytes, second, first, acc, [](int) {});
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this wave has read the chunk
    wait_loads<(C::kStages - 2) * kLoads>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    aim(c + C::kStages, stage);
    stage = stage + 1 == C::kStages ? 0 : stage + 1;
    half_step<C, 0, 0>(f, ring + stage * C::kStageBytes, first, second, acc, [&](int k) {
#pragma unroll
      for (int n = 0; n < kLoads; ++n)
        if (n * kSteps / kLoads == k) send(n);
    });
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  wait_loads<0>();
}

// The products of one tile over chunks [c0, c1) of the reduction, which has `nk` chunks in all.
// Each instruction takes the B fragment as its row operand, so lane (G, r) receives row r, columns
// 4 G .. 4 G + 3 of every 16x16 tile. On return other waves may still read the stages. kMore adds to
// what acc holds instead of starting from zero.
template <class C, bool kMore = false>
__device__ __forceinline__ void multiply(const Operand& A, const Operand& B, int64_t i0,
                                         int64_t j0, int64_t c0, int64_t c1, int64_t nk,
                                         lds_u8* s0, lds_u8* s1, v4f (&acc)[C::MI][C::NJ]) {
  if constexpr (C::kRing) {
    multiply_ring<C, kMore>(A, B, i0, j0, c0, c1, nk, s0, acc);
    return;
  }
  // In 8-wave tiles half of the waves load a chunk, the halves alternating: the two waves of a SIMD
  // are in different halves, so one of them keeps the matrix core busy while the other feeds the
  // memory pipeline.
  constexpr bool kPingPong = C::kWaves == 8;
  constexpr int kIssuers = kPingPong ? 4 : C::kWaves;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  Stager<C::kTransA, C::BM, kIssuers> sa;
  Stager<C::kTransB, C::BN, kIssuers> sb;
  sa.init(A, i0, wave % kIssuers, lane);
  sb.init(B, j0, wave % kIssuers, lane);
  Fragments<C> f;
  f.fa.init(0, wm * C::WM, lane);
  f.fb.init(C::kBOff, wn * C::WN, lane);
  if constexpr (!kMore) {
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi)
#pragma unroll
      for (int nj = 0; nj < C::NJ; ++nj) acc[mi][nj] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }

  auto issue_a = [&](lds_u8* st, int64_t c) {
    if (!kPingPong || wave / kIssuers == static_cast<int>(c & 1)) sa.issue(st, c, c == nk - 1);
  };
  auto issue_b = [&](lds_u8* st, int64_t c) {
    if (!kPingPong || wave / kIssuers == static_cast<int>(c & 1))
      sb.issue(st + C::kBOff, c, c == nk - 1);
  };
  auto half = [&](lds_u8* cur, lds_u8* nxt, int64_t c) {
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (c + 1 < c1) issue_a(nxt, c + 1);
    f.a[0][0] = f.fa.template read<0, 0>(cur);
    f.a[0][1] = f.fa.template read<0, 1>(cur);
    __builtin_amdgcn_sched_barrier(0);
    load_b<C, 0>(cur, f);
    chunk_step<C, 0>(cur, f, acc, [&]() {
      if (c + 1 < c1) issue_b(nxt, c + 1);
    });
    // Pinned at the chunk's end: the compiler otherwise moves products past the next barrier and
    // keeps their fragments live.
#pragma unroll
    for (int mi = 0; mi < C::MI; ++mi)
#pragma unroll
      for (int nj = 0; nj < C::NJ; ++nj) asm volatile("" : "+v"(acc[mi][nj]));
  };
  if (c0 < c1) {
    issue_a(s0, c0);
    issue_b(s0, c0);
  }
  int64_t c = c0;
  for (; c + 1 < c1; c += 2) {
    half(s0, s1, c);
    half(s1, s0, c + 1);
  }
  if (c < c1) half(s0, s1, c);
}

// Tile indices of block b of a product with ti x tj tiles: blocks are dealt round-robin to the 8
// XCDs, so ids are first regrouped so that neighbouring tiles share an XCD's cache, then walked in
// bands of `band` tile rows, column by column.
__device__ __forceinline__ int64_t regroup(int64_t b, int64_t n) {
  return (n & 7) == 0 ? (b & 7) * (n >> 3) + (b >> 3) : b;
}
__device__ __forceinline__ void tile_at(int64_t b, int64_t ti, int64_t tj, int64_t band,
                                        int64_t& i, int64_t& j) {
  const int64_t s = b / (band * tj);
  const int64_t rows = band < ti - s * band ? band : ti - s * band;
  const int64_t local = b - s * band * tj;
  i = s * band + local % rows;
  j = local / rows;
}

// Reads of another matrix at a wave's results (rows from r0, columns from q0): the four elements that a
// lane needs beside tile (mi, nj), through a resource, so that a read behind the last row gives zeros
// and no branch keeps the compiler from sending many at once (with branches, each waited for its own).
// Columns behind the row's end read the next row: results there are not stored. T: 2 or 4 bytes.
template <int kBytes>
struct Beside {
  rsrc_t r;
  uint32_t lane_off, ld;
  // rows x ld elements, at least up to the last row's `cols`
  __device__ __forceinline__ Beside(const void* p, int64_t rows, int64_t cols, int64_t ld_, int64_t r0,
                                    int64_t q0, int lane)
      : ld(static_cast<uint32_t>(ld_) * kBytes) {
    const int64_t at = uniform64(r0 * ld_ + q0);
    r = make_rsrc(static_cast<const uint8_t*>(p) + at * kBytes,
                  (uniform64((rows - 1) * ld_ + cols) - at) * kBytes);
    lane_off = (lane & 15) * ld + 4 * (lane >> 4) * kBytes;
  }
  __device__ __forceinline__ uint32_t off(int mi, int nj) const {
    return lane_off + 16 * mi * ld + 16 * nj * kBytes;
  }
  __device__ __forceinline__ v2i half4(int mi, int nj) const {
    static_assert(kBytes == 2, "16-bit elements");
    return __builtin_bit_cast(
        v2i, __builtin_amdgcn_raw_buffer_load_b64(r, static_cast<int>(off(mi, nj)), 0, 0));
  }
  __device__ __forceinline__ v4f float4(int mi, int nj) const {
    static_assert(kBytes == 4, "32-bit elements");
    return __builtin_bit_cast(
        v4f, __builtin_amdgcn_raw_buffer_load_b128(r, static_cast<int>(off(mi, nj)), 0, 0));
  }
};

// A wave's WM x 64 block as 16-bit values in its own LDS region, rows of 128 bytes with their
// 16-byte units XOR-permuted: pack(mi, nj, value) gives the two dwords of four adjacent columns. The
// region is then read by whole rows, or transposed.
template <class C>
struct Region {
  static constexpr int kBytes = C::WM * kRowBytes;
  lds_u8* p;
  int lane;
  // from the block's two LDS arrays
  __device__ __forceinline__ Region(lds_u8* s0, lds_u8* s1, int wave, int lane_) : lane(lane_) {
    constexpr int kFirst = C::kLds0 / kBytes;  // regions that fit the first
    static_assert(kFirst >= C::kWaves || kFirst + C::kLds1 / kBytes >= C::kWaves, "regions fit");
    p = wave < kFirst ? s0 + wave * kBytes : s1 + (wave - kFirst) * kBytes;
  }
  // Unit swizzle: the writes of 16 rows at one unit meet on no bank as row bits 1-3 enter, the
  // transposing reads (4 rows x 2 blocks of 8 rows at two units) as bits 1 and 3 enter above bit 0.
  static __device__ __forceinline__ int swz(int row) {
    return (row & 2) | ((row >> 1) & 4) | ((row >> 2) & 1);
  }
  __device__ __forceinline__ void put(int mi, int nj, v2i v) const {
    const int row = 16 * mi + (lane & 15), unit = 2 * nj + (lane >> 5);
    *reinterpret_cast<lds_v2i*>(p + row * kRowBytes + 16 * (unit ^ swz(row)) +
                                8 * ((lane >> 4) & 1)) = v;
  }
  // other lanes' writes are read next: wait for them
  __device__ __forceinline__ void settle() const {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
  // 8 columns from 8 (lane % 8) on, of row 8 n + lane / 8
  __device__ __forceinline__ v4i row8(int n) const {
    const int row = 8 * n + (lane >> 3);
    return *reinterpret_cast<const lds_v4i*>(p + row * kRowBytes + 16 * ((lane & 7) ^ swz(row)));
  }
  // 8 rows from 32 n + 8 (lane / 16) on, of column 16 b + lane % 16
  __device__ __forceinline__ v4i col8(int n, int b) const {
    const int G = lane >> 4, r = lane & 15;
    const int row = 32 * n + 8 * G + (r >> 2);
    const int unit = 2 * b + ((r & 3) >> 1);
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(
        p + row * kRowBytes + 16 * (unit ^ swz(row)) + 8 * (r & 1)));
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(
        p + (row + 4) * kRowBytes + 16 * (unit ^ swz(row + 4)) + 8 * (r & 1)));
    return __builtin_bit_cast(v4i, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const half2_t v = {static_cast<_Float16>(lo), static_cast<_Float16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}

}  // namespace mma16
}  // namespace puro
