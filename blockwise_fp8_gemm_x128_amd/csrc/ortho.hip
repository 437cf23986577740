// The update direction of the optimizer's projected step: momentum of a weight gradient and its
// orthogonalisation by Newton-Schulz products, for several matrices of one shape in every launch.
//
//   m' = beta m + (1 - beta) g,  v = beta m' + (1 - beta) g (Nesterov) or m';   X = v / |v|_F
//   steps times:  A = X X',  X <- a X + (b A + c A A) X;     u = scale X
//
// with X' X and products from the right instead where the matrix is taller than wide (the same
// polynomial), so that A has the shorter side's size. A and its polynomial are symmetric: only
// tiles on and below the diagonal are multiplied, and each is stored twice.
//
// Precision. The products run on fp16 operands with fp32 sums. fp16 instead of bf16 (the same
// rate): every entry is at most a small constant, so no exponent range is needed, and fixed powers
// of two (kX, kA, kB) keep entries far below the largest in fp16's normal range. What a rounding
// of X adds in a direction of small singular values is amplified by a = 3.4 a step, as that
// direction itself is, so the early steps' roundings count most: all but the last two steps keep X
// as two halves, X = hi + lo, and form a X from both in fp32, while the product with X reads hi alone.
// It may: the polynomial is large only where X's large directions are, so hi's rounding comes out of
// it along those. Relative errors of u (2-norm, four spectra of 512 x 512 and 512 x 1536, all operands
// rounded as here): 0.7 to 1.2e-3, against 1.2 to 12e-3 with X in one half throughout, 10 to
// 57e-3 in bf16, and 1.7e-3 for the rounding of u itself to bf16.
#include <math.h>

#include "mma16.hpp"

namespace puro {
namespace {

using namespace mma16;

constexpr int kMax = PURO_NS_GROUP_MAX;
// X, A and the polynomial are held times these.
constexpr float kX = 4096.0f, kA = 16384.0f, kB = 2048.0f, kLo = 2048.0f;

struct Items {
  const float* g[kMax];
  const float* m[kMax];
  float* mo[kMax];
  uint16_t* u[kMax];
};

struct Momentum {
  bool on, nesterov;
  float beta, rest;  // rest = 1 - beta
};

__device__ __forceinline__ float direction(float g, float m_new, const Momentum& k) {
  return k.on ? (k.nesterov ? fmaf(k.beta, m_new, k.rest * g) : m_new) : g;
}

constexpr int kThreads = 256;
constexpr int kMaxParts = 512;

__device__ __forceinline__ double block_sum(double x, double* sh) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) x += __shfl_xor(x, off, 64);
  const int t = threadIdx.x;
  if ((t & 63) == 0) sh[t >> 6] = x;
  __syncthreads();
  return (sh[0] + sh[1]) + (sh[2] + sh[3]);
}

// Momentum, and the sum of squares of v by blocks (in fp64, in a fixed order). kVec: four elements
// at a time (all addresses of the group are 16-byte aligned and numel a multiple of 4).
template <bool kVec>
__global__ __launch_bounds__(kThreads) void ns_momentum_kernel(Items it, int64_t numel, Momentum k,
                                                               double* __restrict__ parts) {
  __shared__ double sh[kThreads / 64];
  const int n = blockIdx.y;
  const float* g = it.g[n];
  const float* m = it.m[n];
  float* mo = it.mo[n];
  double acc = 0.0;
  const int64_t step = int64_t(gridDim.x) * kThreads;
  if constexpr (kVec) {
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < numel / 4; i += step) {
      const v4f gg = reinterpret_cast<const v4f*>(g)[i];
      v4f v = gg;
      if (k.on) {
        v4f mm = reinterpret_cast<const v4f*>(m)[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          mm[e] = fmaf(k.beta, mm[e], k.rest * gg[e]);
          v[e] = direction(gg[e], mm[e], k);
        }
        reinterpret_cast<v4f*>(mo)[i] = mm;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) acc += double(v[e]) * v[e];
    }
  } else {
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < numel; i += step) {
      const float gg = g[i];
      float v = gg;
      if (k.on) {
        const float mm = fmaf(k.beta, m[i], k.rest * gg);
        v = direction(gg, mm, k);
        mo[i] = mm;
      }
      acc += double(v) * v;
    }
  }
  const double s = block_sum(acc, sh);
  if (threadIdx.x == 0) parts[int64_t(n) * gridDim.x + blockIdx.x] = s;
}

// X = v / |v| (zero where |v| is), times kX, in halves: hi [rows][ldx], zeros behind the columns, and
// lo, what hi leaves, times kLo.
template <bool kVec>
__global__ __launch_bounds__(kThreads) void ns_convert_kernel(Items it, int64_t rows, int64_t cols,
                                                              int64_t ldx, Momentum k,
                                                              const double* __restrict__ parts,
                                                              int count_parts,
                                                              _Float16* __restrict__ hi,
                                                              _Float16* __restrict__ lo,
                                                              int64_t hi_stride,
                                                              int64_t lo_stride) {
  __shared__ double sh[kThreads / 64];
  const int n = blockIdx.y;
  double acc = 0.0;
  for (int i = threadIdx.x; i < count_parts; i += kThreads)
    acc += parts[int64_t(n) * count_parts + i];
  const double ss = block_sum(acc, sh);
  const double f = ss == 0.0 ? 0.0 : double(kX) / sqrt(ss);
  const float* g = it.g[n];
  const float* m = it.mo[n];
  hi += n * hi_stride;
  lo += n * lo_stride;
  const int64_t groups = ldx / 4;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < rows * groups;
       i += int64_t(gridDim.x) * kThreads) {
    const int64_t row = i / groups, c = (i - row * groups) * 4;
    const int64_t at = row * cols + c;
    v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (kVec) {
      if (c < cols) {
        v = *reinterpret_cast<const v4f*>(g + at);
        if (k.on) {
          const v4f mm = *reinterpret_cast<const v4f*>(m + at);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = direction(v[e], mm[e], k);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < cols) v[e] = direction(g[at + e], k.on ? m[at + e] : 0.0f, k);
    }
    v2i h, l;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float x0 = static_cast<float>(v[2 * e] * f), x1 = static_cast<float>(v[2 * e + 1] * f);
      const _Float16 h0 = static_cast<_Float16>(x0), h1 = static_cast<_Float16>(x1);
      h[e] = static_cast<int>(__builtin_bit_cast(uint32_t, half2_t{h0, h1}));
      l[e] = static_cast<int>(pack_half2((x0 - float(h0)) * kLo, (x1 - float(h1)) * kLo));
    }
    *reinterpret_cast<v2i*>(hi + row * ldx + c) = h;
    *reinterpret_cast<v2i*>(lo + row * ldx + c) = l;
  }
}

// One matrix of a group per `stride` elements.
struct Batch {
  const _Float16* p;
  int64_t stride, rows, cols, ld;
  __device__ __forceinline__ Operand at(int64_t n) const {
    return {reinterpret_cast<const uint8_t*>(p + n * stride), rows, cols, ld};
  }
};

// Row and column of tile t of the lower triangle (t = row (row + 1) / 2 + column).
__device__ __forceinline__ void triangle_at(int t, int& i, int& j) {
  i = static_cast<int>((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
  while (i * (i + 1) / 2 > t) --i;
  while ((i + 1) * (i + 2) / 2 <= t) ++i;
  j = t - i * (i + 1) / 2;
}

// A symmetric product: A = X X' (kPoly false; kTrans: X' X), or the polynomial's matrix
// b A + c A A, with a on the diagonal where `diagonal` says so (kPoly, X = A).
template <class C, bool kPoly>
__global__ __launch_bounds__(C::kThreads) void ns_symmetric_kernel(Batch x, _Float16* out,
                                                                   int64_t out_stride, int64_t n,
                                                                   int64_t ld, int tiles,
                                                                   float a, float b, float c,
                                                                   bool diagonal) {
  __shared__ __attribute__((aligned(1024))) uint8_t s0[C::kStageBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t s1[C::kStageBytes];
  const int64_t id = regroup(blockIdx.x, gridDim.x);
  const int64_t item = id / tiles;
  int ti, tj;
  triangle_at(static_cast<int>(id - item * tiles), ti, tj);
  const int64_t i0 = uniform64(int64_t(ti) * C::BM), j0 = uniform64(int64_t(tj) * C::BN);
  const Operand X = x.at(uniform64(item));
  const int64_t nk = ((C::kTransA ? X.rows : X.cols) + kChunk - 1) / kChunk;
  v4f acc[C::MI][C::NJ];
  multiply<C>(X, X, i0, j0, 0, nk, nk, (lds_u8*)s0, (lds_u8*)s1, acc);
  __syncthreads();

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  const int G = lane >> 4, r = lane & 15;
  constexpr int kFirst = C::kStageBytes / Region<C>::kBytes;
  const Region<C> region(wave < kFirst ? (lds_u8*)s0 : (lds_u8*)s1,
                         wave < kFirst ? wave : wave - kFirst, lane);
  const int64_t r0 = i0 + wm * C::WM, q0 = j0 + wn * C::WN;
  const _Float16* src = reinterpret_cast<const _Float16*>(X.p);
  out += item * out_stride;
#pragma unroll
  for (int mi = 0; mi < C::MI; ++mi)
#pragma unroll
    for (int nj = 0; nj < C::NJ; ++nj) {
      v4f v = acc[mi][nj];
      if constexpr (kPoly) {
        const int64_t row = r0 + 16 * mi + r, col = q0 + 16 * nj + 4 * G;
        typedef _Float16 v4h __attribute__((ext_vector_type(4)));
        v4h old = {0, 0, 0, 0};
        if (row < n && col < ld) old = *reinterpret_cast<const v4h*>(src + row * ld + col);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = fmaf(c * (kB / kA / kA), v[e], b * (kB / kA) * float(old[e]));
          if (diagonal && row == col + e && row < n) v[e] = fmaf(a, kB, v[e]);
        }
      } else {
        v *= kA / kX / kX;
      }
      region.put(mi, nj, v2i{static_cast<int>(pack_half2(v[0], v[1])),
                             static_cast<int>(pack_half2(v[2], v[3]))});
    }
  region.settle();
#pragma unroll
  for (int k = 0; k < C::WM / 8; ++k) {
    const v4i v = region.row8(k);
    const int64_t row = r0 + 8 * k + (lane >> 3), col = q0 + 8 * (lane & 7);
    if (row < n && col < ld) *reinterpret_cast<v4i*>(out + row * ld + col) = v;
  }
  if (ti == tj) return;
#pragma unroll
  for (int k = 0; k < C::WM / 32; ++k)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const v4i v = region.col8(k, q);
      const int64_t row = q0 + 16 * q + r, col = r0 + 32 * k + 8 * G;
      if (row < n && col < ld) *reinterpret_cast<v4i*>(out + row * ld + col) = v;
    }
}

// X <- P X (or X P, P symmetric), plus a X from its two halves where `lo` is given (lo is replaced
// by the new X's where keep_lo says so). Written as hi [rows][ld], or (u) as bf16 [rows][cols].
struct Apply {
  int64_t rows, cols, ld;
  const _Float16* hi;
  _Float16* lo;
  _Float16* out;
  int64_t hi_stride, lo_stride;
  float a;
  bool add, keep_lo, last;
  float scale;
};

template <class C>
__global__ __launch_bounds__(C::kThreads) void ns_apply_kernel(Batch A, Batch B, Items it, Apply p,
                                                               int64_t tiles_i, int64_t tiles_j) {
  __shared__ __attribute__((aligned(1024))) uint8_t s0[C::kStageBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t s1[C::kStageBytes];
  const int64_t id = regroup(blockIdx.x, gridDim.x);
  const int64_t item = uniform64(id / (tiles_i * tiles_j));
  int64_t ti, tj;
  tile_at(id - item * tiles_i * tiles_j, tiles_i, tiles_j, 4, ti, tj);
  const int64_t i0 = uniform64(ti * C::BM), j0 = uniform64(tj * C::BN);
  const Operand a = A.at(item), b = B.at(item);
  const int64_t nk = (a.cols + kChunk - 1) / kChunk;
  v4f acc[C::MI][C::NJ];
  multiply<C>(a, b, i0, j0, 0, nk, nk, (lds_u8*)s0, (lds_u8*)s1, acc);
  __syncthreads();

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / C::WAVES_N, wn = wave % C::WAVES_N;
  const int G = lane >> 4, r = lane & 15;
  constexpr int kFirst = C::kStageBytes / Region<C>::kBytes;
  const Region<C> region(wave < kFirst ? (lds_u8*)s0 : (lds_u8*)s1,
                         wave < kFirst ? wave : wave - kFirst, lane);
  const int64_t r0 = i0 + wm * C::WM, q0 = j0 + wn * C::WN;
  typedef _Float16 v4h __attribute__((ext_vector_type(4)));
  const _Float16* hi = p.hi + item * p.hi_stride;
  _Float16* lo = p.lo + item * p.lo_stride;
#pragma unroll
  for (int mi = 0; mi < C::MI; ++mi)
#pragma unroll
    for (int nj = 0; nj < C::NJ; ++nj) {
      const int64_t row = r0 + 16 * mi + r, col = q0 + 16 * nj + 4 * G;
      const bool in = row < p.rows && col < p.ld;
      v4f v = acc[mi][nj] * (1.0f / kB);
      if (p.add && in) {
        const v4h h = *reinterpret_cast<const v4h*>(hi + row * p.ld + col);
        const v4h l = *reinterpret_cast<const v4h*>(lo + row * p.ld + col);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = fmaf(p.a, fmaf(float(l[e]), 1.0f / kLo, float(h[e])), v[e]);
      }
      v2i w;
      if (p.last) {
        v *= p.scale;
        w = {static_cast<int>(pack_bf16x2(v[0], v[1])), static_cast<int>(pack_bf16x2(v[2], v[3]))};
      } else {
        w = {static_cast<int>(pack_half2(v[0], v[1])), static_cast<int>(pack_half2(v[2], v[3]))};
        if (p.keep_lo && in) {
          const v4h h = __builtin_bit_cast(v4h, w);
          v4h l;
#pragma unroll
          for (int e = 0; e < 4; ++e) l[e] = static_cast<_Float16>((v[e] - float(h[e])) * kLo);
          *reinterpret_cast<v4h*>(lo + row * p.ld + col) = l;
        }
      }
      region.put(mi, nj, w);
    }
  region.settle();
  uint16_t* u = it.u[item];
  const bool whole = !p.last || (p.cols % 8 == 0 && (reinterpret_cast<uintptr_t>(u) & 15u) == 0);
  const int64_t ld = p.last ? p.cols : p.ld;
  uint16_t* dst = p.last ? u : reinterpret_cast<uint16_t*>(p.out + item * p.hi_stride);
#pragma unroll
  for (int k = 0; k < C::WM / 8; ++k) {
    const v4i v = region.row8(k);
    const int64_t row = r0 + 8 * k + (lane >> 3), col = q0 + 8 * (lane & 7);
    if (row >= p.rows || col >= ld) continue;
    uint16_t* q = dst + row * ld + col;
    if (whole) {
      *reinterpret_cast<v4i*>(q) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col + e < ld) q[e] = static_cast<uint16_t>(uint32_t(v[e / 2]) >> (16 * (e & 1)));
    }
  }
}

// ------------------------------------------------------------------ host
constexpr int64_t kFill = 256;  // compute units: tiles that fill the chip

inline int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
inline int64_t tiles_of(int64_t n, int64_t b) { return (n + b - 1) / b; }

struct Plan {
  int64_t ldx, side, lds;  // row stride of X; the shorter side and its stride
  bool tall;
  int parts;
  double* sums;
  _Float16 *hi[2], *lo, *A, *P;
  int64_t x_stride, s_stride, bytes;
};

Plan plan(int64_t count, int64_t rows, int64_t cols, void* ws) {
  Plan p;
  p.tall = rows > cols;
  p.side = p.tall ? cols : rows;
  p.ldx = up(cols, kChunk);
  p.lds = up(p.side, kChunk);
  const int64_t parts = tiles_of(rows * cols, kThreads * 16);
  p.parts = static_cast<int>(parts > kMaxParts ? kMaxParts : parts);
  p.x_stride = up(rows * p.ldx, 128);
  p.s_stride = up(p.side * p.lds, 128);
  uint8_t* at = static_cast<uint8_t*>(ws);
  auto take = [&](int64_t bytes) {
    uint8_t* q = at + p.bytes;
    p.bytes += up(bytes, 256);
    return q;
  };
  p.bytes = 0;
  p.sums = reinterpret_cast<double*>(take(count * p.parts * 8));
  p.hi[0] = reinterpret_cast<_Float16*>(take(2 * count * p.x_stride));
  p.hi[1] = reinterpret_cast<_Float16*>(take(2 * count * p.x_stride));
  p.lo = reinterpret_cast<_Float16*>(take(2 * count * p.x_stride));
  p.A = reinterpret_cast<_Float16*>(take(2 * count * p.s_stride));
  p.P = reinterpret_cast<_Float16*>(take(2 * count * p.s_stride));
  return p;
}

template <bool kTransA, bool kTransB>
using BigTile = Tile<256, 256, 2, 4, kTransA, kTransB, true>;
template <bool kTransA, bool kTransB>
using SmallTile = Tile<128, 128, 2, 2, kTransA, kTransB, true>;

// Whether 256x256 tiles of `tiles` per matrix fill the chip.
inline bool use_big(int64_t count, int64_t tiles) { return count * tiles >= kFill / 2; }

template <class C, bool kPoly>
void launch_symmetric(const Batch& x, _Float16* out, const Plan& p, int64_t count, float a,
                      float b, float c, bool diagonal, hipStream_t s) {
  const int64_t t = tiles_of(p.side, C::BM);
  const int tiles = static_cast<int>(t * (t + 1) / 2);
  hipLaunchKernelGGL((ns_symmetric_kernel<C, kPoly>), dim3(static_cast<uint32_t>(count * tiles)),
                     dim3(C::kThreads), 0, s, x, out, p.s_stride, p.side, p.lds, tiles, a, b, c,
                     diagonal);
}

template <class C>
void launch_apply(const Batch& A, const Batch& B, const Items& it, const Apply& ap, int64_t count,
                  hipStream_t s) {
  const int64_t ti = tiles_of(ap.rows, C::BM), tj = tiles_of(ap.cols, C::BN);
  hipLaunchKernelGGL(ns_apply_kernel<C>, dim3(static_cast<uint32_t>(count * ti * tj)),
                     dim3(C::kThreads), 0, s, A, B, it, ap, ti, tj);
}

// Whether the steps keep every singular value and matrix inside what the fixed scales hold: the
// default coefficients do (values stay below 1.21); others are followed over a grid of [0, 1].
bool coefficients_ok(const puro_newton_schulz_params& h) {
  const float *k = h.coefficients;
  if (!isfinite(k[0]) || !isfinite(k[1]) || !isfinite(k[2])) return false;
  if (k[0] == 3.4445f && k[1] == -4.7750f && k[2] == 2.0315f) return true;
  double top = 1.0, last = 0.0;
  for (int i = 0; i <= 512; ++i) {
    double x = i / 512.0;
    for (int n = 0; n < h.steps; ++n) {
      const double q = x * x;
      x = x * (k[0] + q * (k[1] + q * k[2]));
      if (!(fabs(x) < 1e4)) return false;
      if (n + 1 < h.steps && fabs(x) > top) top = fabs(x);
      if (fabs(x) > last) last = fabs(x);
    }
  }
  const double q = top * top;
  return top <= 1.75 && last <= 12.0 && fabs(k[0]) + fabs(k[1]) * q + fabs(k[2]) * q * q <= 28.0;
}

puro_status check_sizes(int64_t count, int64_t rows, int64_t cols) {
  if (count < 0 || rows < 0 || cols < 0) return PURO_ERR_SHAPE;
  if (count > kMax) return PURO_ERR_ARG;
  const int64_t side = rows < cols ? rows : cols, other = rows < cols ? cols : rows;
  if (side > PURO_NS_MAX_SIDE || other > PURO_NS_MAX_LONG) return PURO_ERR_SHAPE;
  // launches: 128x128 tiles of every matrix, by 256 threads
  if (!grid_ok(count * tiles_of(rows, 128) * tiles_of(cols, 128), 512)) return PURO_ERR_SHAPE;
  return PURO_OK;
}

}  // namespace
}  // namespace puro

using namespace puro;

extern "C" int64_t puro_newton_schulz_workspace(int64_t count, int64_t rows, int64_t cols) {
  if (check_sizes(count, rows, cols) != PURO_OK || count == 0 || rows == 0 || cols == 0) return 0;
  return plan(count, rows, cols, nullptr).bytes;
}

extern "C" puro_status puro_newton_schulz(const puro_ns_item* items, int count, int64_t rows,
                                          int64_t cols, const puro_newton_schulz_params* hp,
                                          void* workspace, void* stream) {
  PURO_TRY(check_sizes(count, rows, cols));
  if (hp == nullptr) return PURO_ERR_NULL;
  if (hp->steps < 1 || hp->steps > PURO_NS_MAX_STEPS || (hp->nesterov != 0 && hp->nesterov != 1) ||
      !(hp->beta >= 0.0f && hp->beta < 1.0f) || !isfinite(hp->scale) || !coefficients_ok(*hp))
    return PURO_ERR_ARG;
  if (count == 0 || rows == 0 || cols == 0) return PURO_OK;
  if (items == nullptr) return PURO_ERR_NULL;
  Items it = {};
  bool vec = cols % 4 == 0;
  const bool momentum = items[0].m != nullptr;
  for (int n = 0; n < count; ++n) {
    const puro_ns_item& i = items[n];
    if (i.g == nullptr || i.u == nullptr) return PURO_ERR_NULL;
    if ((i.m != nullptr) != momentum) return PURO_ERR_ARG;
    if ((i.m != nullptr) != (i.m_out != nullptr)) return PURO_ERR_NULL;
    const uintptr_t f = reinterpret_cast<uintptr_t>(i.g) | reinterpret_cast<uintptr_t>(i.m) |
                        reinterpret_cast<uintptr_t>(i.m_out);
    if (f % 4 || reinterpret_cast<uintptr_t>(i.u) % 2) return PURO_ERR_ALIGN;
    vec = vec && f % 16 == 0;
    it.g[n] = i.g;
    it.m[n] = i.m;
    it.mo[n] = i.m_out;
    it.u[n] = static_cast<uint16_t*>(i.u);
  }
  PURO_TRY(check_ptr(workspace, false));
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const Plan p = plan(count, rows, cols, workspace);
  const Momentum k = {momentum, hp->nesterov != 0, hp->beta, 1.0f - hp->beta};
  const dim3 sums(p.parts, count);
  int64_t blocks = tiles_of(rows * (p.ldx / 4), kThreads * 4);
  if (blocks > 2048) blocks = 2048;
  const dim3 conv(static_cast<uint32_t>(blocks), count);
  if (vec) {
    hipLaunchKernelGGL(ns_momentum_kernel<true>, sums, dim3(kThreads), 0, s, it, rows * cols, k,
                       p.sums);
    hipLaunchKernelGGL(ns_convert_kernel<true>, conv, dim3(kThreads), 0, s, it, rows, cols, p.ldx,
                       k, p.sums, p.parts, p.hi[0], p.lo, p.x_stride, p.x_stride);
  } else {
    hipLaunchKernelGGL(ns_momentum_kernel<false>, sums, dim3(kThreads), 0, s, it, rows * cols, k,
                       p.sums);
    hipLaunchKernelGGL(ns_convert_kernel<false>, conv, dim3(kThreads), 0, s, it, rows, cols, p.ldx,
                       k, p.sums, p.parts, p.hi[0], p.lo, p.x_stride, p.x_stride);
  }
  const float a = hp->coefficients[0], b = hp->coefficients[1], c = hp->coefficients[2];
  const int64_t side_tiles = tiles_of(p.side, 256);
  const bool big_s = use_big(count, side_tiles * (side_tiles + 1) / 2);
  const bool big_x = use_big(count, tiles_of(rows, 256) * tiles_of(cols, 256));
  const Batch A = {p.A, p.s_stride, p.side, p.lds, p.lds};
  const Batch P = {p.P, p.s_stride, p.side, p.lds, p.lds};
  for (int n = 0; n < hp->steps; ++n) {
    const Batch X = {p.hi[n & 1], p.x_stride, rows, p.ldx, p.ldx};
    const bool both = n + 2 < hp->steps;  // this step's X is in two halves
    if (p.tall) {
      if (big_s)
        launch_symmetric<BigTile<true, true>, false>(X, p.A, p, count, 0, 0, 0, false, s);
      else
        launch_symmetric<SmallTile<true, true>, false>(X, p.A, p, count, 0, 0, 0, false, s);
    } else {
      if (big_s)
        launch_symmetric<BigTile<false, false>, false>(X, p.A, p, count, 0, 0, 0, false, s);
      else
        launch_symmetric<SmallTile<false, false>, false>(X, p.A, p, count, 0, 0, 0, false, s);
    }
    if (big_s)
      launch_symmetric<BigTile<false, false>, true>(A, p.P, p, count, a, b, c, !both, s);
    else
      launch_symmetric<SmallTile<false, false>, true>(A, p.P, p, count, a, b, c, !both, s);
    Apply ap = {};
    ap.rows = rows;
    ap.cols = cols;
    ap.ld = p.ldx;
    ap.hi = p.hi[n & 1];
    ap.lo = p.lo;
    ap.out = p.hi[(n + 1) & 1];
    ap.hi_stride = ap.lo_stride = p.x_stride;
    ap.a = a;
    ap.add = both;
    ap.keep_lo = n + 3 < hp->steps;
    ap.last = n + 1 == hp->steps;
    ap.scale = hp->scale / kX;
    if (p.tall) {
      if (big_x)
        launch_apply<BigTile<false, false>>(X, P, it, ap, count, s);
      else
        launch_apply<SmallTile<false, false>>(X, P, it, ap, count, s);
    } else {
      if (big_x)
        launch_apply<BigTile<false, true>>(P, X, it, ap, count, s);
      else
        launch_apply<SmallTile<false, true>>(P, X, it, ap, count, s);
    }
  }
  return launch_status();
}
