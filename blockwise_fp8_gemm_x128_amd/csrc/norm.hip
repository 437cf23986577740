// The boundary between two blocks of a transformer for gfx950, in one pass: the norm after a
// block, its gate and residual scale, and the norm before the next block.
//
// Per row, over D columns:
//   ry = rsqrt(mean y^2 + eps)      p  = y ry w_post
//   r' = beta r + alpha g p         rr = rsqrt(mean r'^2 + eps)      n = r' rr w_pre
// with the gate g absent, per column, per row or per element. Backward, with yh = y ry and
// rh = r' rr from the stored y and r' (bf16/fp32, or 8-bit checkpoints) and the stored ry, rr:
//   G  = dr' + rr (w_pre dn - rh k1),        k1 = mean(rh w_pre dn)
//   dr = beta G,    dp = alpha g G,    dy = ry (w_post dp - yh mean(yh w_post dp))
//   dw_pre = sum_rows dn rh,  dw_post = sum_rows dp yh,  dgate = alpha w_post yh G (summed)
// The last mean needs G, which needs k1; but with A = dr' + rr w_pre dn and q = yh w_post g it is
// alpha (sum q A - rr k1 sum q rh)/D, so one reduction of three sums serves both.
//
// HBM-bound: every element of every input is read once into registers, where the row stays until
// its last output is written (but for the backward pass of rows of more than 8192 columns, which
// reads a gate per element twice); a row belongs to one team of lanes (16, 32 or 64 lanes of a wave for
// short rows, whole waves or groups of 16 lanes for longer ones), 8 columns per lane and vector.
// All statistics and sums are fp32; r' is normalised unrounded, so n does not see the residual
// stream's rounding.
#include <algorithm>
#include <cmath>

#include "block.hpp"

namespace puro {
namespace {

constexpr int kMaxWaves = 16;  // of a block
// How a row lies over lanes (kLanes): 16, 32 or 64 lanes of a wave, one lane of 16 (kOne: rows of
// fewer than eight columns), whole waves (kWaves) or groups of 16 lanes (kGroups), `wpt` of them.
constexpr int kWaves = 0, kOne = 1, kGroups = 2;

// Sum over the team of each of kN values. Teams across waves go through LDS with one barrier;
// `sh` alternates between calls, so a wave that is already writing the next call's values never
// meets one still reading this call's.
template <int kLanes, int kN, int kMax>
__device__ __forceinline__ void team_sum(float (&v)[kN], float (*sh)[kMax], int wpt) {
  if constexpr (kLanes == kGroups) {
    const int g = threadIdx.x >> 4, l = threadIdx.x & 15, g0 = g - g % wpt;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      v[k] = lanes_sum<16>(v[k]);
      if (l == 0) sh[k][g] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const float t = sh[k][min(g0 + l, kMax - 1)];
      v[k] = lanes_sum<16>(l < wpt ? t : 0.0f);
    }
  } else if constexpr (kLanes != 0) {
#pragma unroll
    for (int k = 0; k < kN; ++k) v[k] = lanes_sum<kLanes == kOne ? 16 : kLanes>(v[k]);
  } else {
    const int wave = threadIdx.x >> 6, w0 = wave - wave % wpt;
#pragma unroll
    for (int k = 0; k < kN; ++k) v[k] = lanes_sum<64>(v[k]);
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < kN; ++k) sh[k][wave] = v[k];
    }
    __syncthreads();
    // lane w of each 16 takes wave w's sum, and the 16 are summed like the lanes before
    const int w = threadIdx.x & 15;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const float t = sh[k][min(w0 + w, kMaxWaves - 1)];
      v[k] = lanes_sum<16>(w < wpt ? t : 0.0f);
    }
  }
}

// Sum over a wave's teams of kLanes lanes, lane by lane.
template <int kLanes>
__device__ __forceinline__ float teams_sum(float v) {
  if constexpr (kLanes == kOne || kLanes == 16) {
    const uint32_t u = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  if constexpr (kLanes == kOne || kLanes == 16 || kLanes == 32) {
    const uint32_t u = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  return v;
}

// The lanes of one team and the rows of one block.
template <int kLanes>
struct Team {
  int lanes, lane, team, teams;
  __device__ __forceinline__ explicit Team(int wpt) {
    lanes = kLanes == kWaves    ? wpt * 64
            : kLanes == kGroups ? wpt * 16
            : kLanes == kOne    ? 16
                                : kLanes;
    team = threadIdx.x / lanes;
    // teams of whole waves: the row is the same in all lanes of a wave, its addresses scalar
    if (kLanes == kWaves || kLanes == 64) team = __builtin_amdgcn_readfirstlane(team);
    lane = threadIdx.x - team * lanes;
    teams = blockDim.x / lanes;
  }
  // Lanes of a block of groups that make no whole team (team == teams) have no row.
  __device__ __forceinline__ bool has_row(int base, int end) const {
    return base + team < end && (kLanes != kGroups || team < teams);
  }
};

// The rows of a block: `teams` a step, in steps dealt out evenly.
template <typename Args>
__device__ __forceinline__ void block_rows(const Args& a, int teams, int& first, int& end) {
  const int b = blockIdx.x;
  first = (b * a.steps + min(b, a.more)) * teams;   // of at most 2^24 rows
  end = min(static_cast<int>(a.rows), first + (a.steps + (b < a.more)) * teams);
}

// Eight of a vector over the columns (a weight, a gate), or `none` where there is none.
template <bool kShort>
__device__ __forceinline__ void row_vector(const float* w, const Span<kShort>& sp, float none,
                                           float* f) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) f[i] = none;
    return;
  }
  F8 r;
  load<false, kShort>(r, row_ptr<true>(w, 0), sp);
  values(r, sp, f);
}

// ------------------------------------------------------------------ forward
struct FwdArgs {
  const uint16_t* y;
  const void* r;
  const float *w_post, *w_pre;
  const void* gate;
  int gate_kind, pow2;
  int64_t rows;
  int cols, wpt, steps, more;   // steps of a block; of the first `more` blocks one more
  float alpha, beta, eps;
  void* r_out;
  uint16_t* n;
  uint8_t* nq;
  float *ns, *rstd_y, *rstd_r;
  uint8_t* yq;
  float* ys;
  uint8_t* rq;
  float* rs;
};

// Where a row's 8-bit form goes.
struct CodeOut {
  uint8_t* q;
  float* s;
};
// A lane's eight codes; `lane` of the 16 that share the group stores its scale.
template <bool kUniform, bool kLater>
__device__ __forceinline__ void store_codes(const CodeOut& o, int64_t row, int64_t rows,
                                            uint32_t cols, uint32_t col, int n, bool in,
                                            const float* f, float r, float scale, uint32_t lane) {
  store8<kLater>(row_ptr<kUniform>(o.q, row * cols) + col, n, encode8(f, r));
  if ((threadIdx.x & 15) == lane && in && (col & ~127u) < cols)
    row_ptr<kUniform>(o.s, row)[static_cast<int64_t>(col >> 7) * rows] = scale;
}

// One row's inputs as loaded.
template <typename R, int kNV>
struct FwdRow {
  typename RawOf<R>::type r[kNV];
  Bf16x8 y[kNV], gate[kNV];
  float gt;
};

template <bool kUniform, typename R, int kNV, bool kShort>
__device__ __forceinline__ void load_row(FwdRow<R, kNV>& w, const FwdArgs& a, int64_t row,
                                         const Span<kShort> (&sp)[kNV]) {
  const int64_t at = row * a.cols;
  w.gt = a.gate_kind == PURO_GATE_TOKEN ? static_cast<const float*>(a.gate)[row] : 1.0f;
#pragma unroll
  for (int j = 0; j < kNV; ++j) {
    if (a.y) load<true, kShort>(w.y[j], row_ptr<kUniform>(a.y, at), sp[j]);
    load<true, kShort>(w.r[j], row_ptr<kUniform>(static_cast<const R*>(a.r), at), sp[j]);
    if (a.gate_kind == PURO_GATE_FULL)
      load<true, kShort>(w.gate[j],
                         row_ptr<kUniform>(static_cast<const uint16_t*>(a.gate), at), sp[j]);
  }
}

template <typename R, int kLanes, int kNV>
__global__ __launch_bounds__(kLanes == kWaves ? 1024 : kLanes == kGroups ? 320 : 256)
void norm_fwd_kernel(const FwdArgs a) {
  constexpr bool kCross = kLanes == kWaves || kLanes == kGroups;  // teams across waves
  __shared__ float sh[2][1][kLanes == kGroups ? 32 : kMaxWaves];
  constexpr bool kShort = kLanes == kOne;  // rows of fewer than eight columns, in one lane of 16
  constexpr bool kUniform = kLanes == kWaves || kLanes == 64;
  const Team<kLanes> tm(a.wpt);
  const float inv_d = 1.0f / static_cast<float>(a.cols);
  const bool channel = a.gate_kind == PURO_GATE_CHANNEL, full = a.gate_kind == PURO_GATE_FULL;
  const bool pow2 = a.pow2 != 0;

  float cw[kNV][kVec], pw[kNV][kVec];  // alpha (gate) w_post; w_pre
  Span<kShort> sp[kNV];
#pragma unroll
  for (int j = 0; j < kNV; ++j) {
    sp[j] = Span<kShort>((j * tm.lanes + tm.lane) * kVec, a.cols,
                         a.cols != tm.lanes * kVec * kNV);
    row_vector(a.w_post, sp[j], 0.0f, cw[j]);
    float g[kVec];
    row_vector(channel ? static_cast<const float*>(a.gate) : nullptr, sp[j], 1.0f, g);
#pragma unroll
    for (int i = 0; i < kVec; ++i) cw[j][i] *= a.alpha * g[i];
    row_vector(a.w_pre, sp[j], 0.0f, pw[j]);
  }

  int first, end;
  block_rows(a, tm.teams, first, end);
  // A team without a row works on the last one again and stores nothing.
  FwdRow<R, kNV> w;
  for (int base = first; base < end; base += tm.teams) {  // the same count for every team
    const int64_t row = min(base + tm.team, end - 1);
    const bool in = tm.has_row(base, end);
    load_row<kUniform>(w, a, row, sp);
    const int64_t at = row * a.cols;
    float y[kNV][kVec], t[kNV][kVec];
    uint32_t ymax[kNV];
    float ry = 0.0f;
    if (a.y) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int j = 0; j < kNV; ++j) {
        settle(w.y[j], sp[j]);
        widen8(w.y[j].v, y[j]);
        ymax[j] = max8(w.y[j]);
#pragma unroll
        for (int i = 0; i < kVec; ++i) ss[0] = fmaf(y[j][i], y[j][i], ss[0]);
      }
      team_sum<kLanes>(ss, sh[0], a.wpt);
      ry = rsqrtf(fmaf(ss[0], inv_d, a.eps));
      if (in && tm.lane == 0) a.rstd_y[row] = ry;
    }
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
      float r[kVec];
      values(w.r[j], sp[j], r);
      if (a.y) {
        const float f = ry * w.gt;
        if (full) {
          float g[kVec];
          values(w.gate[j], sp[j], g);
#pragma unroll
          for (int i = 0; i < kVec; ++i)
            t[j][i] = fmaf(y[j][i] * cw[j][i] * g[i], f, a.beta * r[i]);
        } else {
#pragma unroll
          for (int i = 0; i < kVec; ++i)
            t[j][i] = fmaf(y[j][i] * cw[j][i], f, a.beta * r[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) t[j][i] = a.beta * r[i];
      }
    }
    float ss[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
      const int n = in ? sp[j].n : 0;
#pragma unroll
      for (int i = 0; i < kVec; ++i) ss[0] = fmaf(t[j][i], t[j][i], ss[0]);
      if (a.r_out)
        store8<true>(row_ptr<kUniform>(static_cast<R*>(a.r_out), at) + sp[j].col, n, t[j]);
      if (a.yq && a.rq) {  // both scales from one pair of divisions
        float both[2][kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) both[0][i] = y[j][i], both[1][i] = t[j][i];
        const uint32_t m[2] = {ymax[j], max8<false>(t[j])};
        const RowGroups<2> g = row_groups<2>(m, both, pow2);
        store_codes<kUniform, true>({a.yq, a.ys}, row, a.rows, a.cols, sp[j].col, n, in,
                                    y[j], g.r[0], g.s, 0);
        store_codes<kUniform, true>({a.rq, a.rs}, row, a.rows, a.cols, sp[j].col, n, in,
                                    t[j], g.r[1], g.s, 1);
      } else if (a.yq) {
        const uint32_t m[1] = {ymax[j]};
        const RowGroups<1> g = row_groups<1>(m, &y[j], pow2);
        store_codes<kUniform, true>({a.yq, a.ys}, row, a.rows, a.cols, sp[j].col, n, in,
                                    y[j], g.r[0], g.s, 0);
      } else if (a.rq) {
        const RowGroups<1> g = row_groups<false, 1>(&t[j], pow2);
        store_codes<kUniform, true>({a.rq, a.rs}, row, a.rows, a.cols, sp[j].col, n, in,
                                    t[j], g.r[0], g.s, 0);
      }
    }
    if (!a.w_pre) {
      if constexpr (kCross) __syncthreads();  // before sh[0] is written again
      continue;
    }
    team_sum<kLanes>(ss, sh[1], a.wpt);
    const float rr = rsqrtf(fmaf(ss[0], inv_d, a.eps));
    if (in && tm.lane == 0) a.rstd_r[row] = rr;
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
      const int n = in ? sp[j].n : 0;
      float o[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) o[i] = t[j][i] * rr * pw[j][i];
      if (a.n) store8(row_ptr<kUniform>(a.n, at) + sp[j].col, n, o);
      if (a.nq) {
        const RowGroups<1> g = row_groups<false, 1>(&o, pow2);
        store_codes<kUniform, false>({a.nq, a.ns}, row, a.rows, a.cols, sp[j].col, n, in,
                                     o, g.r[0], g.s, 0);
      }
    }
    if (kCross && !a.y) __syncthreads();  // before sh[1] is written again
  }
}

// ------------------------------------------------------------------ backward
struct BwdArgs {
  const void* dr_out;
  const uint16_t* dn;
  const uint16_t* y;
  const uint8_t* yq;
  const float* ys;
  const void* r;
  const uint8_t* rq;
  const float* rs;
  const float *rstd_y, *rstd_r, *w_post, *w_pre;
  const void* gate;
  int gate_kind;
  int64_t rows;
  int cols, wpt, steps, more;   // steps of a block; of the first `more` blocks one more
  float alpha, beta;
  void* dr;
  uint16_t* dy;
  void* dgate;       // per row or per element; per column through the partial sums
  float* partials;   // [blocks][2][cols]: sums of g yh G and of dn rh
};

// One row's inputs as loaded: the stored activations as codes (kCodes) or as they were.
template <typename R, int kNV, bool kCodes>
struct BwdRow {
  typename RawOf<R>::type d[kNV], r[kNV];
  Bf16x8 dn[kNV], y[kNV], gate[kNV];
  float ry, rr, gt;
};
template <typename R, int kNV>
struct BwdRow<R, kNV, true> {
  typename RawOf<R>::type d[kNV];
  Fp8x8 r[kNV], y[kNV];
  Bf16x8 dn[kNV], gate[kNV];
  float rs[kNV], ys[kNV];
  float ry, rr, gt;
};

template <bool kUniform, bool kShort>
__device__ __forceinline__ void load_gate(Bf16x8& g, const BwdArgs& a, int64_t row,
                                          const Span<kShort>& sp) {
  load<true, kShort>(
      g, row_ptr<kUniform>(static_cast<const uint16_t*>(a.gate), row * a.cols), sp);
}

template <bool kUniform, typename R, int kNV, bool kCodes, bool kShort>
__device__ __forceinline__ void load_row(BwdRow<R, kNV, kCodes>& w, const BwdArgs& a, int64_t row,
                                         const Span<kShort> (&sp)[kNV]) {
  const int64_t at = row * a.cols;
  w.gt = a.gate_kind == PURO_GATE_TOKEN ? static_cast<const float*>(a.gate)[row] : 1.0f;
  w.ry = a.w_post ? a.rstd_y[row] : 0.0f;
  w.rr = a.w_pre ? a.rstd_r[row] : 0.0f;
#pragma unroll
  for (int j = 0; j < kNV; ++j) {
    const int64_t sat = int64_t(min(sp[j].col, a.cols - 1u) >> 7) * a.rows;
    if (a.dr_out)
      load<true, kShort>(w.d[j], row_ptr<kUniform>(static_cast<const R*>(a.dr_out), at), sp[j]);
    if (a.w_pre) {
      load<true, kShort>(w.dn[j], row_ptr<kUniform>(a.dn, at), sp[j]);
      if constexpr (kCodes) {
        load<true, kShort>(w.r[j], row_ptr<kUniform>(a.rq, at), sp[j]);
        w.rs[j] = row_ptr<kUniform>(a.rs, row)[sat];
      } else {
        load<true, kShort>(w.r[j], row_ptr<kUniform>(static_cast<const R*>(a.r), at), sp[j]);
      }
    }
    if (a.w_post) {
      if constexpr (kCodes) {
        load<true, kShort>(w.y[j], row_ptr<kUniform>(a.yq, at), sp[j]);
        w.ys[j] = row_ptr<kUniform>(a.ys, row)[sat];
      } else {
        load<true, kShort>(w.y[j], row_ptr<kUniform>(a.y, at), sp[j]);
      }
    }
    if (kNV == 1 && a.gate_kind == PURO_GATE_FULL) load_gate<kUniform>(w.gate[j], a, row, sp[j]);
  }
}

// The weight after the block times a channel gate, which is how both directions use it.
template <bool kShort>
__device__ __forceinline__ void post_weight(const BwdArgs& a, const Span<kShort>& sp, float* f) {
  row_vector(a.w_post, sp, 0.0f, f);
  float g[kVec];
  row_vector(a.gate_kind == PURO_GATE_CHANNEL ? static_cast<const float*>(a.gate) : nullptr, sp,
             1.0f, g);
#pragma unroll
  for (int i = 0; i < kVec; ++i) f[i] *= g[i];
}

// Eight sums of a lane in LDS, its own: no other lane reads or writes them.
__device__ __forceinline__ void lds_add(float4* lo, float4* hi, const float* f) {
  float4 a = *lo, b = *hi;
  a.x += f[0], a.y += f[1], a.z += f[2], a.w += f[3];
  b.x += f[4], b.y += f[5], b.z += f[6], b.w += f[7];
  *lo = a, *hi = b;
}

// Two vectors per lane (kWide: rows of more than 8192 columns, one per block of up to 1024 threads)
// would take 190 registers where 128 are to be had: there the column sums stand in LDS (128 KB, one
// block per CU as before), and the weights and a gate per element are read again where they are
// used, from the caches. 4096 x 16384 in 182 us instead of 504, which were spills.
template <typename R, int kLanes, int kNV, bool kCodes>
__global__ __launch_bounds__(kLanes == kWaves ? 1024 : 512, kLanes == kGroups ? 4 : 1)
void norm_bwd_kernel(const BwdArgs a) {
  constexpr bool kCross = kLanes == kWaves || kLanes == kGroups;  // teams across waves
  __shared__ float sh[2][3][kLanes == kGroups ? 32 : kMaxWaves];
  constexpr bool kWide = kNV == 2;
  constexpr bool kShort = kLanes == kOne;  // rows of fewer than eight columns, in one lane of 16
  constexpr bool kUniform = kLanes == kWaves || kLanes == 64;
  const Team<kLanes> tm(a.wpt);
  const float inv_d = 1.0f / static_cast<float>(a.cols);
  const bool full = a.gate_kind == PURO_GATE_FULL;
  const bool post = a.w_post != nullptr, pre = a.w_pre != nullptr;

  float wg[kNV][kVec], wp[kNV][kVec];  // w_post (times a channel gate); w_pre
  __shared__ float4 own[kWide ? 2 : 1][kWide ? 2 * kNV : 1][kWide ? 1024 : 1];
  float acc[2][kNV][kVec] = {};
  Span<kShort> sp[kNV];
#pragma unroll
  for (int j = 0; j < kNV; ++j) {
    sp[j] = Span<kShort>((j * tm.lanes + tm.lane) * kVec, a.cols,
                         a.cols != tm.lanes * kVec * kNV);
    if constexpr (kWide) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        own[k][2 * j][threadIdx.x] = own[k][2 * j + 1][threadIdx.x] = make_float4(0, 0, 0, 0);
    } else {
      post_weight(a, sp[j], wg[j]);
      row_vector(a.w_pre, sp[j], 0.0f, wp[j]);
    }
  }

  int first, end;
  block_rows(a, tm.teams, first, end);
  const int t = threadIdx.x;
  int buf = 0;
  BwdRow<R, kNV, kCodes> w;
  load_row<kUniform>(w, a, min(first + tm.team, end - 1), sp);
  for (int base = first; base < end; base += tm.teams, buf ^= 1) {
    // A team without a row has loaded the last one again; it takes its values as zero, whatever
    // they are (that row may be changing in place), and stores nothing.
    const int64_t row = min(base + tm.team, end - 1);
    const bool in = tm.has_row(base, end);
    const float ry = in ? w.ry : 0.0f, rr = in ? w.rr : 0.0f, gt = in ? w.gt : 0.0f;
    float A[kNV][kVec], yh[kNV][kVec], rh[kNV][kVec];
    Bf16x8 graw[kNV];
    float sums[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
      if (a.dr_out && in) {
        values(w.d[j], sp[j], A[j]);
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) A[j][i] = 0.0f;
      }
      if (pre && in) {
        if constexpr (kWide) row_vector(a.w_pre, sp[j], 0.0f, wp[j]);
        float dn[kVec];
        values(w.dn[j], sp[j], dn);
        if constexpr (kCodes)
          values(w.r[j], sp[j], w.rs[j], rh[j]);
        else
          values(w.r[j], sp[j], rh[j]);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          rh[j][i] *= rr;
          const float x = wp[j][i] * dn[i];
          A[j][i] = fmaf(rr, x, A[j][i]);
          sums[0] = fmaf(rh[j][i], x, sums[0]);
          if constexpr (kWide)
            dn[i] *= rh[j][i];
          else
            acc[1][j][i] = fmaf(dn[i], rh[j][i], acc[1][j][i]);
        }
        if constexpr (kWide) lds_add(&own[1][2 * j][t], &own[1][2 * j + 1][t], dn);
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) rh[j][i] = 0.0f;
      }
      if (post && in) {
        if constexpr (kWide) post_weight(a, sp[j], wg[j]);
        if constexpr (kCodes)
          values(w.y[j], sp[j], w.ys[j], yh[j]);
        else
          values(w.y[j], sp[j], yh[j]);
        float q[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          yh[j][i] *= ry;
          q[i] = yh[j][i] * wg[j][i];
        }
        if (full) {
          float g[kVec];
          if constexpr (kWide)
            load_gate<kUniform>(graw[j], a, row, sp[j]);
          else
            graw[j] = w.gate[j];
          values(graw[j], sp[j], g);
#pragma unroll
          for (int i = 0; i < kVec; ++i) q[i] *= g[i];
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          sums[1] = fmaf(q[i], A[j][i], sums[1]);
          sums[2] = fmaf(q[i], rh[j][i], sums[2]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) yh[j][i] = 0.0f;
      }
    }
    // the next row's loads go out before this one's sums and stores
    if (base + tm.teams < end)
      load_row<kUniform>(w, a, min(base + tm.teams + tm.team, end - 1), sp);
    team_sum<kLanes>(sums, sh[buf], a.wpt);
    const float k1 = rr * sums[0] * inv_d;
    const float qg = sums[1] - k1 * sums[2];  // sum of q G
    const float ag = a.alpha * ry;
    const float k2 = -ag * gt * qg * inv_d;
    if (a.gate_kind == PURO_GATE_TOKEN && in && tm.lane == 0)
      static_cast<float*>(a.dgate)[row] = a.alpha * qg;
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
      const int n = in ? sp[j].n : 0;
      const int64_t at = row * a.cols;
      const uint32_t col = sp[j].col;
      float G[kVec], o[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        G[i] = fmaf(-k1, rh[j][i], A[j][i]);
        o[i] = a.beta * G[i];
      }
      if (a.dr) store8<true>(row_ptr<kUniform>(static_cast<R*>(a.dr), at) + col, n, o);
      if (post) {
        if constexpr (kWide) post_weight(a, sp[j], wg[j]);
        if (full && in) {
          float g[kVec];
          if constexpr (kWide) load_gate<kUniform>(graw[j], a, row, sp[j]);
          values(graw[j], sp[j], g);
#pragma unroll
          for (int i = 0; i < kVec; ++i) o[i] = a.alpha * yh[j][i] * wg[j][i] * G[i];
          store8(row_ptr<kUniform>(static_cast<uint16_t*>(a.dgate), at) + col, n, o);
#pragma unroll
          for (int i = 0; i < kVec; ++i) G[i] *= g[i];
        }
        // a channel gate is left out of the column sum, which so serves dw_post and dgate
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          G[i] *= gt;
          if constexpr (!kWide) acc[0][j][i] = fmaf(yh[j][i], G[i], acc[0][j][i]);
          o[i] = fmaf(wg[j][i] * ag, G[i], k2 * yh[j][i]);
        }
        store8(row_ptr<kUniform>(a.dy, at) + col, n, o);
        if constexpr (kWide) {
#pragma unroll
          for (int i = 0; i < kVec; ++i) G[i] *= yh[j][i];
          lds_add(&own[0][2 * j][t], &own[0][2 * j + 1][t], G);
        }
      }
    }
  }

  if constexpr (kWide) {
#pragma unroll
    for (int j = 0; j < kNV; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float4 lo = own[k][2 * j][t], hi = own[k][2 * j + 1][t];
        const float f[kVec] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        store8(a.partials + (int64_t(blockIdx.x) * 2 + k) * a.cols + sp[j].col, sp[j].n, f);
      }
    return;
  }
  // Column sums of the block: over the teams of a wave in registers, over the others through LDS,
  // where each thread then sums whole columns; one partial per block.
  extern __shared__ float red[];
  const int lanes = tm.lanes;
  const int rows = kCross ? tm.teams : static_cast<int>(blockDim.x >> 6);
  const int at = kCross ? threadIdx.x
                             : (threadIdx.x >> 6) * lanes + (threadIdx.x & 63);  // of kLanes lanes
  const int width = lanes * kVec;
#pragma unroll
  for (int j = 0; j < kNV; ++j) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[k][j][i] = teams_sum<kLanes>(acc[k][j][i]);
    }
    if (rows == 1) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
        store8(a.partials + (int64_t(blockIdx.x) * 2 + k) * a.cols + sp[j].col,
               tm.team < tm.teams ? sp[j].n : 0, acc[k][j]);
      continue;
    }
    __syncthreads();
    if (kCross ? tm.team < tm.teams : kLanes == 64 || (threadIdx.x & 63) < lanes)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float4* dst = reinterpret_cast<float4*>(red + k * rows * width + at * kVec);
        dst[0] = make_float4(acc[k][j][0], acc[k][j][1], acc[k][j][2], acc[k][j][3]);
        dst[1] = make_float4(acc[k][j][4], acc[k][j][5], acc[k][j][6], acc[k][j][7]);
      }
    __syncthreads();
    for (int t = threadIdx.x; t < 2 * width; t += blockDim.x) {
      const int k = t >= width, c = t - k * width;
      float v = 0.0f;
      for (int w = 0; w < rows; ++w) v += red[(k * rows + w) * width + c];
      if (j * width + c < a.cols)
        a.partials[(int64_t(blockIdx.x) * 2 + k) * a.cols + j * width + c] = v;
    }
  }
}

// Sum of the block partials per column in a fixed order: a block of 1024 threads has 32 columns,
// four to a thread, and every 128th partial to a thread; then a tree over the threads in LDS.
struct ReduceArgs {
  const float* partials;
  int blocks, cols, gate_kind, accumulate;
  float alpha;
  const float *w_post, *gate;
  float *dw_post, *dw_pre, *dgate;
};

constexpr int kRedCols = 32, kRedRows = 128;

__global__ __launch_bounds__(1024) void norm_reduce_kernel(const ReduceArgs a) {
  __shared__ float sh[kRedRows][kRedCols + 4];
  const int k = blockIdx.y, y = threadIdx.x >> 3, c0 = (threadIdx.x & 7) * 4;
  const int col = blockIdx.x * kRedCols + c0, n = a.cols - col;
  float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (n >= 4) {
#pragma unroll 4
    for (int b = y; b < a.blocks; b += kRedRows) {
      const f32x4_el v =
          *reinterpret_cast<const f32x4_el*>(a.partials + (int64_t(b) * 2 + k) * a.cols + col);
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] += v[i];
    }
  } else {
    for (int b = y; b < a.blocks; b += kRedRows)
      for (int i = 0; i < n; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          t[j] += i == j ? a.partials[(int64_t(b) * 2 + k) * a.cols + col + i] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) sh[y][c0 + i] = t[i];
  __syncthreads();
  // 32 threads per column: four partials each, then over the 32 lanes
  const int c = blockIdx.x * kRedCols + (threadIdx.x >> 5), l = threadIdx.x & 31;
  float v = 0.0f;
#pragma unroll
  for (int i = 0; i < kRedRows / 32; ++i) v += sh[i * 32 + l][threadIdx.x >> 5];
  v = lanes_sum<32>(v);
  if (l != 0 || c >= a.cols) return;
  if (k == 1) {
    if (a.dw_pre) a.dw_pre[c] = v + (a.accumulate ? a.dw_pre[c] : 0.0f);
    return;
  }
  const bool channel = a.gate_kind == PURO_GATE_CHANNEL;
  if (a.dw_post)
    a.dw_post[c] = a.alpha * (channel ? a.gate[c] : 1.0f) * v +
                   (a.accumulate ? a.dw_post[c] : 0.0f);
  if (channel && a.dgate)
    a.dgate[c] = a.alpha * a.w_post[c] * v + (a.accumulate ? a.dgate[c] : 0.0f);
}

// The gradient of a gate per row where there are no columns to sum over.
__global__ __launch_bounds__(256) void zero_kernel(float* p, int64_t n) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

// ------------------------------------------------------------------ host side
// How a row is laid over lanes: 16, 32 or 64 lanes of 8 columns up to 512 columns, then whole
// waves, one vector per lane up to a number of columns and two beyond; or, up to 2048 columns,
// groups of 16 lanes in a block of `least` to `most` threads.
struct Shape {
  int lanes;     // 16, 32, 64, kOne, kGroups or kWaves
  int nv;        // vectors of 8 columns per lane
  int wpt;       // waves or groups per team
  int threads;   // per block
  int teams;     // per block
};
struct Blocks {
  int threads, least, most;   // of several teams; of groups
  int one;                    // vectors of the longest row with one per lane
};
// Forward, rows of more than twelve waves leave room for one block per CU, whose phases nothing
// overlaps: two vectors per lane there make two blocks, 4096 x 7168 in 57.3 us instead of 64.0, 8192
// columns 64.1 instead of 66.0; but 5120 columns 51.4 instead of 40.3. Backward the second vector
// does not fit the registers: 8192 columns in 117 us instead of 69.
constexpr Blocks kFwdBlocks = {256, 192, 320, 768}, kBwdBlocks = {512, 256, 448, 1024};

// Groups are taken where they leave fewer lanes idle, and at most one in twelve. They cost vector
// registers for addresses and a reduction across waves. In 16.8 M elements with checkpoints rows of
// 384 columns (3 groups in 4 groups' lanes before) take 33.6 us forward against 35.7 with whole
// waves, of 640 33.8 against 38.5, 768 33.5 against 36.0, 1280 33.4 against 35.2; backward 384 37.2
// against 40.4, 640 38.8 against 44.1, 896 37.0 against 39.0, 1152 37.1 against 45.1. Where a block
// does not come out even they lose: 1408 columns forward, 35.6 against 34.0.
Shape shape_of(int64_t cols, const Blocks& b) {
  const int64_t vecs = ceil_div(cols, kVec);
  const int m = static_cast<int>(ceil_div(cols, 128));
  const int in_waves = m <= 4 ? (m == 3 ? 4 : m) : static_cast<int>(ceil_div(m, 4)) * 4;
  if (m < in_waves && m <= 16) {
    Shape s = {kGroups, 1, m, 0, 0};
    double most = 0;  // part of the lanes in use
    for (int t = b.least; t <= b.most; t += 64) {
      const int groups = t / 16, teams = groups / m;
      const double used = double(teams * m) / groups;
      if (used > most) most = used, s.threads = t, s.teams = teams;
    }
    if (most > double(m) / in_waves && most > 0.91) return s;
  }
  Shape s = {kWaves, 1, 0, b.threads, 0};
  if (vecs <= 64) {
    s.lanes = cols < kVec ? kOne : vecs <= 16 ? 16 : vecs <= 32 ? 32 : 64;
    s.teams = s.threads / std::max(s.lanes, 16);
    return s;
  }
  s.nv = vecs <= b.one ? 1 : 2;
  s.wpt = static_cast<int>(ceil_div(vecs, 64 * s.nv));
  s.teams = std::max(1, b.threads / (64 * s.wpt));
  s.threads = 64 * s.wpt * s.teams;
  return s;
}

bool gate_ok(int kind) { return kind >= PURO_GATE_NONE && kind <= PURO_GATE_FULL; }
bool res_ok(int type) { return type == PURO_TYPE_BF16 || type == PURO_TYPE_FP32; }
bool norm_dims_ok(int64_t rows, int64_t cols) {
  return any_dim_ok(rows) && cols >= 0 && cols <= PURO_NORM_MAX_COLS;
}

// Blocks, and steps of one row per team for each. A block keeps its weights (and column sums) over
// consecutive rows, so the grid is what the chip holds at once: `waves` per CU, which the kernel's
// registers allow, in whole blocks. Steps are dealt out evenly, the first `more` blocks taking one
// more, so that the CUs, which get every 256th block, differ by a step at most (blocks of equal
// length left some CUs a block's length ahead of others: 896 columns forward 42.5 -> 34.3 us, 1152
// backward 55.9 -> 45.1); and only as many CUs are used as the busiest one's steps ask for, which
// saves partial sums.
constexpr int kCus = 256;
struct Split {
  int blocks, steps, more;
};
Split split_rows(int64_t rows, const Shape& s, int waves, int most_blocks) {
  const int64_t steps = ceil_div(rows, s.teams);
  const int per_cu = std::min(most_blocks / kCus, std::max(1, waves / (s.threads / 64)));
  const int64_t cus = ceil_div(steps, ceil_div(steps, kCus));
  Split p;
  p.blocks = static_cast<int>(std::min(steps, per_cu * cus));
  p.steps = static_cast<int>(steps / p.blocks);
  p.more = static_cast<int>(steps % p.blocks);
  return p;
}
constexpr int kBwdWaves = 16;
// Forward: as many waves as the registers allow, but 16 (where blocks make 16) for rows of a
// multiple of 4 KB in bf16. That is a rule by measurement, with both norms; what causes it was not
// found: 8192 x 2048 32.2 us against 33.5 with 24, in fp32 47.9 against 50.9, 4096 x 4096 31.6
// against 33.4; but 1792 columns 35.6 against 34.3, and 6144 columns, where it would be 12 waves,
// 55.8 against 47.6. The norm before a block alone, which has one load per lane in flight where
// the two norms have two, takes 20.2 us at 8192 x 2048 under it, 3.4 TB/s.
int fwd_waves(const Shape& s, int64_t cols) {
  if (s.nv == 2 || s.lanes == kGroups) return 16;
  if (cols % 2048 == 0 && 16 % (s.threads / 64) == 0) return 16;
  return s.lanes == kWaves || s.lanes == 64 ? 24 : 20;
}

template <typename R>
void launch_fwd(const FwdArgs& a, const Shape& s, int blocks, hipStream_t st) {
  const auto k = s.lanes == kOne      ? norm_fwd_kernel<R, kOne, 1>
                 : s.lanes == kGroups ? norm_fwd_kernel<R, kGroups, 1>
                 : s.lanes == 16      ? norm_fwd_kernel<R, 16, 1>
                 : s.lanes == 32      ? norm_fwd_kernel<R, 32, 1>
                 : s.lanes == 64      ? norm_fwd_kernel<R, 64, 1>
                 : s.nv == 1          ? norm_fwd_kernel<R, kWaves, 1>
                                      : norm_fwd_kernel<R, kWaves, 2>;
  hipLaunchKernelGGL(k, dim3(blocks), dim3(s.threads), 0, st, a);
}

template <typename R, bool kCodes>
void launch_bwd(const BwdArgs& a, const Shape& s, int blocks, hipStream_t st) {
  const dim3 grid(blocks), block(s.threads);
  // two accumulators of the teams (of the waves, for teams within one) as whole rows
  const bool cross = s.lanes == kWaves || s.lanes == kGroups;
  const int rows = cross ? s.teams : s.threads / 64;
  const int lanes = s.lanes == kWaves    ? s.wpt * 64
                    : s.lanes == kGroups ? s.wpt * 16
                                         : std::max(s.lanes, 16);
  const size_t lds = rows > 1 ? size_t(2) * rows * lanes * kVec * sizeof(float) : 0;
  const auto k = s.lanes == kOne      ? norm_bwd_kernel<R, kOne, 1, kCodes>
                 : s.lanes == kGroups ? norm_bwd_kernel<R, kGroups, 1, kCodes>
                 : s.lanes == 16      ? norm_bwd_kernel<R, 16, 1, kCodes>
                 : s.lanes == 32      ? norm_bwd_kernel<R, 32, 1, kCodes>
                 : s.lanes == 64      ? norm_bwd_kernel<R, 64, 1, kCodes>
                 : s.nv == 1          ? norm_bwd_kernel<R, kWaves, 1, kCodes>
                                      : norm_bwd_kernel<R, kWaves, 2, kCodes>;
  hipLaunchKernelGGL(k, grid, block, lds, st, a);
}

// A pair of code and scale pointers: both or neither.
puro_status check_pair(const void* q, const float* s) {
  if (q == nullptr && s == nullptr) return PURO_OK;
  PURO_TRY(check_ptr(q, false));
  return check_ptr(s, false);
}

}  // namespace
}  // namespace puro

using namespace puro;

extern "C" puro_status puro_block_norm_fwd(const puro_block_norm* d, void* stream) {
  if (d == nullptr) return PURO_ERR_NULL;
  if (!norm_dims_ok(d->rows, d->cols)) return PURO_ERR_SHAPE;
  if (!gate_ok(d->gate_kind) || !res_ok(d->residual_type) || (d->pow2 != 0 && d->pow2 != 1))
    return PURO_ERR_ARG;
  if (!std::isfinite(d->alpha) || !std::isfinite(d->beta) || !std::isfinite(d->eps) ||
      !(d->eps > 0))
    return PURO_ERR_ARG;
  if (d->cols == 0) return PURO_OK;  // empty tensors, whose addresses may all be NULL
  const bool post = d->w_post != nullptr, pre = d->w_pre != nullptr;
  if (!post && (d->gate_kind != PURO_GATE_NONE || d->y || d->yq || d->ys)) return PURO_ERR_ARG;
  if (!pre && (d->n || d->nq || d->ns)) return PURO_ERR_ARG;
  if (d->rows == 0) return PURO_OK;
  if (!post && !pre) return PURO_ERR_NULL;
  PURO_TRY(check_ptr(d->r, false));
  PURO_TRY(check_optional(d->r_out));
  if (post) {
    if (d->r_out == nullptr) return PURO_ERR_NULL;
    PURO_TRY(check_ptr(d->y, false));
    PURO_TRY(check_ptr(d->w_post, false));
    PURO_TRY(check_ptr(d->rstd_y, false));
    if (d->gate_kind != PURO_GATE_NONE) PURO_TRY(check_ptr(d->gate, false));
  }
  if (pre) {
    PURO_TRY(check_ptr(d->w_pre, false));
    PURO_TRY(check_ptr(d->rstd_r, false));
    if (d->n == nullptr && d->nq == nullptr) return PURO_ERR_NULL;
    PURO_TRY(check_optional(d->n));
  }
  PURO_TRY(check_pair(d->nq, d->ns));
  PURO_TRY(check_pair(d->yq, d->ys));
  PURO_TRY(check_pair(d->rq, d->rs));

  const Shape s = shape_of(d->cols, kFwdBlocks);
  FwdArgs a = {static_cast<const uint16_t*>(d->y), d->r, d->w_post, d->w_pre, d->gate,
               d->gate_kind, d->pow2, d->rows, static_cast<int>(d->cols), s.wpt, 0, 0, d->alpha,
               d->beta, d->eps, d->r_out, static_cast<uint16_t*>(d->n),
               static_cast<uint8_t*>(d->nq), d->ns, d->rstd_y, d->rstd_r,
               static_cast<uint8_t*>(d->yq), d->ys, static_cast<uint8_t*>(d->rq), d->rs};
  const Split p = split_rows(d->rows, s, fwd_waves(s, d->cols), INT32_MAX);
  a.steps = p.steps, a.more = p.more;
  if (d->residual_type == PURO_TYPE_BF16)
    launch_fwd<uint16_t>(a, s, p.blocks, static_cast<hipStream_t>(stream));
  else
    launch_fwd<float>(a, s, p.blocks, static_cast<hipStream_t>(stream));
  return launch_status();
}

extern "C" int64_t puro_block_norm_workspace(int64_t rows, int64_t cols) {
  if (!norm_dims_ok(rows, cols) || rows == 0 || cols == 0) return 0;
  const Shape s = shape_of(cols, kBwdBlocks);
  const Split p = split_rows(rows, s, kBwdWaves, PURO_NORM_MAX_BLOCKS);
  return int64_t(p.blocks) * 2 * cols * sizeof(float);
}

extern "C" puro_status puro_block_norm_bwd(const puro_block_norm_grad* d, void* workspace,
                                           void* stream) {
  if (d == nullptr) return PURO_ERR_NULL;
  if (!norm_dims_ok(d->rows, d->cols)) return PURO_ERR_SHAPE;
  if (!gate_ok(d->gate_kind) || !res_ok(d->residual_type) ||
      (d->accumulate != 0 && d->accumulate != 1))
    return PURO_ERR_ARG;
  if (!std::isfinite(d->alpha) || !std::isfinite(d->beta)) return PURO_ERR_ARG;
  const bool empty = d->rows == 0;
  if (d->cols == 0) {  // empty tensors, whose addresses may all be NULL
    if (empty || d->gate_kind != PURO_GATE_TOKEN) return PURO_OK;
    PURO_TRY(check_ptr(d->dgate, false));
    hipLaunchKernelGGL(zero_kernel, dim3(static_cast<uint32_t>(ceil_div(d->rows, 256))), dim3(256),
                       0, static_cast<hipStream_t>(stream), static_cast<float*>(d->dgate), d->rows);
    return launch_status();
  }
  const bool post = d->w_post != nullptr, pre = d->w_pre != nullptr;
  if (!post && (d->gate_kind != PURO_GATE_NONE || d->y || d->yq || d->dy || d->dw_post))
    return PURO_ERR_ARG;
  if (!pre && (d->dn || d->r || d->rq || d->dw_pre)) return PURO_ERR_ARG;
  if ((d->y && d->yq) || (d->r && d->rq)) return PURO_ERR_ARG;
  if (!empty) {
    if (!post && !pre) return PURO_ERR_NULL;
    if (!pre && d->dr_out == nullptr) return PURO_ERR_NULL;
    PURO_TRY(check_optional(d->dr_out));
    PURO_TRY(check_optional(d->dr));
    if (post) {
      if (d->yq == nullptr) PURO_TRY(check_ptr(d->y, false));
      PURO_TRY(check_ptr(d->rstd_y, false));
      PURO_TRY(check_ptr(d->dy, false));
    }
    if (pre) {
      if (d->rq == nullptr) PURO_TRY(check_ptr(d->r, false));
      PURO_TRY(check_ptr(d->dn, false));
      PURO_TRY(check_ptr(d->rstd_r, false));
    }
    PURO_TRY(check_pair(d->yq, d->ys));
    PURO_TRY(check_pair(d->rq, d->rs));
    if ((d->yq && d->r) || (d->y && d->rq)) return PURO_ERR_ARG;  // one form for both
    PURO_TRY(check_ptr(workspace, false));
  }
  if (post) {
    PURO_TRY(check_ptr(d->w_post, false));
    if (d->gate_kind != PURO_GATE_NONE) {
      const bool none = empty && d->gate_kind != PURO_GATE_CHANNEL;
      PURO_TRY(check_ptr(d->gate, none));
      PURO_TRY(check_ptr(d->dgate, none));
    }
  }
  if (pre) PURO_TRY(check_ptr(d->w_pre, false));
  PURO_TRY(check_optional(d->dw_post));
  PURO_TRY(check_optional(d->dw_pre));

  const hipStream_t st = static_cast<hipStream_t>(stream);
  const Shape s = shape_of(d->cols, kBwdBlocks);
  int blocks = 0;
  if (!empty) {
    BwdArgs a = {d->dr_out, static_cast<const uint16_t*>(d->dn),
                 static_cast<const uint16_t*>(d->y), static_cast<const uint8_t*>(d->yq), d->ys,
                 d->r, static_cast<const uint8_t*>(d->rq), d->rs, d->rstd_y, d->rstd_r, d->w_post,
                 d->w_pre, d->gate, d->gate_kind, d->rows, static_cast<int>(d->cols), s.wpt, 0,
                 0, d->alpha, d->beta, d->dr, static_cast<uint16_t*>(d->dy), d->dgate,
                 static_cast<float*>(workspace)};
    const Split p = split_rows(d->rows, s, kBwdWaves, PURO_NORM_MAX_BLOCKS);
    a.steps = p.steps, a.more = p.more;
    blocks = p.blocks;
    const bool codes = d->yq != nullptr || d->rq != nullptr;
    const auto launch = d->residual_type == PURO_TYPE_BF16
                            ? (codes ? launch_bwd<uint16_t, true> : launch_bwd<uint16_t, false>)
                            : (codes ? launch_bwd<float, true> : launch_bwd<float, false>);
    launch(a, s, blocks, st);
    PURO_TRY(launch_status());
  }
  const bool channel = d->gate_kind == PURO_GATE_CHANNEL;
  if (d->dw_post == nullptr && d->dw_pre == nullptr && !channel) return PURO_OK;
  const ReduceArgs ra = {static_cast<const float*>(workspace), blocks, static_cast<int>(d->cols),
                         d->gate_kind, d->accumulate, d->alpha, d->w_post,
                         static_cast<const float*>(d->gate), d->dw_post, d->dw_pre,
                         channel ? static_cast<float*>(d->dgate) : nullptr};
  hipLaunchKernelGGL(norm_reduce_kernel,
                     dim3(static_cast<uint32_t>(ceil_div(d->cols, kRedCols)), 2),
                     dim3(1024), 0, st, ra);
  return launch_status();
}
