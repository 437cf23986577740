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
// its last output is written; a row belongs to one team of lanes (16, 32 or 64 lanes of a wave for
// short rows, whole waves for longer ones), 8 columns per lane and vector. All statistics and
// sums are fp32; r' is normalised unrounded, so n does not see the residual stream's rounding.
#include <algorithm>
#include <cmath>

#include "block.hpp"

namespace puro {
namespace {

constexpr int kMaxWaves = 16;  // of a block

// Sum over the team of each of kN values. Teams of whole waves go through LDS with one barrier;
// `buf` alternates between calls, so a wave that is already writing the next call's values never
// meets one still reading this call's. kLanes = 0: a team of `wpt` waves.
template <int kLanes, int kN>
__device__ __forceinline__ void team_sum(float (&v)[kN], float (*sh)[kMaxWaves], int wpt) {
  if constexpr (kLanes != 0) {
#pragma unroll
    for (int k = 0; k < kN; ++k) v[k] = lanes_sum<kLanes>(v[k]);
  } else {
    const int wave = threadIdx.x >> 6, w0 = wave - wave % wpt;
#pragma unroll
    for (int k = 0; k < kN; ++k) v[k] = lanes_sum<64>(v[k]);
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < kN; ++k) sh[k][wave] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      float t = sh[k][w0];
      for (int w = 1; w < wpt; ++w) t += sh[k][w0 + w];
      v[k] = t;
    }
  }
}

// The lanes of one team and the rows of one block.
template <int kLanes>
struct Team {
  int lanes, lane, team, teams;
  __device__ __forceinline__ explicit Team(int wpt) {
    lanes = kLanes ? kLanes : wpt * 64;
    team = threadIdx.x / lanes;
    lane = threadIdx.x - team * lanes;
    teams = blockDim.x / lanes;
  }
};

// ------------------------------------------------------------------ forward
struct FwdArgs {
  const uint16_t* y;
  const void* r;
  const float *w_post, *w_pre;
  const void* gate;
  int gate_kind, pow2;
  int64_t rows;
  int cols, wpt, rows_per_block;
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

template <bool kRaw>
__device__ __forceinline__ void store_codes(uint8_t* q, float* s, int64_t row, int64_t rows,
                                            int cols, int col, int n, const float* f, bool pow2) {
  const RowGroups<1> g = row_groups<kRaw, 1>(reinterpret_cast<const float(*)[kVec]>(f), pow2);
  if (n <= 0) return;
  store8(q + row * cols + col, n, encode8(f, g.r[0]));
  if ((threadIdx.x & 15) == 0) s[static_cast<int64_t>(col >> 7) * rows + row] = g.s;
}

template <typename R, int kLanes, int kNV>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void norm_fwd_kernel(const FwdArgs a) {
  __shared__ float sh[2][1][kMaxWaves];
  const Team<kLanes> tm(a.wpt);
  const float inv_d = 1.0f / static_cast<float>(a.cols);
  const bool channel = a.gate_kind == PURO_GATE_CHANNEL;

  float cw[kNV][kVec], pw[kNV][kVec];  // alpha (gate) w_post; w_pre
  int col[kNV], left[kNV];
#pragma unroll
  for (int j = 0; j < kNV; ++j) {
    col[j] = (j * tm.lanes + tm.lane) * kVec;
    left[j] = a.cols - col[j];
    F8 w = {}, g = {};
    if (a.w_post) w = load8<false>(a.w_post + col[j], left[j]);
    if (channel) g = load8<false>(static_cast<const float*>(a.gate) + col[j], left[j]);
#pragma unroll
    for (int i = 0; i < kVec; ++i) cw[j][i] = a.alpha * w.f[i] * (channel ? g.f[i] : 1.0f);
    F8 p = {};
    if (a.w_pre) p = load8<false>(a.w_pre + col[j], left[j]);
#pragma unroll
    for (int i = 0; i < kVec; ++i) pw[j][i] = p.f[i];
  }

  const int64_t first = int64_t(blockIdx.x) * a.rows_per_block;
  const int64_t end = min(a.rows, first + a.rows_per_block);
  for (int64_t base = first; base < end; base += tm.teams) {  // the same count for every team
    const int64_t row = base + tm.team;
    const bool in = row < end;
    float t[kNV][kVec];
    {
      F8 y[kNV], r[kNV];
      int n[kNV];
#pragma unroll
      for (int j = 0; j < kNV; ++j) {
        n[j] = in ? left[j] : 0;
        if (a.y) y[j] = load8<true>(a.y + row * a.cols + col[j], n[j]);
        r[j] = load8<true>(static_cast<const R*>(a.r) + row * a.cols + col[j], n[j]);
      }
      float ry = 0.0f;
      if (a.y) {
        float ss[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < kNV; ++j)
#pragma unroll
          for (int i = 0; i < kVec; ++i) ss[0] = fmaf(y[j].f[i], y[j].f[i], ss[0]);
        team_sum<kLanes, 1>(ss, sh[0], a.wpt);
        ry = rsqrtf(fmaf(ss[0], inv_d, a.eps));
        if (in && tm.lane == 0) a.rstd_y[row] = ry;
        if (a.yq)
#pragma unroll
          for (int j = 0; j < kNV; ++j)
            store_codes<true>(a.yq, a.ys, row, a.rows, a.cols, col[j], n[j], y[j].f, a.pow2 != 0);
      }
      float gt = 1.0f;
      if (a.gate_kind == PURO_GATE_TOKEN && in) gt = static_cast<const float*>(a.gate)[row];
#pragma unroll
      for (int j = 0; j < kNV; ++j) {
        F8 g;
        if (a.gate_kind == PURO_GATE_FULL)
          g = load8<true>(static_cast<const uint16_t*>(a.gate) + row * a.cols + col[j], n[j]);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          float p = 0.0f;
          if (a.y) {
            p = y[j].f[i] * ry * cw[j][i] * gt;
            if (a.gate_kind == PURO_GATE_FULL) p *= g.f[i];
          }
          t[j][i] = fmaf(a.beta, r[j].f[i], p);
        }
        if (a.r_out) store8(static_cast<R*>(a.r_out) + row * a.cols + col[j], n[j], t[j]);
        if (a.rq)
          store_codes<false>(a.rq, a.rs, row, a.rows, a.cols, col[j], n[j], t[j], a.pow2 != 0);
      }
    }
    if (!a.w_pre) {
      if constexpr (kLanes == 0) __syncthreads();  // before sh[0] is written again
      continue;
    }
    float ss[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < kNV; ++j)
#pragma unroll
      for (int i = 0; i < kVec; ++i) ss[0] = fmaf(t[j][i], t[j][i], ss[0]);
    team_sum<kLanes, 1>(ss, sh[1], a.wpt);
    const float rr = rsqrtf(fmaf(ss[0], inv_d, a.eps));
    if (in && tm.lane == 0) a.rstd_r[row] = rr;
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
      const int n = in ? left[j] : 0;
      float o[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) o[i] = t[j][i] * rr * pw[j][i];
      if (a.n) store8(a.n + row * a.cols + col[j], n, o);
      if (a.nq) store_codes<false>(a.nq, a.ns, row, a.rows, a.cols, col[j], n, o, a.pow2 != 0);
    }
    if (kLanes == 0 && !a.y) __syncthreads();  // before sh[1] is written again
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
  int cols, wpt, rows_per_block;
  float alpha, beta;
  void* dr;
  uint16_t* dy;
  void* dgate;       // per row or per element; per column through the partial sums
  float* partials;   // [blocks][2][cols]: sums of g yh G and of dn rh
};

template <typename R, int kLanes, int kNV>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void norm_bwd_kernel(const BwdArgs a) {
  __shared__ float sh[2][3][kMaxWaves];
  const Team<kLanes> tm(a.wpt);
  const float inv_d = 1.0f / static_cast<float>(a.cols);
  const bool channel = a.gate_kind == PURO_GATE_CHANNEL;
  const bool post = a.w_post != nullptr, pre = a.w_pre != nullptr;

  float wo[kNV][kVec], wp[kNV][kVec], gc[kNV][kVec];
  float acc[2][kNV][kVec] = {};
  int col[kNV], left[kNV];
#pragma unroll
  for (int j = 0; j < kNV; ++j) {
    col[j] = (j * tm.lanes + tm.lane) * kVec;
    left[j] = a.cols - col[j];
    F8 w = {}, p = {}, g = {};
    if (post) w = load8<false>(a.w_post + col[j], left[j]);
    if (pre) p = load8<false>(a.w_pre + col[j], left[j]);
    if (channel) g = load8<false>(static_cast<const float*>(a.gate) + col[j], left[j]);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      wo[j][i] = w.f[i];
      wp[j][i] = p.f[i];
      gc[j][i] = channel ? g.f[i] : 1.0f;
    }
  }

  const int64_t first = int64_t(blockIdx.x) * a.rows_per_block;
  const int64_t end = min(a.rows, first + a.rows_per_block);
  int buf = 0;
  for (int64_t base = first; base < end; base += tm.teams, buf ^= 1) {
    const int64_t row = base + tm.team;
    const bool in = row < end;
    float A[kNV][kVec], yh[kNV][kVec], rh[kNV][kVec], g[kNV][kVec];
    float sums[3] = {0.0f, 0.0f, 0.0f};
    const float ry = post && in ? a.rstd_y[row] : 0.0f;
    const float rr = pre && in ? a.rstd_r[row] : 0.0f;
    float gt = 1.0f;
    if (a.gate_kind == PURO_GATE_TOKEN && in) gt = static_cast<const float*>(a.gate)[row];
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
      const int n = in ? left[j] : 0;
      const int64_t at = row * a.cols + col[j];
      const int64_t sat = static_cast<int64_t>(col[j] >> 7) * a.rows + row;
      F8 d = {}, dn = {}, y = {}, r = {};
      if (a.dr_out) d = load8<true>(static_cast<const R*>(a.dr_out) + at, n);
      if (pre) {
        dn = load8<true>(a.dn + at, n);
        if (a.rq)
          decode8(load_raw<true>(a.rq + at, n), n > 0 ? a.rs[sat] : 0.0f, r.f);
        else
          r = load8<true>(static_cast<const R*>(a.r) + at, n);
      }
      if (post) {
        if (a.yq)
          decode8(load_raw<true>(a.yq + at, n), n > 0 ? a.ys[sat] : 0.0f, y.f);
        else
          y = load8<true>(a.y + at, n);
      }
      F8 ge;
      if (a.gate_kind == PURO_GATE_FULL)
        ge = load8<true>(static_cast<const uint16_t*>(a.gate) + at, n);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        g[j][i] = a.gate_kind == PURO_GATE_FULL ? ge.f[i] : gc[j][i];
        yh[j][i] = y.f[i] * ry;
        rh[j][i] = r.f[i] * rr;
        const float x = wp[j][i] * dn.f[i];
        A[j][i] = fmaf(rr, x, d.f[i]);
        sums[0] = fmaf(rh[j][i], x, sums[0]);
        const float q = yh[j][i] * wo[j][i] * g[j][i];
        sums[1] = fmaf(q, A[j][i], sums[1]);
        sums[2] = fmaf(q, rh[j][i], sums[2]);
        acc[1][j][i] = fmaf(dn.f[i], rh[j][i], acc[1][j][i]);
      }
    }
    team_sum<kLanes, 3>(sums, sh[buf], a.wpt);
    const float k1 = rr * sums[0] * inv_d;
    const float qg = sums[1] - k1 * sums[2];           // sum of q G
    const float k2 = a.alpha * gt * qg * inv_d;
    if (a.gate_kind == PURO_GATE_TOKEN && in && tm.lane == 0)
      static_cast<float*>(a.dgate)[row] = a.alpha * qg;
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
      const int n = in ? left[j] : 0;
      const int64_t at = row * a.cols + col[j];
      float dr[kVec], dy[kVec], dg[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const float G = fmaf(-k1, rh[j][i], A[j][i]);
        const float gg = g[j][i] * gt;
        dr[i] = a.beta * G;
        const float dp = a.alpha * gg * G;
        dy[i] = ry * fmaf(wo[j][i], dp, -k2 * yh[j][i]);
        dg[i] = a.alpha * yh[j][i] * wo[j][i] * G;
        // a channel gate is factored out of the column sum, which then serves dw_post and dgate
        acc[0][j][i] = fmaf(yh[j][i] * (channel ? 1.0f : gg), G, acc[0][j][i]);
      }
      if (a.dr) store8(static_cast<R*>(a.dr) + at, n, dr);
      if (post) {
        store8(a.dy + at, n, dy);
        if (a.gate_kind == PURO_GATE_FULL)
          store8(static_cast<uint16_t*>(a.dgate) + at, n, dg);
      }
    }
  }

  // Column sums of the block: over its teams through LDS, then one partial per block.
  extern __shared__ float red[];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
      if (tm.teams > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kVec; ++i) red[i * blockDim.x + threadIdx.x] = acc[k][j][i];
        __syncthreads();
        if (tm.team == 0)
#pragma unroll
          for (int i = 0; i < kVec; ++i)
            for (int w = 1; w < tm.teams; ++w)
              acc[k][j][i] += red[i * blockDim.x + w * tm.lanes + tm.lane];
      }
      if (tm.team == 0)
        store8(a.partials + (int64_t(blockIdx.x) * 2 + k) * a.cols + col[j], left[j],
               acc[k][j]);
    }
}

// Sum of the block partials per column in a fixed order: 32 columns x 32 rows of threads
// per block, each thread every 32nd partial.
struct ReduceArgs {
  const float* partials;
  int blocks, cols, gate_kind, accumulate;
  float alpha;
  const float *w_post, *gate;
  float *dw_post, *dw_pre, *dgate;
};

constexpr int kRedCols = 32, kRedRows = 32;

__global__ __launch_bounds__(kRedCols* kRedRows) void norm_reduce_kernel(const ReduceArgs a) {
  __shared__ float sh[kRedRows][kRedCols + 1];
  const int c = blockIdx.x * kRedCols + threadIdx.x % kRedCols;
  const int k = blockIdx.y, y = threadIdx.x / kRedCols;
  float t = 0.0f;
  if (c < a.cols)
    for (int b = y; b < a.blocks; b += kRedRows)
      t += a.partials[(int64_t(b) * 2 + k) * a.cols + c];
  sh[y][threadIdx.x % kRedCols] = t;
  __syncthreads();
  if (y != 0 || c >= a.cols) return;
  for (int w = 1; w < kRedRows; ++w) t += sh[w][threadIdx.x];
  if (k == 1) {
    if (a.dw_pre) a.dw_pre[c] = t + (a.accumulate ? a.dw_pre[c] : 0.0f);
    return;
  }
  const bool channel = a.gate_kind == PURO_GATE_CHANNEL;
  if (a.dw_post)
    a.dw_post[c] = a.alpha * (channel ? a.gate[c] : 1.0f) * t +
                   (a.accumulate ? a.dw_post[c] : 0.0f);
  if (channel && a.dgate)
    a.dgate[c] = a.alpha * a.w_post[c] * t + (a.accumulate ? a.dgate[c] : 0.0f);
}

// ------------------------------------------------------------------ host side
// How a row is laid over lanes: 16, 32 or 64 lanes of 8 columns up to 512 columns, then whole
// waves, one vector per lane up to 8192 columns and two beyond.
struct Shape {
  int lanes;     // 16, 32, 64, or 0 for whole waves
  int nv;        // vectors of 8 columns per lane
  int wpt;       // waves per team (whole waves)
  int threads;   // per block
  int teams;     // per block
};

Shape shape_of(int64_t cols, int most_threads) {
  Shape s = {0, 1, 0, 256, 0};
  const int64_t vecs = ceil_div(cols, kVec);
  if (vecs <= 64) {
    s.lanes = vecs <= 16 ? 16 : vecs <= 32 ? 32 : 64;
    s.teams = s.threads / s.lanes;
    return s;
  }
  s.nv = vecs <= 1024 ? 1 : 2;
  s.wpt = static_cast<int>(ceil_div(vecs, 64 * s.nv));
  s.teams = std::max(1, most_threads / (64 * s.wpt));
  s.threads = 64 * s.wpt * s.teams;
  return s;
}

bool gate_ok(int kind) { return kind >= PURO_GATE_NONE && kind <= PURO_GATE_FULL; }
bool res_ok(int type) { return type == PURO_TYPE_BF16 || type == PURO_TYPE_FP32; }
bool norm_dims_ok(int64_t rows, int64_t cols) {
  return any_dim_ok(rows) && cols >= 0 && cols <= PURO_NORM_MAX_COLS;
}

// Blocks and rows per block: enough blocks to fill the chip, each with consecutive rows.
void split_rows(int64_t rows, const Shape& s, int64_t most_blocks, int* per_block, int* blocks) {
  const int64_t steps = ceil_div(rows, s.teams);             // of the whole grid, one team row each
  const int64_t per = std::max<int64_t>(1, ceil_div(steps, most_blocks));
  *per_block = static_cast<int>(per * s.teams);
  *blocks = static_cast<int>(ceil_div(rows, *per_block));
}

constexpr int kBwdBlocks = PURO_NORM_MAX_BLOCKS;

template <typename R>
void launch_fwd(const FwdArgs& a, const Shape& s, int blocks, hipStream_t st) {
  const dim3 grid(blocks), block(s.threads);
  switch (s.lanes) {
    case 16: hipLaunchKernelGGL((norm_fwd_kernel<R, 16, 1>), grid, block, 0, st, a); return;
    case 32: hipLaunchKernelGGL((norm_fwd_kernel<R, 32, 1>), grid, block, 0, st, a); return;
    case 64: hipLaunchKernelGGL((norm_fwd_kernel<R, 64, 1>), grid, block, 0, st, a); return;
  }
  if (s.nv == 1)
    hipLaunchKernelGGL((norm_fwd_kernel<R, 0, 1>), grid, block, 0, st, a);
  else
    hipLaunchKernelGGL((norm_fwd_kernel<R, 0, 2>), grid, block, 0, st, a);
}

template <typename R>
void launch_bwd(const BwdArgs& a, const Shape& s, int blocks, hipStream_t st) {
  const dim3 grid(blocks), block(s.threads);
  const size_t lds = s.teams > 1 ? size_t(s.threads) * kVec * sizeof(float) : 0;
  switch (s.lanes) {
    case 16: hipLaunchKernelGGL((norm_bwd_kernel<R, 16, 1>), grid, block, lds, st, a); return;
    case 32: hipLaunchKernelGGL((norm_bwd_kernel<R, 32, 1>), grid, block, lds, st, a); return;
    case 64: hipLaunchKernelGGL((norm_bwd_kernel<R, 64, 1>), grid, block, lds, st, a); return;
  }
  if (s.nv == 1)
    hipLaunchKernelGGL((norm_bwd_kernel<R, 0, 1>), grid, block, lds, st, a);
  else
    hipLaunchKernelGGL((norm_bwd_kernel<R, 0, 2>), grid, block, lds, st, a);
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
  const bool post = d->w_post != nullptr, pre = d->w_pre != nullptr;
  if (!post && (d->gate_kind != PURO_GATE_NONE || d->y || d->yq || d->ys)) return PURO_ERR_ARG;
  if (!pre && (d->n || d->nq || d->ns)) return PURO_ERR_ARG;
  if (d->rows == 0 || d->cols == 0) return PURO_OK;
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

  const Shape s = shape_of(d->cols, 256);
  FwdArgs a = {static_cast<const uint16_t*>(d->y), d->r, d->w_post, d->w_pre, d->gate,
               d->gate_kind, d->pow2, d->rows, static_cast<int>(d->cols), s.wpt, 0, d->alpha,
               d->beta, d->eps, d->r_out, static_cast<uint16_t*>(d->n),
               static_cast<uint8_t*>(d->nq), d->ns, d->rstd_y, d->rstd_r,
               static_cast<uint8_t*>(d->yq), d->ys, static_cast<uint8_t*>(d->rq), d->rs};
  int blocks;
  split_rows(d->rows, s, 2048, &a.rows_per_block, &blocks);
  if (d->residual_type == PURO_TYPE_BF16)
    launch_fwd<uint16_t>(a, s, blocks, static_cast<hipStream_t>(stream));
  else
    launch_fwd<float>(a, s, blocks, static_cast<hipStream_t>(stream));
  return launch_status();
}

extern "C" int64_t puro_block_norm_workspace(int64_t rows, int64_t cols) {
  if (!norm_dims_ok(rows, cols) || rows == 0 || cols == 0) return 0;
  const Shape s = shape_of(cols, 512);
  int per, blocks;
  split_rows(rows, s, kBwdBlocks, &per, &blocks);
  return int64_t(blocks) * 2 * cols * sizeof(float);
}

extern "C" puro_status puro_block_norm_bwd(const puro_block_norm_grad* d, void* workspace,
                                           void* stream) {
  if (d == nullptr) return PURO_ERR_NULL;
  if (!norm_dims_ok(d->rows, d->cols)) return PURO_ERR_SHAPE;
  if (!gate_ok(d->gate_kind) || !res_ok(d->residual_type) ||
      (d->accumulate != 0 && d->accumulate != 1))
    return PURO_ERR_ARG;
  if (!std::isfinite(d->alpha) || !std::isfinite(d->beta)) return PURO_ERR_ARG;
  const bool post = d->w_post != nullptr, pre = d->w_pre != nullptr;
  if (!post && (d->gate_kind != PURO_GATE_NONE || d->y || d->yq || d->dy || d->dw_post))
    return PURO_ERR_ARG;
  if (!pre && (d->dn || d->r || d->rq || d->dw_pre)) return PURO_ERR_ARG;
  if ((d->y && d->yq) || (d->r && d->rq)) return PURO_ERR_ARG;
  if (d->cols == 0) return PURO_OK;
  const bool empty = d->rows == 0;
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
  const Shape s = shape_of(d->cols, 512);
  int blocks = 0;
  if (!empty) {
    BwdArgs a = {d->dr_out, static_cast<const uint16_t*>(d->dn),
                 static_cast<const uint16_t*>(d->y), static_cast<const uint8_t*>(d->yq), d->ys,
                 d->r, static_cast<const uint8_t*>(d->rq), d->rs, d->rstd_y, d->rstd_r, d->w_post,
                 d->w_pre, d->gate, d->gate_kind, d->rows, static_cast<int>(d->cols), s.wpt, 0,
                 d->alpha, d->beta, d->dr, static_cast<uint16_t*>(d->dy), d->dgate,
                 static_cast<float*>(workspace)};
    split_rows(d->rows, s, kBwdBlocks, &a.rows_per_block, &blocks);
    if (d->residual_type == PURO_TYPE_BF16)
      launch_bwd<uint16_t>(a, s, blocks, st);
    else
      launch_bwd<float>(a, s, blocks, st);
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
                     dim3(kRedCols * kRedRows), 0, st, ra);
  return launch_status();
}
