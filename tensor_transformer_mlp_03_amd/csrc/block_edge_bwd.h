// The edge between two blocks, backward.  With u = dx w_pre, xh and s the
// normalised r' and its 1 / deviation, and yh, sy those of y (yh = y, sy = 1
// without a norm after the block):
//
//   d  = dr' + s (u - [mean u] - xh mean(u xh))      ([..]: LayerNorm only)
//   dr = alpha d
//   v  = g d w_post,  dy = sy (v - [mean v] - yh mean(v yh))
//   T1 = sum_rows dx xh = dw_pre,   T0 = sum_rows dx = db_pre
//   S1 = sum_rows d yh, S0 = sum_rows d, for each row of the gate, from which
//   dw_post = sum_g g S1, db_post = sum_g g S0, dgate = w_post S1 + b_post S0.
//
// The statistics of r' and y are recomputed from the rows, which are in registers
// anyway, so the forward saves nothing but the r' that the next block keeps.
//
// A workgroup walks the rows of its chunk, all under one row of the gate, W waves
// to a row as in the forward, and keeps the column sums of its elements in
// registers; at the end it writes them to its slice of the workspace, and the
// finishing kernel adds the slices in their order.  No atomics: the results do
// not depend on timing.
//
// Bound by bandwidth where there are many rows: 32768 x 3584 in float32 478 us with the
// finish, 5.4 TB/s (a plain kernel of four reads and two writes reaches 5.25); 8192 x
// 4096 with LayerNorms 145 us, 5.1 TB/s.  With few rows by latency: 1001 x 1000 with 13
// gate rows 11 + 6 us for 20 MB.
//
// Instantiated by the two .hip files that include this (RMSNorm only, and with a
// LayerNorm on either side, which needs twice the column sums).
#pragma once

#include "block_dev.h"

#include <algorithm>

namespace tpmlp {
namespace edge {

// The sums of a row: c^2, t c, b^2, dr' v b, t v b, c v b, and with a LayerNorm t, v b,
// dr' v, t v, c v, v (c, b, t and v as below).
constexpr int SUMS_RMS = 6, SUMS_LAYER = 12;

template <bool HAS_Y, bool LAYER, int N>
__device__ __forceinline__ void add_sums(float (&q)[N], float r, float u, float d, float y, float w, float v, float mean_r,
                                         float mean_y, bool in) {
  const float c = LAYER ? (in ? r - mean_r : 0.0f) : r, t = u * w;
  q[0] = __builtin_fmaf(c, c, q[0]);
  q[1] = __builtin_fmaf(t, c, q[1]);
  if constexpr (LAYER) q[6] += t;
  if constexpr (HAS_Y) {
    const float b = LAYER ? (in ? y - mean_y : 0.0f) : y, vb = v * b;
    q[2] = __builtin_fmaf(b, b, q[2]);
    q[3] = __builtin_fmaf(d, vb, q[3]);
    q[4] = __builtin_fmaf(t, vb, q[4]);
    q[5] = __builtin_fmaf(c, vb, q[5]);
    if constexpr (LAYER) {
      q[7] += vb;
      q[8] = __builtin_fmaf(d, v, q[8]);
      q[9] = __builtin_fmaf(t, v, q[9]);
      q[10] = __builtin_fmaf(c, v, q[10]);
      q[11] += v;
    }
  }
}

// What the second sweep needs of them:
//   d = dr' + s (t - m - c k) with k = s^2 mean(t c),   dy = sy (d v - my - b ky).
struct RowTerms {
  float s, k, m, sy, ky, my;
};

template <bool LAYER, int N>
__device__ __forceinline__ RowTerms row_terms(const float (&q)[N], float inv, float eps, bool has_dx, bool post,
                                              bool pre_layer, bool post_layer) {
  RowTerms z{0.0f, 0.0f, 0.0f, 1.0f, 0.0f, 0.0f};
  if (has_dx) {
    z.s = 1.0f / sqrtf(__builtin_fmaf(q[0], inv, eps));
    z.k = q[1] * inv * z.s * z.s;
    if constexpr (LAYER) z.m = pre_layer ? q[6] * inv : 0.0f;
  }
  if (post) {
    z.sy = 1.0f / sqrtf(__builtin_fmaf(q[2], inv, eps));
    float dvb = q[4] - z.k * q[5];
    if constexpr (LAYER) {
      dvb -= z.m * q[7];
      z.my = post_layer ? __builtin_fmaf(z.s, q[9] - z.k * q[10] - z.m * q[11], q[8]) * inv : 0.0f;
    }
    z.ky = __builtin_fmaf(z.s, dvb, q[3]) * inv * z.sy * z.sy;
  }
  return z;
}

// One element of the second sweep.
struct Out {
  float d, dy;
};
template <bool LAYER>
__device__ __forceinline__ Out row_out(const RowTerms& z, float c, float u, float d, float b, float w, float v, bool post) {
  float g = __builtin_fmaf(-c, z.k, u * w);
  if (LAYER) g -= z.m;
  d = __builtin_fmaf(g, z.s, d);
  float h = d * v;
  if (post) {  // uniform; without a norm y has no part in dy, not even an infinite one
    h = __builtin_fmaf(-b, z.ky, h);
    if (LAYER) h -= z.my;
    h *= z.sy;
  }
  return Out{d, h};
}

// Rows whose elements a workgroup holds W waves wide and NV chunks deep.
//
// A row is worked on in two sweeps over the registers that its loads filled.  The
// first makes every sum of the row at once.  The sum behind dy depends on d, and d on
// the sums before it, but only linearly: with c = r' - mu, b = y - mu_y, t = u = dx
// w_pre and v = g w_post,
//   sum d v b = sum dr' v b + s (sum t v b - [mean t] sum v b - dot s sum c v b),
// and likewise without b for a LayerNorm's mean.  So a row costs one exchange between
// the waves (a LayerNorm one more, for the means).  The second sweep finishes the row
// chunk by chunk and loads the next row's chunk into the registers it has just
// consumed, so that a row's loads are in flight during the stores and sums before it
// without registers of their own.
//
// The parameter products stay in registers over all rows.  Rows wider than 16 waves
// hold so take the two kernels below.
template <class YT, class RT, bool HAS_Y, bool LAYER, class DXT, int W, int NV, bool FULL, bool NT>
__global__ void __launch_bounds__(W == 1 ? 256 : 64 * W, FULL && NV <= 2 ? 4 : 1) edge_bwd_kernel(EdgeBwdArgs a) {
  constexpr int NACC = LAYER ? EDGE_ACC_LAYER : EDGE_ACC_RMS;
  constexpr int NSUM = LAYER ? SUMS_LAYER : SUMS_RMS;
  constexpr int SLOT = (NSUM + (LAYER ? 2 : 0)) * W;  // floats of one row's sums; two sets, used in turn
  __shared__ float slots[2 * SLOT];
  const int lane = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int H = a.H;
  const float inv = 1.0f / (float)H;
  const int64_t group = blockIdx.x / a.chunks;
  const int chunk = (int)(blockIdx.x % a.chunks);
  // The group's workgroups take its rows in turn, so that those at work at one time
  // read neighbouring rows: with a run of rows each, their addresses are a multiple of
  // the run apart and fall on few memory channels.
  constexpr int LINES = W == 1 ? 4 : 1;  // rows at once
  const int64_t row1 = min((group + 1) * a.gate_rows, a.M), STEP = (int64_t)a.chunks * LINES;
  const int64_t row0 = group * a.gate_rows + (int64_t)chunk * LINES + (W == 1 ? wave : 0);
  const bool has_dx = a.dx != nullptr, has_dr = a.dr_out != nullptr, post = HAS_Y && a.post != TPMLP_NORM_NONE;
  const bool pre_layer = LAYER && a.pre == TPMLP_NORM_LAYER, post_layer = LAYER && a.post == TPMLP_NORM_LAYER;
  auto at = [&](int p) { return 4 * (p * 64 * W + lane); };

  // A row as loaded.
  typedef Row<RT, FULL, NT> RR;
  typedef Row<YT, FULL, NT> RY;
  typedef Row<DXT, FULL, NT> RX;
  typename RR::raw d0[NV], r0[NV];
  typename RY::raw y0[NV];
  typename RX::raw u0[NV];
  // The rows behind a pass over the matrices' row `row`; those that are not there, or
  // lie past the group's end, have no length and read zeros.
  struct In {
    RR r, d;
    RX u;
    RY y;
  };
  const int len_x = has_dx ? H : 0, len_d = has_dr ? H : 0, len_y = HAS_Y ? H : 0;
  auto rows_at = [&](int64_t row) {
    const bool on = row < row1;
    return In{RR(a.r, row * a.ld_r, on ? len_x : 0), RR(a.dr_out, row * a.ld_dr_out, on ? len_d : 0),
              RX(a.dx, row * a.ld_dx, on ? len_x : 0), RY(a.y, row * a.ld_y, on ? len_y : 0)};
  };
  auto load_chunk = [&](const In& in, int p) {
    r0[p] = in.r.load_raw(at(p));
    u0[p] = in.u.load_raw(at(p));
    d0[p] = in.d.load_raw(at(p));
    if (HAS_Y) y0[p] = in.y.load_raw(at(p));
  };
  {
    const In in = rows_at(row0);
#pragma unroll
    for (int p = 0; p < NV; ++p) load_chunk(in, p);
  }

  // w_pre, and v = g w_post
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f}, one = {1.0f, 1.0f, 1.0f, 1.0f};
  f32x4 wu[NV], wv[NV];
  {
    Params<NV, FULL> w1, w2, w3;
    if (has_dx) w1.fetch(a.w_pre, a.p_bf16, 0, at, H);
    if (post) w2.fetch(a.w_post, a.p_bf16, 0, at, H);
    if (HAS_Y && a.gate) w3.fetch(a.gate, a.p_bf16, group * a.ld_gate, at, H);
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      wu[p] = has_dx ? w1.get(p, a.p_bf16, at(p), H) : zero;
      wv[p] = post ? w2.get(p, a.p_bf16, at(p), H) : one;
      if (HAS_Y && a.gate) wv[p] *= w3.get(p, a.p_bf16, at(p), H);
    }
  }

  f32x4 S1[NV], T1[NV], S0[LAYER ? NV : 1], T0[LAYER ? NV : 1];
#pragma unroll
  for (int p = 0; p < NV; ++p) {
    S1[p] = T1[p] = zero;
    if (LAYER) S0[p] = T0[p] = zero;
  }

  int turn = 0;
  for (int64_t row = row0; row < row1; row += STEP, turn ^= 1) {
    float* slot = slots + turn * SLOT;
    auto r_at = [&](int p) { return RR::widen_raw(r0[p], at(p), H); };
    auto u_at = [&](int p) { return RX::widen_raw(u0[p], at(p), H); };
    auto d_at = [&](int p) { return RR::widen_raw(d0[p], at(p), H); };
    auto y_at = [&](int p) { return HAS_Y ? RY::widen_raw(y0[p], at(p), H) : zero; };
    float mean[2] = {0.0f, 0.0f};  // of r' and of y
    if (LAYER) {
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        const f32x4 r = r_at(p), y = y_at(p);
        mean[0] += (r[0] + r[1]) + (r[2] + r[3]);
        mean[1] += (y[0] + y[1]) + (y[2] + y[3]);
      }
      row_sum<W>(mean, slot + NSUM * W, wave);
      mean[0] = pre_layer ? mean[0] * inv : 0.0f;
      mean[1] = post_layer ? mean[1] * inv : 0.0f;
    }
    float q[NSUM] = {};
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const f32x4 r = r_at(p), u = u_at(p), d = d_at(p), y = y_at(p), w = wu[p], v = wv[p];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        add_sums<HAS_Y, LAYER>(q, r[e], u[e], d[e], y[e], w[e], v[e], mean[0], mean[1], FULL ? at(p) < H : at(p) + e < H);
    }
    row_sum<W>(q, slot, wave);
    const RowTerms z = row_terms<LAYER>(q, inv, a.eps, has_dx, post, pre_layer, post_layer);

    const RR dr(a.dr, row * a.ld_dr, H);
    const Row<BF16, FULL, NT> dyr(a.dy, HAS_Y ? row * a.ld_dy : 0, H);
    const In next = rows_at(row + STEP);
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const f32x4 r = r_at(p), u = u_at(p), d0p = d_at(p), y = y_at(p);
      load_chunk(next, p);
      f32x4 d = zero, g = zero;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float c = LAYER ? r[e] - mean[0] : r[e], b = LAYER ? y[e] - mean[1] : y[e];
        const Out o = row_out<LAYER>(z, c, u[e], d0p[e], b, wu[p][e], wv[p][e], post);
        d[e] = o.d;
        g[e] = o.dy;
        T1[p][e] = __builtin_fmaf(u[e], c * z.s, T1[p][e]);
        if (LAYER) T0[p][e] += u[e];
        if (HAS_Y) S1[p][e] = __builtin_fmaf(o.d, b * z.sy, S1[p][e]);
        if (HAS_Y && LAYER) S0[p][e] += o.d;
      }
      dr.store(at(p), d * a.alpha);
      if (HAS_Y) dyr.store(at(p), g);
    }
  }

  if (!a.part) return;
  const int64_t part = (int64_t)blockIdx.x * NACC * H;
  auto sum_of = [&](int k, int p) { return k == 0 ? S1[p] : k == 1 ? T1[p] : k == 2 ? S0[LAYER ? p : 0] : T0[LAYER ? p : 0]; };
  if (W > 1) {
#pragma unroll
    for (int k = 0; k < NACC; ++k) {
      const Row<F32, FULL> m(a.part, part + (int64_t)k * H, H);
#pragma unroll
      for (int p = 0; p < NV; ++p) m.store(at(p), sum_of(k, p));
    }
    return;
  }
  // One wave per row: the workgroup's four waves add their sums, wave 0 first.
  __shared__ f32x4 joint[W == 1 ? 4 * 64 * NV : 1];
#pragma unroll
  for (int k = 0; k < NACC; ++k) {
    __syncthreads();
#pragma unroll
    for (int p = 0; p < NV; ++p) joint[wave * 64 * NV + p * 64 + lane] = sum_of(k, p);
    __syncthreads();
    if (wave == 0) {
      const Row<F32, FULL> m(a.part, part + (int64_t)k * H, H);
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        f32x4 t = joint[p * 64 + lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) t += joint[w * 64 * NV + p * 64 + lane];
        m.store(at(p), t);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Wide rows (H above 8192, or above 4096 where the rows are not FULL): too much for
// the registers of one workgroup, so the two sweeps are two kernels.  The first
// makes a row's sums and keeps the six or eight numbers that come of them; the
// second, a thread to four columns, walks the rows of its chunk with them.  It reads
// the inputs once more, but neither kernel waits for anything but memory.  2048 x 20480:
// 277 us (176 at the rate of one reading); the one-kernel form took 338 with its spills, 410
// with the next row in flight and more of them, and 1060 us for 2048 x 20001, which takes
// 333.  The second kernel takes the rows in the first's order, which evicts what the cache
// still holds before it is reached; bands of rows or the reverse order were not tried.
// ---------------------------------------------------------------------------
constexpr int WIDE_THREADS = 1024, WIDE_COLS = 1024;  // columns of one workgroup of the second kernel

template <class YT, class RT, bool HAS_Y, bool LAYER, class DXT, bool FULL>
__global__ void __launch_bounds__(WIDE_THREADS) edge_wide_sums_kernel(EdgeBwdArgs a) {
  constexpr int W = WIDE_THREADS / 64, NSUM = LAYER ? SUMS_LAYER : SUMS_RMS;
  __shared__ float slots[(NSUM + 2) * W];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), H = a.H;
  const float inv = 1.0f / (float)H;
  const int64_t row = a.first_row + blockIdx.x;
  const bool has_dx = a.dx != nullptr, has_dr = a.dr_out != nullptr, post = HAS_Y && a.post != TPMLP_NORM_NONE;
  const bool pre_layer = LAYER && a.pre == TPMLP_NORM_LAYER, post_layer = LAYER && a.post == TPMLP_NORM_LAYER;
  const Row<RT, FULL> r(a.r, row * a.ld_r, has_dx ? H : 0), d(a.dr_out, row * a.ld_dr_out, has_dr ? H : 0);
  const Row<DXT, FULL> u(a.dx, row * a.ld_dx, has_dx ? H : 0);
  const Row<YT, FULL> y(a.y, row * a.ld_y, HAS_Y ? H : 0);
  const int64_t gate_at = a.gate ? row / a.gate_rows * a.ld_gate : 0;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f}, one = {1.0f, 1.0f, 1.0f, 1.0f};
  float mean[2] = {0.0f, 0.0f};
  if (LAYER) {
#pragma unroll 4
    for (int i = 4 * (int)threadIdx.x; i < H; i += 4 * WIDE_THREADS) {
      const f32x4 rv = r.load(i), yv = HAS_Y ? y.load(i) : zero;
      mean[0] += (rv[0] + rv[1]) + (rv[2] + rv[3]);
      mean[1] += (yv[0] + yv[1]) + (yv[2] + yv[3]);
    }
    row_sum<W>(mean, slots + NSUM * W, wave);
    mean[0] = pre_layer ? mean[0] * inv : 0.0f;
    mean[1] = post_layer ? mean[1] * inv : 0.0f;
  }
  float q[NSUM] = {};
#pragma unroll 2
  for (int i = 4 * (int)threadIdx.x; i < H; i += 4 * WIDE_THREADS) {
    const f32x4 rv = r.load(i), uv = u.load(i), dv = d.load(i), yv = HAS_Y ? y.load(i) : zero;
    const f32x4 w = has_dx ? load_params<FULL>(a.w_pre, a.p_bf16, 0, i, H) : zero;
    f32x4 v = post ? load_params<FULL>(a.w_post, a.p_bf16, 0, i, H) : one;
    if (HAS_Y && a.gate) v *= load_params<FULL>(a.gate, a.p_bf16, gate_at, i, H);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      add_sums<HAS_Y, LAYER>(q, rv[e], uv[e], dv[e], yv[e], w[e], v[e], mean[0], mean[1], FULL || i + e < H);
  }
  row_sum<W>(q, slots, wave);
  if (threadIdx.x == 0) {
    const RowTerms z = row_terms<LAYER>(q, inv, a.eps, has_dx, post, pre_layer, post_layer);
    float* t = a.terms + 8 * row;
    *reinterpret_cast<f32x4*>(t) = f32x4{z.s, z.k, z.m, z.sy};
    *reinterpret_cast<f32x4*>(t + 4) = f32x4{z.ky, z.my, mean[0], mean[1]};
  }
}

template <class YT, class RT, bool HAS_Y, bool LAYER, class DXT, bool FULL>
__global__ void __launch_bounds__(WIDE_COLS / 4) edge_wide_kernel(EdgeBwdArgs a) {
  constexpr int NACC = LAYER ? EDGE_ACC_LAYER : EDGE_ACC_RMS;
  const int H = a.H, tiles = (H + WIDE_COLS - 1) / WIDE_COLS;
  const int64_t slice = blockIdx.x / tiles, group = slice / a.chunks;
  const int i = (int)(blockIdx.x % tiles) * WIDE_COLS + 4 * (int)threadIdx.x;
  if (i >= H) return;
  const int64_t row1 = min((group + 1) * a.gate_rows, a.M), row0 = group * a.gate_rows + slice % a.chunks;
  const bool has_dx = a.dx != nullptr, has_dr = a.dr_out != nullptr, post = HAS_Y && a.post != TPMLP_NORM_NONE;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f}, one = {1.0f, 1.0f, 1.0f, 1.0f};
  const f32x4 w = has_dx ? load_params<FULL>(a.w_pre, a.p_bf16, 0, i, H) : zero;
  f32x4 v = post ? load_params<FULL>(a.w_post, a.p_bf16, 0, i, H) : one;
  if (HAS_Y && a.gate) v *= load_params<FULL>(a.gate, a.p_bf16, group * a.ld_gate, i, H);
  f32x4 S1 = zero, T1 = zero, S0 = zero, T0 = zero;
#pragma unroll 2
  for (int64_t row = row0; row < row1; row += a.chunks) {
    const float* t = a.terms + 8 * row;
    const RowTerms z{t[0], t[1], t[2], t[3], t[4], t[5]};
    const f32x4 r = Row<RT, FULL, true>(a.r, row * a.ld_r, has_dx ? H : 0).load(i);
    const f32x4 u = Row<DXT, FULL, true>(a.dx, row * a.ld_dx, has_dx ? H : 0).load(i);
    const f32x4 d0 = Row<RT, FULL, true>(a.dr_out, row * a.ld_dr_out, has_dr ? H : 0).load(i);
    const f32x4 y = Row<YT, FULL, true>(a.y, row * a.ld_y, HAS_Y ? H : 0).load(i);
    f32x4 d = zero, g = zero;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float c = LAYER ? r[e] - t[6] : r[e], b = LAYER ? y[e] - t[7] : y[e];
      const Out o = row_out<LAYER>(z, c, u[e], d0[e], b, w[e], v[e], post);
      d[e] = o.d;
      g[e] = o.dy;
      T1[e] = __builtin_fmaf(u[e], c * z.s, T1[e]);
      if (LAYER) T0[e] += u[e];
      if (HAS_Y) S1[e] = __builtin_fmaf(o.d, b * z.sy, S1[e]);
      if (HAS_Y && LAYER) S0[e] += o.d;
    }
    Row<RT, FULL, true>(a.dr, row * a.ld_dr, H).store(i, d * a.alpha);
    if (HAS_Y) Row<BF16, FULL, true>(a.dy, row * a.ld_dy, H).store(i, g);
  }
  if (!a.part) return;
  const int64_t part = slice * NACC * H;
  Row<F32, FULL>(a.part, part, H).store(i, S1);
  Row<F32, FULL>(a.part, part + H, H).store(i, T1);
  if (LAYER) {
    Row<F32, FULL>(a.part, part + 2 * (int64_t)H, H).store(i, S0);
    Row<F32, FULL>(a.part, part + 3 * (int64_t)H, H).store(i, T0);
  }
}

template <class YT, class RT, bool HAS_Y, bool LAYER, class DXT, bool FULL>
hipError_t launch_wide(const EdgeBwdArgs& a, int64_t slices, hipStream_t s) {
  const int64_t blocks = slices * ((a.H + WIDE_COLS - 1) / WIDE_COLS);
  if (!a.terms || !block_grid_ok(blocks, WIDE_COLS / 4)) return hipErrorInvalidConfiguration;
  EdgeBwdArgs b = a;
  for (b.first_row = 0; b.first_row < a.M; b.first_row += BLOCK_LAUNCH_ROWS) {
    const int64_t rows = std::min(BLOCK_LAUNCH_ROWS, a.M - b.first_row);
    const hipError_t e = launch_kernel(edge_wide_sums_kernel<YT, RT, HAS_Y, LAYER, DXT, FULL>, dim3((unsigned)rows),
                                       dim3(WIDE_THREADS), s, b);
    if (e != hipSuccess) return e;
  }
  return launch_kernel(edge_wide_kernel<YT, RT, HAS_Y, LAYER, DXT, FULL>, dim3((unsigned)blocks), dim3(WIDE_COLS / 4), s, a);
}

template <class YT, class RT, bool HAS_Y, bool LAYER, class DXT, bool NT>
hipError_t launch_form(const EdgeBwdArgs& a, int64_t blocks, bool full, hipStream_t s) {
  const dim3 grid((unsigned)blocks);
#define EDGE_FORM(W, NV, FULL, NT_) \
  return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, DXT, W, NV, FULL, NT_>, grid, dim3(W == 1 ? 256 : 64 * W), s, a)
  switch (edge_bwd_shape(a.H, full)) {
    case EDGE_1x1: EDGE_FORM(1, 1, true, NT);
    case EDGE_1x2: EDGE_FORM(1, 2, true, NT);
    case EDGE_4x1: EDGE_FORM(4, 1, true, NT);
    case EDGE_4x2: EDGE_FORM(4, 2, true, NT);
    case EDGE_8x2: EDGE_FORM(8, 2, true, NT);
    case EDGE_16x2: EDGE_FORM(16, 2, true, NT);
    case EDGE_WIDE: return launch_wide<YT, RT, HAS_Y, LAYER, DXT, true>(a, blocks, s);
    case EDGE_ANY_1x1: EDGE_FORM(1, 1, false, false);
    case EDGE_ANY_1x2: EDGE_FORM(1, 2, false, false);
    case EDGE_ANY_4x1: EDGE_FORM(4, 1, false, false);
    case EDGE_ANY_8x2: EDGE_FORM(8, 2, false, false);
    case EDGE_ANY_WIDE: return launch_wide<YT, RT, HAS_Y, LAYER, DXT, false>(a, blocks, s);
  }
#undef EDGE_FORM
  return hipErrorInvalidValue;
}

template <class YT, class RT, bool HAS_Y, bool LAYER>
hipError_t launch_shape(const EdgeBwdArgs& a, int64_t blocks, bool full, hipStream_t s) {
  if (a.dx_bf16)
    return a.nt ? launch_form<YT, RT, HAS_Y, LAYER, BF16, true>(a, blocks, full, s)
                : launch_form<YT, RT, HAS_Y, LAYER, BF16, false>(a, blocks, full, s);
  return a.nt ? launch_form<YT, RT, HAS_Y, LAYER, F32, true>(a, blocks, full, s)
              : launch_form<YT, RT, HAS_Y, LAYER, F32, false>(a, blocks, full, s);
}

template <bool LAYER>
hipError_t launch_types(const EdgeBwdArgs& a, int64_t blocks, int y_type, int r_type, bool full, hipStream_t s) {
  const bool rb = r_type == TPMLP_BF16;
  if (y_type < 0)
    return rb ? launch_shape<F32, BF16, false, LAYER>(a, blocks, full, s) : launch_shape<F32, F32, false, LAYER>(a, blocks, full, s);
  if (y_type == TPMLP_BF16)
    return rb ? launch_shape<BF16, BF16, true, LAYER>(a, blocks, full, s) : launch_shape<BF16, F32, true, LAYER>(a, blocks, full, s);
  return rb ? launch_shape<F32, BF16, true, LAYER>(a, blocks, full, s) : launch_shape<F32, F32, true, LAYER>(a, blocks, full, s);
}

}  // namespace edge

// Defined by the two instantiating files.
hipError_t launch_edge_bwd_rms(const EdgeBwdArgs& a, int64_t blocks, int y_type, int r_type, bool full, hipStream_t s);
hipError_t launch_edge_bwd_layer(const EdgeBwdArgs& a, int64_t blocks, int y_type, int r_type, bool full, hipStream_t s);

}  // namespace tpmlp
