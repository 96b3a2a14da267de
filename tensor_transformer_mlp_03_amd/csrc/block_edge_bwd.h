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
// Instantiated by the two .hip files that include this (RMSNorm only, and with a
// LayerNorm on either side, which needs twice the column sums).
#pragma once

#include "block_dev.h"

namespace tpmlp {
namespace edge {

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
// The parameter products stay in registers over all rows for up to two chunks a lane
// and in LDS for more (loads of them between the row's would wait for those).
template <class YT, class RT, bool HAS_Y, bool LAYER, class DXT, int W, int NV, bool FULL, bool NT>
__global__ void __launch_bounds__(W == 1 ? 256 : 64 * W, FULL && NV <= 2 ? 4 : 1) edge_bwd_kernel(EdgeBwdArgs a) {
  constexpr int NACC = LAYER ? EDGE_ACC_LAYER : EDGE_ACC_RMS;
  constexpr bool KEEP = NV <= 2, W_LDS = !KEEP && NV <= 4;
  constexpr int NSUM = LAYER ? 12 : 6;
  constexpr int SLOT = (NSUM + (LAYER ? 2 : 0)) * W;  // floats of one row's sums; two sets, used in turn
  __shared__ float slots[2 * SLOT];
  __shared__ f32x4 v_lds[KEEP ? 1 : NV * 64 * W], w_lds[W_LDS ? NV * 64 * W : 1];
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
  f32x4 wu[KEEP ? NV : 1], wv[KEEP ? NV : 1];
  {
    constexpr int N = KEEP ? NV : 1;
#pragma unroll
    for (int p0 = 0; p0 < NV; p0 += N) {
      auto place = [&](int p) { return at(p0 + p); };
      Params<N, FULL> w1, w2, w3;
      if (has_dx) w1.fetch(a.w_pre, a.p_bf16, 0, place, H);
      if (post) w2.fetch(a.w_post, a.p_bf16, 0, place, H);
      if (HAS_Y && a.gate) w3.fetch(a.gate, a.p_bf16, group * a.ld_gate, place, H);
#pragma unroll
      for (int p = 0; p < N; ++p) {
        const f32x4 w = has_dx ? w1.get(p, a.p_bf16, place(p), H) : zero;
        f32x4 v = post ? w2.get(p, a.p_bf16, place(p), H) : one;
        if (HAS_Y && a.gate) v *= w3.get(p, a.p_bf16, place(p), H);
        if (KEEP) {
          wu[p] = w;
          wv[p] = v;
        } else {
          v_lds[(p0 + p) * 64 * W + lane] = v;
          if (W_LDS) w_lds[(p0 + p) * 64 * W + lane] = w;
        }
      }
    }
  }
  // (each lane reads back only what it wrote)
  auto w_at = [&](int p) {
    return KEEP ? wu[KEEP ? p : 0] : W_LDS ? w_lds[p * 64 * W + lane] : load_params<FULL>(a.w_pre, a.p_bf16, 0, at(p), H);
  };
  auto v_at = [&](int p) { return KEEP ? wv[KEEP ? p : 0] : v_lds[p * 64 * W + lane]; };

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
    // sums of c^2, t c, b^2, dr' v b, t v b, c v b; LayerNorm: t, v b, dr' v, t v, c v, v
    float q[NSUM] = {};
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const f32x4 r = r_at(p), u = u_at(p), d = d_at(p), y = y_at(p), w = w_at(p), v = v_at(p);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool in = FULL ? at(p) < H : at(p) + e < H;
        const float c = LAYER ? (in ? r[e] - mean[0] : 0.0f) : r[e], t = u[e] * w[e];
        q[0] = __builtin_fmaf(c, c, q[0]);
        q[1] = __builtin_fmaf(t, c, q[1]);
        if (LAYER) q[LAYER ? 6 : 0] += t;
        if (HAS_Y) {
          const float b = LAYER ? (in ? y[e] - mean[1] : 0.0f) : y[e], vb = v[e] * b;
          q[2] = __builtin_fmaf(b, b, q[2]);
          q[3] = __builtin_fmaf(d[e], vb, q[3]);
          q[4] = __builtin_fmaf(t, vb, q[4]);
          q[5] = __builtin_fmaf(c, vb, q[5]);
          if (LAYER) {
            q[LAYER ? 7 : 0] += vb;
            q[LAYER ? 8 : 0] = __builtin_fmaf(d[e], v[e], q[LAYER ? 8 : 0]);
            q[LAYER ? 9 : 0] = __builtin_fmaf(t, v[e], q[LAYER ? 9 : 0]);
            q[LAYER ? 10 : 0] = __builtin_fmaf(c, v[e], q[LAYER ? 10 : 0]);
            q[LAYER ? 11 : 0] += v[e];
          }
        }
      }
    }
    row_sum<W>(q, slot, wave);
    // pre: d = dr' + s (t - m - c k) with k = s^2 mean(t c); post: dy = sy (d v - my - b ky)
    float s = 0.0f, k = 0.0f, m = 0.0f, sy = 1.0f, ky = 0.0f, my = 0.0f;
    if (has_dx) {
      s = 1.0f / sqrtf(__builtin_fmaf(q[0], inv, a.eps));
      k = q[1] * inv * s * s;
      m = pre_layer ? q[LAYER ? 6 : 0] * inv : 0.0f;
    }
    if (post) {
      sy = 1.0f / sqrtf(__builtin_fmaf(q[2], inv, a.eps));
      float dvb = q[4] - k * q[5], dv = 0.0f;
      if (LAYER) {
        dvb -= m * q[LAYER ? 7 : 0];
        dv = q[LAYER ? 9 : 0] - k * q[LAYER ? 10 : 0] - m * q[LAYER ? 11 : 0];
        my = post_layer ? __builtin_fmaf(s, dv, q[LAYER ? 8 : 0]) * inv : 0.0f;
      }
      ky = __builtin_fmaf(s, dvb, q[3]) * inv * sy * sy;
    }

    const RR dr(a.dr, row * a.ld_dr, H);
    const Row<BF16, FULL, NT> dyr(a.dy, HAS_Y ? row * a.ld_dy : 0, H);
    const In next = rows_at(row + STEP);
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      f32x4 d = d_at(p);
      if (has_dx) {
        const f32x4 u = u_at(p), c = LAYER ? r_at(p) - mean[0] : r_at(p);
        T1[p] += u * (c * s);
        if (LAYER) T0[p] += u;
        f32x4 g = u * w_at(p) - c * k;
        if (LAYER) g -= m;
        d += g * s;
      }
      const f32x4 y = y_at(p);
      load_chunk(next, p);
      dr.store(at(p), d * a.alpha);
      if (HAS_Y) {
        f32x4 g = d * v_at(p);
        if (post) {
          const f32x4 b = LAYER ? y - mean[1] : y;
          S1[p] += d * (b * sy);
          if (LAYER) S0[p] += d;
          g -= b * ky;
          if (LAYER) g -= my;
          g *= sy;
        } else {
          S1[p] += d * y;
        }
        dyr.store(at(p), g);
      }
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

template <class YT, class RT, bool HAS_Y, bool LAYER, class DXT, bool NT>
hipError_t launch_form(const EdgeBwdArgs& a, int64_t blocks, bool full, hipStream_t s) {
  const dim3 grid((unsigned)blocks);
#define EDGE_FORM(W, NV, FULL, NT_) \
  return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, DXT, W, NV, FULL, NT_>, grid, dim3(W == 1 ? 256 : 64 * W), s, a)
  switch (edge_bwd_shape(a.H, full)) {
    case EDGE_1x2: EDGE_FORM(1, 2, true, NT);
    case EDGE_4x1: EDGE_FORM(4, 1, true, NT);
    case EDGE_4x2: EDGE_FORM(4, 2, true, NT);
    case EDGE_8x2: EDGE_FORM(8, 2, true, NT);
    case EDGE_16x2: EDGE_FORM(16, 2, true, NT);
    // rows this wide are seldom few: one form each
    case EDGE_16x4: EDGE_FORM(16, 4, true, true);
    case EDGE_16x5: EDGE_FORM(16, 5, true, true);
    case EDGE_16x8: EDGE_FORM(16, 8, true, true);
    case EDGE_ANY_4x1: EDGE_FORM(4, 1, false, false);
    case EDGE_ANY_8x2: EDGE_FORM(8, 2, false, false);
    case EDGE_ANY_16x8: EDGE_FORM(16, 8, false, false);
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
