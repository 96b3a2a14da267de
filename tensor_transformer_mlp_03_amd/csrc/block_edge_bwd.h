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

// Rows whose elements a workgroup holds W waves wide and NV chunks deep.  Up to two
// chunks a lane, the two parameter products stay in registers over all rows; with
// four or more (wider rows than 16 waves hold in two) they are read again for every
// row, and T1, which one lane alone adds to, lives in LDS.  Where the registers allow
// it without losing a resident workgroup, a row's loads are issued before the row
// before it is worked on, so that they are in flight during its sums and barriers.
template <class YT, class RT, bool HAS_Y, bool LAYER, class DXT, int W, int NV, bool FULL>
__global__ void __launch_bounds__(W == 1 ? 256 : 64 * W) edge_bwd_kernel(EdgeBwdArgs a) {
  constexpr int NACC = LAYER ? EDGE_ACC_LAYER : EDGE_ACC_RMS;
  constexpr bool KEEP = NV <= 2, AHEAD = NV == 1 || (NV == 2 && !LAYER), T_LDS = W == 16 && NV >= 4;
  constexpr int SLOT = 8 * W;  // floats of one row's sums; two sets, used in turn
  __shared__ float slots[2 * SLOT];
  __shared__ f32x4 t_lds[T_LDS ? NV * 64 * W : 1];
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
  const int64_t row0 = group * a.gate_rows + (int64_t)chunk * LINES;
  const int64_t gate_at = group * a.ld_gate;
  const bool has_dx = a.dx != nullptr, post = HAS_Y && a.post != TPMLP_NORM_NONE;
  const bool pre_layer = LAYER && a.pre == TPMLP_NORM_LAYER, post_layer = LAYER && a.post == TPMLP_NORM_LAYER;
  auto at = [&](int p) { return 4 * (p * 64 * W + lane); };
  auto inside = [&](int i, int e) { return FULL ? i < H : i + e < H; };
  // w_pre, and the product of w_post and the gate's row: what scales dx and d
  auto pre_scale = [&](int p) { return load_params<FULL>(a.w_pre, a.p_bf16, 0, at(p), H); };
  auto post_scale = [&](int p) {
    f32x4 v = {1.0f, 1.0f, 1.0f, 1.0f};
    if (post) v = load_params<FULL>(a.w_post, a.p_bf16, 0, at(p), H);
    if (a.gate) v *= load_params<FULL>(a.gate, a.p_bf16, gate_at, at(p), H);
    return v;
  };

  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  f32x4 S1[NV], T1[T_LDS ? 1 : NV], S0[LAYER ? NV : 1], T0[LAYER ? NV : 1], wu[KEEP ? NV : 1], wv[KEEP ? NV : 1];
#pragma unroll
  for (int p = 0; p < NV; ++p) {
    S1[p] = zero;
    if (T_LDS) t_lds[p * 64 * W + lane] = zero;
    else T1[p] = zero;
    if (LAYER) S0[p] = T0[p] = zero;
  }
  if constexpr (KEEP) {
    Params<NV, FULL> w1, w2, w3;
    if (has_dx) w1.fetch(a.w_pre, a.p_bf16, 0, at, H);
    if (post) w2.fetch(a.w_post, a.p_bf16, 0, at, H);
    if (HAS_Y && a.gate) w3.fetch(a.gate, a.p_bf16, gate_at, at, H);
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      wu[p] = has_dx ? w1.get(p, a.p_bf16, at(p), H) : zero;
      wv[p] = f32x4{1.0f, 1.0f, 1.0f, 1.0f};
      if (post) wv[p] = w2.get(p, a.p_bf16, at(p), H);
      if (HAS_Y && a.gate) wv[p] *= w3.get(p, a.p_bf16, at(p), H);
    }
  }

  // What a row needs, as loaded.
  typedef typename Row<RT, FULL>::raw rraw;
  struct In {
    rraw d[NV], r[NV];
    typename Row<YT, FULL>::raw y[NV];
    typename Row<DXT, FULL>::raw u[NV];
  };
  auto fetch = [&](int64_t row, In& in) {
    if (a.dr_out) {
      const Row<RT, FULL> m(a.dr_out, row * a.ld_dr_out, H);
#pragma unroll
      for (int p = 0; p < NV; ++p) in.d[p] = m.load_raw(at(p));
    }
    if (has_dx) {
      const Row<RT, FULL> m(a.r, row * a.ld_r, H);
#pragma unroll
      for (int p = 0; p < NV; ++p) in.r[p] = m.load_raw(at(p));
      const Row<DXT, FULL> mu(a.dx, row * a.ld_dx, H);
#pragma unroll
      for (int p = 0; p < NV; ++p) in.u[p] = mu.load_raw(at(p));
    }
    if (HAS_Y) {
      const Row<YT, FULL> m(a.y, row * a.ld_y, H);
#pragma unroll
      for (int p = 0; p < NV; ++p) in.y[p] = m.load_raw(at(p));
    }
  };

  In in;
  int64_t row = row0 + (W == 1 ? wave : 0);
  if (AHEAD && row < row1) fetch(row, in);
  for (int turn = 0; row < row1; row += STEP, turn ^= 1) {
    float* slot = slots + turn * SLOT;
    f32x4 d[NV], y[NV], r[NV], u[NV];
    auto load_y = [&] {
      const Row<YT, FULL> m(a.y, row * a.ld_y, H);
#pragma unroll
      for (int p = 0; p < NV; ++p) y[p] = m.load(at(p));
    };
    if (AHEAD) {
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        d[p] = a.dr_out ? Row<RT, FULL>::widen_raw(in.d[p], at(p), H) : zero;
        if (HAS_Y) y[p] = Row<YT, FULL>::widen_raw(in.y[p], at(p), H);
        if (has_dx) {
          r[p] = Row<RT, FULL>::widen_raw(in.r[p], at(p), H);
          u[p] = Row<DXT, FULL>::widen_raw(in.u[p], at(p), H);
        }
      }
      if (row + STEP < row1) fetch(row + STEP, in);
    } else {
      if (has_dx) {
        const Row<RT, FULL> m(a.r, row * a.ld_r, H);
        const Row<DXT, FULL> mu(a.dx, row * a.ld_dx, H);
#pragma unroll
        for (int p = 0; p < NV; ++p) r[p] = m.load(at(p));
#pragma unroll
        for (int p = 0; p < NV; ++p) u[p] = mu.load(at(p));
      }
      const Row<RT, FULL> m(a.dr_out, row * a.ld_dr_out, H);
#pragma unroll
      for (int p = 0; p < NV; ++p) d[p] = a.dr_out ? m.load(at(p)) : zero;
      if (HAS_Y && (KEEP || !has_dx)) load_y();
    }
    if (has_dx) {
      if (pre_layer) {
        float t[1] = {0.0f};
#pragma unroll
        for (int p = 0; p < NV; ++p) t[0] += (r[p][0] + r[p][1]) + (r[p][2] + r[p][3]);
        row_sum<W>(t, slot, wave);
        const float mean = t[0] * inv;
#pragma unroll
        for (int p = 0; p < NV; ++p)
#pragma unroll
          for (int e = 0; e < 4; ++e) r[p][e] = inside(at(p), e) ? r[p][e] - mean : 0.0f;
      }
      // sum c^2, sum u w c, and for a LayerNorm sum u w, with c = r' - mean
      float q[LAYER ? 3 : 2] = {};
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        const f32x4 w = KEEP ? wu[p] : pre_scale(p);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float t = u[p][e] * w[e];
          q[0] = __builtin_fmaf(r[p][e], r[p][e], q[0]);
          q[1] = __builtin_fmaf(t, r[p][e], q[1]);
          if (LAYER) q[LAYER ? 2 : 0] += t;
        }
      }
      if (HAS_Y && !KEEP) load_y();  // no sooner: beside r' and dx there is no room for it
      row_sum<W>(q, slot + W, wave);
      const float rstd = 1.0f / sqrtf(__builtin_fmaf(q[0], inv, a.eps));
      const float dot = q[1] * rstd * inv, mu = pre_layer ? q[LAYER ? 2 : 0] * inv : 0.0f;
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        const f32x4 w = KEEP ? wu[p] : pre_scale(p), xh = r[p] * rstd;
        if (T_LDS) t_lds[p * 64 * W + lane] += u[p] * xh;
        else T1[p] += u[p] * xh;
        if (LAYER) T0[p] += u[p];
        f32x4 g = u[p] * w - xh * dot;
        if (LAYER) g -= mu;
        d[p] += g * rstd;
      }
    }
    {
      const Row<RT, FULL> m(a.dr, row * a.ld_dr, H);
#pragma unroll
      for (int p = 0; p < NV; ++p) m.store(at(p), d[p] * a.alpha);
    }
    if (!HAS_Y) continue;
    const Row<BF16, FULL> dyr(a.dy, row * a.ld_dy, H);
    if (!post) {
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        S1[p] += d[p] * y[p];
        dyr.store(at(p), d[p] * (KEEP ? wv[p] : post_scale(p)));
      }
      continue;
    }
    if (post_layer) {
      float t[1] = {0.0f};
#pragma unroll
      for (int p = 0; p < NV; ++p) t[0] += (y[p][0] + y[p][1]) + (y[p][2] + y[p][3]);
      row_sum<W>(t, slot + 4 * W, wave);
      const float mean = t[0] * inv;
#pragma unroll
      for (int p = 0; p < NV; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[p][e] = inside(at(p), e) ? y[p][e] - mean : 0.0f;
    }
    float q[LAYER ? 3 : 2] = {};
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const f32x4 v = KEEP ? wv[p] : post_scale(p);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float t = d[p][e] * v[e];  // v is 0 past the row's end
        q[0] = __builtin_fmaf(y[p][e], y[p][e], q[0]);
        q[1] = __builtin_fmaf(t, y[p][e], q[1]);
        if (LAYER) q[LAYER ? 2 : 0] += t;
      }
    }
    row_sum<W>(q, slot + 5 * W, wave);
    const float rstd = 1.0f / sqrtf(__builtin_fmaf(q[0], inv, a.eps));
    const float dot = q[1] * rstd * inv, mu = post_layer ? q[LAYER ? 2 : 0] * inv : 0.0f;
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const f32x4 v = KEEP ? wv[p] : post_scale(p), yh = y[p] * rstd;
      S1[p] += d[p] * yh;
      if (LAYER) S0[p] += d[p];
      f32x4 g = d[p] * v - yh * dot;
      if (LAYER) g -= mu;
      dyr.store(at(p), g * rstd);
    }
  }

  if (!a.part) return;
  const int64_t part = (int64_t)blockIdx.x * NACC * H;
  auto sum_of = [&](int k, int p) {
    return k == 0 ? S1[p] : k == 1 ? (T_LDS ? t_lds[p * 64 * W + lane] : T1[T_LDS ? 0 : p]) : k == 2 ? S0[LAYER ? p : 0] : T0[LAYER ? p : 0];
  };
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

template <class YT, class RT, bool HAS_Y, bool LAYER, class DXT>
hipError_t launch_form(const EdgeBwdArgs& a, int64_t blocks, bool full, hipStream_t s) {
  const dim3 grid((unsigned)blocks);
  switch (edge_bwd_shape(a.H, full)) {
    case EDGE_1x2: return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, DXT, 1, 2, true>, grid, dim3(256), s, a);
    case EDGE_4x1: return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, DXT, 4, 1, true>, grid, dim3(256), s, a);
    case EDGE_4x2: return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, DXT, 4, 2, true>, grid, dim3(256), s, a);
    case EDGE_8x2: return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, DXT, 8, 2, true>, grid, dim3(512), s, a);
    case EDGE_16x2: return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, DXT, 16, 2, true>, grid, dim3(1024), s, a);
    case EDGE_16x4: return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, DXT, 16, 4, true>, grid, dim3(1024), s, a);
    case EDGE_16x5: return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, DXT, 16, 5, true>, grid, dim3(1024), s, a);
    case EDGE_16x8: return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, DXT, 16, 8, true>, grid, dim3(1024), s, a);
    case EDGE_ANY_4x1: return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, DXT, 4, 1, false>, grid, dim3(256), s, a);
    case EDGE_ANY_8x2: return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, DXT, 8, 2, false>, grid, dim3(512), s, a);
    case EDGE_ANY_16x8: return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, DXT, 16, 8, false>, grid, dim3(1024), s, a);
  }
  return hipErrorInvalidValue;
}

template <class YT, class RT, bool HAS_Y, bool LAYER>
hipError_t launch_shape(const EdgeBwdArgs& a, int64_t blocks, bool full, hipStream_t s) {
  return a.dx_bf16 ? launch_form<YT, RT, HAS_Y, LAYER, BF16>(a, blocks, full, s)
                   : launch_form<YT, RT, HAS_Y, LAYER, F32>(a, blocks, full, s);
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
