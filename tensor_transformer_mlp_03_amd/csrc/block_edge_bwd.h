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

template <class YT, class RT, bool HAS_Y, bool LAYER, int W, int NV>
__global__ void __launch_bounds__(W == 1 ? 256 : 64 * W) edge_bwd_kernel(EdgeBwdArgs a) {
  constexpr int NACC = LAYER ? EDGE_ACC_LAYER : EDGE_ACC_RMS;
  constexpr int SLOT = 8 * W;  // floats of one row's sums; two sets, used in turn
  __shared__ float slots[2 * SLOT];
  const int lane = W == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int wave = threadIdx.x >> 6;
  const int H = a.H;
  const float inv = 1.0f / (float)H;
  const int64_t group = blockIdx.x / a.chunks;
  const int chunk = (int)(blockIdx.x % a.chunks);
  const int64_t g_end = min((group + 1) * a.gate_rows, a.M);
  const int64_t row0 = min(group * a.gate_rows + chunk * a.chunk_rows, g_end);
  const int64_t row1 = min(row0 + a.chunk_rows, g_end);
  const char* gp = static_cast<const char*>(a.gate) + group * a.ld_gate * (a.p_bf16 ? 2 : 4);
  const bool pre_layer = LAYER && a.pre == TPMLP_NORM_LAYER, post_layer = LAYER && a.post == TPMLP_NORM_LAYER;

  f32x4 S1[NV], T1[NV], S0[LAYER ? NV : 1], T0[LAYER ? NV : 1];
#pragma unroll
  for (int p = 0; p < NV; ++p) {
    S1[p] = T1[p] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (LAYER) S0[p] = T0[p] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  int turn = 0;
  for (int64_t row = row0 + (W == 1 ? wave : 0); row < row1; row += W == 1 ? 4 : 1, turn ^= 1) {
    float* slot = slots + turn * SLOT;
    f32x4 d[NV], y[NV];
    if (a.dr_out) {
      const auto* p0 = static_cast<const typename RT::elem*>(a.dr_out) + row * a.ld_dr_out;
#pragma unroll
      for (int p = 0; p < NV; ++p) d[p] = load4<RT>(p0, 4 * (p * 64 * W + lane), H);
    } else {
#pragma unroll
      for (int p = 0; p < NV; ++p) d[p] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    if (HAS_Y) {
      const auto* p0 = static_cast<const typename YT::elem*>(a.y) + row * a.ld_y;
#pragma unroll
      for (int p = 0; p < NV; ++p) y[p] = load4<YT>(p0, 4 * (p * 64 * W + lane), H);
    }
    if (a.dx) {
      f32x4 r[NV], u[NV];
      const auto* p0 = static_cast<const typename RT::elem*>(a.r) + row * a.ld_r;
#pragma unroll
      for (int p = 0; p < NV; ++p) r[p] = load4<RT>(p0, 4 * (p * 64 * W + lane), H);
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        const int i = 4 * (p * 64 * W + lane);
        u[p] = a.dx_bf16 ? load4<BF16>(static_cast<const uint16_t*>(a.dx) + row * a.ld_dx, i, H)
                         : load4<F32>(static_cast<const float*>(a.dx) + row * a.ld_dx, i, H);
      }
      float mean = 0.0f;
      if (pre_layer) {
        float t[1] = {0.0f};
#pragma unroll
        for (int p = 0; p < NV; ++p) t[0] += (r[p][0] + r[p][1]) + (r[p][2] + r[p][3]);
        row_sum<W>(t, slot, wave);
        mean = t[0] * inv;
      }
      // sum c^2, sum u w c, sum u w with c = r' - mean
      float q[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        const int i = 4 * (p * 64 * W + lane);
        const f32x4 w = load4_param(a.w_pre, a.p_bf16, i, H);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float c = i + e < H ? r[p][e] - mean : 0.0f;
          r[p][e] = c;
          q[0] = __builtin_fmaf(c, c, q[0]);
          q[1] = __builtin_fmaf(u[p][e] * w[e], c, q[1]);
          q[2] = __builtin_fmaf(u[p][e], w[e], q[2]);
        }
      }
      row_sum<W>(q, slot + W, wave);
      const float rstd = 1.0f / sqrtf(__builtin_fmaf(q[0], inv, a.eps));
      const float dot = q[1] * rstd * inv, mu = pre_layer ? q[2] * inv : 0.0f;
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        const int i = 4 * (p * 64 * W + lane);
        const f32x4 w = load4_param(a.w_pre, a.p_bf16, i, H);
        const f32x4 xh = r[p] * rstd;
        T1[p] += u[p] * xh;
        if (LAYER) T0[p] += u[p];
        d[p] += (u[p] * w - mu - xh * dot) * rstd;
      }
    }
    {
      auto* p0 = static_cast<typename RT::elem*>(a.dr) + row * a.ld_dr;
#pragma unroll
      for (int p = 0; p < NV; ++p) store4<RT>(p0, 4 * (p * 64 * W + lane), H, d[p] * a.alpha);
    }
    if (!HAS_Y) continue;
    uint16_t* dyp = a.dy + row * a.ld_dy;
    if (a.post == TPMLP_NORM_NONE) {
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        const int i = 4 * (p * 64 * W + lane);
        S1[p] += d[p] * y[p];
        if (a.gate) d[p] *= load4_param(gp, a.p_bf16, i, H);
        store4<BF16>(dyp, i, H, d[p]);
      }
      continue;
    }
    float mean = 0.0f;
    if (post_layer) {
      float t[1] = {0.0f};
#pragma unroll
      for (int p = 0; p < NV; ++p) t[0] += (y[p][0] + y[p][1]) + (y[p][2] + y[p][3]);
      row_sum<W>(t, slot + 4 * W, wave);
      mean = t[0] * inv;
    }
    float q[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const int i = 4 * (p * 64 * W + lane);
      f32x4 v = load4_param(a.w_post, a.p_bf16, i, H);
      if (a.gate) v *= load4_param(gp, a.p_bf16, i, H);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float c = i + e < H ? y[p][e] - mean : 0.0f, t = i + e < H ? d[p][e] * v[e] : 0.0f;
        y[p][e] = c;
        q[0] = __builtin_fmaf(c, c, q[0]);
        q[1] = __builtin_fmaf(t, c, q[1]);
        q[2] += t;
      }
    }
    row_sum<W>(q, slot + 5 * W, wave);
    const float rstd = 1.0f / sqrtf(__builtin_fmaf(q[0], inv, a.eps));
    const float dot = q[1] * rstd * inv, mu = post_layer ? q[2] * inv : 0.0f;
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const int i = 4 * (p * 64 * W + lane);
      f32x4 v = load4_param(a.w_post, a.p_bf16, i, H);
      if (a.gate) v *= load4_param(gp, a.p_bf16, i, H);
      const f32x4 yh = y[p] * rstd;
      S1[p] += d[p] * yh;
      if (LAYER) S0[p] += d[p];
      store4<BF16>(dyp, i, H, (d[p] * v - mu - yh * dot) * rstd);
    }
  }

  if (!a.part) return;
  float* part = a.part + (int64_t)blockIdx.x * NACC * H;
  if (W > 1) {
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const int i = 4 * (p * 64 * W + lane);
      store4<F32>(part, i, H, S1[p]);
      store4<F32>(part + H, i, H, T1[p]);
      if (LAYER) {
        store4<F32>(part + 2 * (int64_t)H, i, H, S0[p]);
        store4<F32>(part + 3 * (int64_t)H, i, H, T0[p]);
      }
    }
    return;
  }
  // One wave per row: the workgroup's four waves add their sums, wave 0 first.
  __shared__ f32x4 joint[W == 1 ? 4 * 64 * NV : 1];
#pragma unroll
  for (int k = 0; k < NACC; ++k) {
    __syncthreads();
#pragma unroll
    for (int p = 0; p < NV; ++p)
      joint[wave * 64 * NV + p * 64 + lane] = k == 0 ? S1[p] : k == 1 ? T1[p] : k == 2 ? S0[LAYER ? p : 0] : T0[LAYER ? p : 0];
    __syncthreads();
    if (wave == 0)
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        f32x4 t = joint[p * 64 + lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) t += joint[w * 64 * NV + p * 64 + lane];
        store4<F32>(part + (int64_t)k * H, 4 * (p * 64 + lane), H, t);
      }
  }
}

template <class YT, class RT, bool HAS_Y, bool LAYER>
hipError_t launch_shape(const EdgeBwdArgs& a, int64_t blocks, hipStream_t s) {
  const dim3 grid((unsigned)blocks);
  if (a.H <= 512) return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, 1, 2>, grid, dim3(256), s, a);
  if (a.H <= 1024) return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, 1, 4>, grid, dim3(256), s, a);
  if (a.H <= 2048) return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, 4, 2>, grid, dim3(256), s, a);
  if (a.H <= 4096) return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, 4, 4>, grid, dim3(256), s, a);
  if (a.H <= 8192) return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, 8, 4>, grid, dim3(512), s, a);
  if (a.H <= 16384) return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, 16, 4>, grid, dim3(1024), s, a);
  if (a.H <= 20480) return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, 16, 5>, grid, dim3(1024), s, a);
  if (a.H <= TPMLP_EDGE_MAX_H) return launch_kernel(edge_bwd_kernel<YT, RT, HAS_Y, LAYER, 16, 8>, grid, dim3(1024), s, a);
  return hipErrorInvalidValue;
}

template <bool LAYER>
hipError_t launch_types(const EdgeBwdArgs& a, int64_t blocks, int y_type, int r_type, hipStream_t s) {
  const bool rb = r_type == TPMLP_BF16;
  if (y_type < 0)
    return rb ? launch_shape<F32, BF16, false, LAYER>(a, blocks, s) : launch_shape<F32, F32, false, LAYER>(a, blocks, s);
  if (y_type == TPMLP_BF16)
    return rb ? launch_shape<BF16, BF16, true, LAYER>(a, blocks, s) : launch_shape<BF16, F32, true, LAYER>(a, blocks, s);
  return rb ? launch_shape<F32, BF16, true, LAYER>(a, blocks, s) : launch_shape<F32, F32, true, LAYER>(a, blocks, s);
}

}  // namespace edge

// Defined by the two instantiating files.
hipError_t launch_edge_bwd_rms(const EdgeBwdArgs& a, int64_t blocks, int y_type, int r_type, hipStream_t s);
hipError_t launch_edge_bwd_layer(const EdgeBwdArgs& a, int64_t blocks, int y_type, int r_type, hipStream_t s);

}  // namespace tpmlp
