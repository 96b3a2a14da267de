// The edge between two blocks, forward:
//
//   r' = alpha r + g (.) N_post(y),   x = N_pre(r')
//
// with y the output of the block before (the MLP's float32 sum of partials), r the
// residual stream, g the gate (one row per gate_rows tokens) and x the bf16 input
// of the block after.  N is RMSNorm, v rsqrt(mean v^2 + eps) w, or LayerNorm,
// (v - mean v) rsqrt(var v + eps) w + b, or nothing.  (Norms, dropout and residual
// additions as the token-wise operations between the tensor-parallel parts: QLM
// page §2.1.3; fusing them to save memory round trips: asorrir.com survey, part 三.)
//
// W waves hold one row in registers, each lane 4 NV elements of it as NV chunks of
// four neighbours (16-byte float32 and 8-byte bf16 accesses, a wave's chunks
// contiguous), so y and r are read once and r' and x written once, whatever the
// norms: 14 bytes an element with float32 y and r.  Statistics are float32;
// LayerNorm's variance is the mean of squares about the mean, a second pass over
// the registers.  x is the norm of the unrounded r', so a bf16 stream costs x no
// second rounding.

#include "block_dev.h"

namespace tpmlp {
namespace {

// Statistics of a row held in registers: its mean (0 for RMSNorm) and
// 1 / sqrt(mean of squares about it + eps).
template <int W, int NV, bool FULL>
__device__ __forceinline__ void row_stats(const f32x4 (&v)[NV], int kind, int lane, int H, float eps, float* slot, int wave,
                                          float& mean, float& rstd) {
  const float inv = 1.0f / (float)H;
  mean = 0.0f;
  float q[1] = {0.0f};
  if (kind == TPMLP_NORM_LAYER) {
    float s[1] = {0.0f};
#pragma unroll
    for (int p = 0; p < NV; ++p) s[0] += (v[p][0] + v[p][1]) + (v[p][2] + v[p][3]);
    row_sum<W>(s, slot, wave);
    mean = s[0] * inv;
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const int i = 4 * (p * 64 * W + lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float c = (FULL ? i < H : i + e < H) ? v[p][e] - mean : 0.0f;
        q[0] = __builtin_fmaf(c, c, q[0]);
      }
    }
  } else {  // zeros past the row's end add nothing
#pragma unroll
    for (int p = 0; p < NV; ++p)
#pragma unroll
      for (int e = 0; e < 4; ++e) q[0] = __builtin_fmaf(v[p][e], v[p][e], q[0]);
  }
  row_sum<W>(q, slot + W, wave);
  rstd = 1.0f / sqrtf(__builtin_fmaf(q[0], inv, eps));
}

template <class YT, class RT, bool HAS_Y, int W, int NV, bool FULL>
__global__ void __launch_bounds__(W == 1 ? 256 : 64 * W, W == 16 && NV <= 5 ? 8 : 1) edge_fwd_kernel(EdgeFwdArgs a) {
  __shared__ float slots[4 * W];
  const int lane = W == 1 ? threadIdx.x & 63 : threadIdx.x;  // of the row
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + wave : (int64_t)blockIdx.x;
  if (row >= a.M) return;  // W == 1 only, where no barrier follows
  const int H = a.H;
  f32x4 r[NV], y[NV];
  const Row<RT, FULL> rr(a.r, row * a.ld_r, H);
#pragma unroll
  for (int p = 0; p < NV; ++p) r[p] = rr.load(4 * (p * 64 * W + lane));
  if (HAS_Y) {
    const Row<YT, FULL> yr(a.y, row * a.ld_y, H);
#pragma unroll
    for (int p = 0; p < NV; ++p) y[p] = yr.load(4 * (p * 64 * W + lane));
    float mean = 0.0f, rstd = 1.0f;
    if (a.post != TPMLP_NORM_NONE) row_stats<W, NV, FULL>(y, a.post, lane, H, a.eps, slots, wave, mean, rstd);
    const int64_t g0 = a.gate ? (row / a.gate_rows) * a.ld_gate : 0;
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const int i = 4 * (p * 64 * W + lane);
      f32x4 n = y[p];
      if (a.post != TPMLP_NORM_NONE) {
        n = (n - mean) * rstd * load_params<FULL>(a.w_post, a.p_bf16, 0, i, H);
        if (a.b_post) n += load_params<FULL>(a.b_post, a.p_bf16, 0, i, H);
      }
      if (a.gate) n *= load_params<FULL>(a.gate, a.p_bf16, g0, i, H);
      r[p] = r[p] * a.alpha + n;
    }
  } else {
#pragma unroll
    for (int p = 0; p < NV; ++p) r[p] *= a.alpha;
  }
  if (a.r_out) {
    const Row<RT, FULL> ro(a.r_out, row * a.ld_r_out, H);
#pragma unroll
    for (int p = 0; p < NV; ++p) ro.store(4 * (p * 64 * W + lane), r[p]);
  }
  if (a.x) {
    float mean, rstd;
    row_stats<W, NV, FULL>(r, a.pre, lane, H, a.eps, slots + 2 * W, wave, mean, rstd);
    const Row<BF16, FULL> xr(a.x, row * a.ld_x, H);
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const int i = 4 * (p * 64 * W + lane);
      f32x4 n = (r[p] - mean) * rstd * load_params<FULL>(a.w_pre, a.p_bf16, 0, i, H);
      if (a.b_pre) n += load_params<FULL>(a.b_pre, a.p_bf16, 0, i, H);
      xr.store(i, n);
    }
  }
}

template <class YT, class RT, bool HAS_Y>
hipError_t launch_shape(const EdgeFwdArgs& a, bool full, hipStream_t s) {
  const dim3 rows((unsigned)a.M), rows4((unsigned)((a.M + 3) / 4));
  if (!full) {
    if (a.H <= 1024) return launch_kernel(edge_fwd_kernel<YT, RT, HAS_Y, 1, 4, false>, rows4, dim3(256), s, a);
    if (a.H <= 4096) return launch_kernel(edge_fwd_kernel<YT, RT, HAS_Y, 4, 4, false>, rows, dim3(256), s, a);
    if (a.H <= TPMLP_EDGE_MAX_H) return launch_kernel(edge_fwd_kernel<YT, RT, HAS_Y, 16, 8, false>, rows, dim3(1024), s, a);
    return hipErrorInvalidValue;
  }
  if (a.H <= 512) return launch_kernel(edge_fwd_kernel<YT, RT, HAS_Y, 1, 2, true>, rows4, dim3(256), s, a);
  if (a.H <= 1024) return launch_kernel(edge_fwd_kernel<YT, RT, HAS_Y, 1, 4, true>, rows4, dim3(256), s, a);
  if (a.H <= 2048) return launch_kernel(edge_fwd_kernel<YT, RT, HAS_Y, 4, 2, true>, rows, dim3(256), s, a);
  if (a.H <= 4096) return launch_kernel(edge_fwd_kernel<YT, RT, HAS_Y, 4, 4, true>, rows, dim3(256), s, a);
  if (a.H <= 8192) return launch_kernel(edge_fwd_kernel<YT, RT, HAS_Y, 8, 4, true>, rows, dim3(512), s, a);
  if (a.H <= 12288) return launch_kernel(edge_fwd_kernel<YT, RT, HAS_Y, 16, 3, true>, rows, dim3(1024), s, a);
  if (a.H <= 20480) return launch_kernel(edge_fwd_kernel<YT, RT, HAS_Y, 16, 5, true>, rows, dim3(1024), s, a);
  if (a.H <= TPMLP_EDGE_MAX_H) return launch_kernel(edge_fwd_kernel<YT, RT, HAS_Y, 16, 8, true>, rows, dim3(1024), s, a);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_edge_fwd(const EdgeFwdArgs& a, int y_type, int r_type, bool full, hipStream_t s) {
  if (a.M < 1 || a.M > INT32_MAX || a.H < 4 || (a.gate && a.gate_rows < 1)) return hipErrorInvalidValue;
  const bool rb = r_type == TPMLP_BF16;
  if (y_type < 0) return rb ? launch_shape<F32, BF16, false>(a, full, s) : launch_shape<F32, F32, false>(a, full, s);
  if (y_type == TPMLP_BF16) return rb ? launch_shape<BF16, BF16, true>(a, full, s) : launch_shape<BF16, F32, true>(a, full, s);
  return rb ? launch_shape<F32, BF16, true>(a, full, s) : launch_shape<F32, F32, true>(a, full, s);
}

}  // namespace tpmlp
