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
//
// Bound by bandwidth: 2048 x 20480 (float32 y, bf16 r, a gate) 76 us, 5.5 TB/s; 4096 x
// 1024 LayerNorm in float32 10.2 us, 5.8 TB/s; one token of 4096 3.2 us, its latency.
// The widths were taken for occupancy: one wave to a row up to 1024 elements (no
// barrier), then four and eight with four chunks a lane; 16 waves of at most 64
// registers above 8192, so that two rows share a CU (eight waves of ten chunks: 112
// against 96 us at 2048 x 20480, before non-temporal accesses).  Rows that are not FULL have
// fewer forms, above 4096 elements one of 16 waves of eight chunks, whatever of it lies past
// the row: with float32 y and r 2048 x 4101 takes 88 us, 4100 20; 20483 150, 20480 98.

#include "block_dev.h"

#include <algorithm>

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

// Rows up to four chunks a lane have their parameters loaded with the row, so that no
// load waits behind a sum (one token 4.9 -> 3.8 us); wider ones would lose a resident
// workgroup to the registers.
template <class YT, class RT, class PT, bool HAS_Y, int W, int NV, bool FULL, bool NT>
__global__ void __launch_bounds__(W == 1 ? 256 : 64 * W, W == 16 && NV <= 5 ? 8 : 1) edge_fwd_kernel(EdgeFwdArgs a) {
  constexpr bool EARLY = NV <= 4 && W < 16;
  __shared__ float slots[4 * W];
  const int lane = W == 1 ? threadIdx.x & 63 : threadIdx.x;  // of the row
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = a.first_row + (W == 1 ? (int64_t)blockIdx.x * 4 + wave : (int64_t)blockIdx.x);
  if (row >= a.M) return;  // W == 1 only, where no barrier follows
  const int H = a.H;
  auto at = [&](int p) { return 4 * (p * 64 * W + lane); };
  const bool post = HAS_Y && a.post != TPMLP_NORM_NONE, gated = HAS_Y && a.gate;
  const Row<PT, FULL> w_post(a.w_post, 0, H), b_post(a.b_post, 0, H), w_pre(a.w_pre, 0, H), b_pre(a.b_pre, 0, H);
  const Row<PT, FULL> gate(a.gate, gated ? (row / a.gate_rows) * a.ld_gate : 0, H);
  typedef typename Row<PT, FULL>::raw praw;
  auto value = [&](praw v, int p) { return Row<PT, FULL>::widen_raw(v, at(p), H); };

  f32x4 r[NV], y[NV];
  praw wp[NV], g[NV], wn[NV];
  const Row<RT, FULL, NT> rr(a.r, row * a.ld_r, H);
  const Row<YT, FULL, NT> yr(a.y, row * a.ld_y, H);
  typename Row<RT, FULL, NT>::raw r0[NV];
  typename Row<YT, FULL, NT>::raw y0[NV];
  if (HAS_Y)
#pragma unroll
    for (int p = 0; p < NV; ++p) y0[p] = yr.load_raw(at(p));
#pragma unroll
  for (int p = 0; p < NV; ++p) r0[p] = rr.load_raw(at(p));
  if (EARLY) {
    if (post)
#pragma unroll
      for (int p = 0; p < NV; ++p) wp[p] = w_post.load_raw(at(p));
    if (gated)
#pragma unroll
      for (int p = 0; p < NV; ++p) g[p] = gate.load_raw(at(p));
    if (a.x)
#pragma unroll
      for (int p = 0; p < NV; ++p) wn[p] = w_pre.load_raw(at(p));
  }
#pragma unroll
  for (int p = 0; p < NV; ++p) {
    if (HAS_Y) y[p] = Row<YT, FULL, NT>::widen_raw(y0[p], at(p), H);
    r[p] = Row<RT, FULL, NT>::widen_raw(r0[p], at(p), H);
  }
  if (HAS_Y) {
    float mean = 0.0f, rstd = 1.0f;
    if (post) row_stats<W, NV, FULL>(y, a.post, lane, H, a.eps, slots, wave, mean, rstd);
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      f32x4 n = y[p];
      if (post) {
        n = (n - mean) * rstd * (EARLY ? value(wp[p], p) : w_post.load(at(p)));
        if (a.b_post) n += b_post.load(at(p));
      }
      if (gated) n *= EARLY ? value(g[p], p) : gate.load(at(p));
      r[p] = r[p] * a.alpha + n;
    }
  } else {
#pragma unroll
    for (int p = 0; p < NV; ++p) r[p] *= a.alpha;
  }
  if (a.r_out) {
    const Row<RT, FULL, NT> ro(a.r_out, row * a.ld_r_out, H);
#pragma unroll
    for (int p = 0; p < NV; ++p) ro.store(at(p), r[p]);
  }
  if (a.x) {
    praw bn[NV];
    if (EARLY && a.b_pre)
#pragma unroll
      for (int p = 0; p < NV; ++p) bn[p] = b_pre.load_raw(at(p));
    float mean, rstd;
    row_stats<W, NV, FULL>(r, a.pre, lane, H, a.eps, slots + 2 * W, wave, mean, rstd);
    const Row<BF16, FULL, NT> xr(a.x, row * a.ld_x, H);
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      f32x4 n = (r[p] - mean) * rstd * (EARLY ? value(wn[p], p) : w_pre.load(at(p)));
      if (a.b_pre) n += EARLY ? value(bn[p], p) : b_pre.load(at(p));
      xr.store(at(p), n);
    }
  }
}

template <class YT, class RT, class PT, bool HAS_Y, bool NT>
hipError_t launch_form(const EdgeFwdArgs& a, bool full, hipStream_t s) {
  const int64_t n = std::min(BLOCK_LAUNCH_ROWS, a.M - a.first_row);
  const dim3 rows((unsigned)n), rows4((unsigned)((n + 3) / 4));
#define EDGE_FORM(W, NV, FULL, NT_) \
  return launch_kernel(edge_fwd_kernel<YT, RT, PT, HAS_Y, W, NV, FULL, NT_>, W == 1 ? rows4 : rows, dim3(W == 1 ? 256 : 64 * W), s, a)
  if (a.H > TPMLP_EDGE_MAX_H) return hipErrorInvalidValue;
  if (!full) {
    if (a.H <= 256) EDGE_FORM(1, 1, false, false);
    if (a.H <= 1024) EDGE_FORM(1, 4, false, false);
    if (a.H <= 4096) EDGE_FORM(4, 4, false, false);
    EDGE_FORM(16, 8, false, false);
  }
  if (a.H <= 256) EDGE_FORM(1, 1, true, NT);
  if (a.H <= 512) EDGE_FORM(1, 2, true, NT);
  if (a.H <= 1024) EDGE_FORM(1, 4, true, NT);
  if (a.H <= 2048) EDGE_FORM(4, 2, true, NT);
  if (a.H <= 4096) EDGE_FORM(4, 4, true, NT);
  if (a.H <= 8192) EDGE_FORM(8, 4, true, NT);
  if (a.H <= 12288) EDGE_FORM(16, 3, true, NT);
  if (a.H <= 20480) EDGE_FORM(16, 5, true, NT);
  EDGE_FORM(16, 8, true, NT);
#undef EDGE_FORM
}

template <class YT, class RT, bool HAS_Y>
hipError_t launch_shape(const EdgeFwdArgs& a, bool full, hipStream_t s) {
  if (a.p_bf16)
    return a.nt ? launch_form<YT, RT, BF16, HAS_Y, true>(a, full, s) : launch_form<YT, RT, BF16, HAS_Y, false>(a, full, s);
  return a.nt ? launch_form<YT, RT, F32, HAS_Y, true>(a, full, s) : launch_form<YT, RT, F32, HAS_Y, false>(a, full, s);
}

}  // namespace

namespace {
hipError_t launch_rows(const EdgeFwdArgs& a, int y_type, int r_type, bool full, hipStream_t s) {
  const bool rb = r_type == TPMLP_BF16;
  if (y_type < 0) return rb ? launch_shape<F32, BF16, false>(a, full, s) : launch_shape<F32, F32, false>(a, full, s);
  if (y_type == TPMLP_BF16) return rb ? launch_shape<BF16, BF16, true>(a, full, s) : launch_shape<BF16, F32, true>(a, full, s);
  return rb ? launch_shape<F32, BF16, true>(a, full, s) : launch_shape<F32, F32, true>(a, full, s);
}
}  // namespace

hipError_t launch_edge_fwd(EdgeFwdArgs a, int y_type, int r_type, bool full, hipStream_t s) {
  if (a.M < 1 || a.H < 8 || (a.gate && a.gate_rows < 1)) return hipErrorInvalidValue;
  for (a.first_row = 0; a.first_row < a.M; a.first_row += BLOCK_LAUNCH_ROWS) {
    const hipError_t e = launch_rows(a, y_type, r_type, full, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace tpmlp
