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

#include "block_edge_fwd.h"

#include <algorithm>

namespace tpmlp {
namespace {

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
