// The edge between two blocks, forward, with the next block's input in 8 bits:
//
//   r' = alpha r + g (.) N_post(y),   x = N_pre(r'),   codes = e4m3(x / scale)
//
// The row that the edge's kernel holds in registers gives its largest magnitude, a row's or
// every 32 values', so x is never stored in a wider type: 11 bytes an element for a float32
// y and a bf16 stream against 12 with a bf16 x, and 3 more for quantizing that one.

#include "block_edge_fwd.h"

#include <algorithm>

namespace tpmlp {
namespace {

template <class YT, class RT, class PT, bool HAS_Y, bool NT>
hipError_t launch_form(const EdgeFwdArgs& a, bool full, hipStream_t s) {
  const int64_t n = std::min(BLOCK_LAUNCH_ROWS, a.M - a.first_row);
  const dim3 rows((unsigned)n), rows4((unsigned)((n + 3) / 4));
#define EDGE_FORM(W, NV, FULL, NT_) \
  return launch_kernel(edge_fwd_kernel<YT, RT, PT, HAS_Y, W, NV, FULL, NT_, true>, W == 1 ? rows4 : rows, dim3(W == 1 ? 256 : 64 * W), s, a)
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

hipError_t launch_edge_fwd_fp8(EdgeFwdArgs a, int y_type, int r_type, bool full, hipStream_t s) {
  if (a.M < 1 || a.H < 8 || (a.gate && a.gate_rows < 1)) return hipErrorInvalidValue;
  for (a.first_row = 0; a.first_row < a.M; a.first_row += BLOCK_LAUNCH_ROWS) {
    const hipError_t e = launch_rows(a, y_type, r_type, full, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace tpmlp
