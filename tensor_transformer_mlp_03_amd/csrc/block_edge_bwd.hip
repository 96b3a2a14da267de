// The edge's backward with RMSNorm or no norm on its sides (block_edge_bwd.h), the
// cut of the rows into workgroups, and the kernel that finishes the column sums.

#include "block_edge_bwd.h"

namespace tpmlp {
namespace {

// One workgroup finishes 16 columns: 16 lanes side by side on a row of the partial
// sums, and 64 lines of them down the slices.  The largest power of two of lines that
// lets the 64 work on different rows of the gate shares one row's slices.  A line
// adds all four sums of its slices in one walk, eight slices' loads issued before
// the first is added: the slices come from other XCDs' writes, through memory, and
// the kernel is bound by the latency of these loads.  With a gate row for every few
// tokens a group is one slice, which the eight loads of a batch share, and the sums are as
// many as the data: 8192 x 4096 in float32 takes 134 us with one gate row, 155 with one for
// 16 tokens and 445 with one for each (268 MB of sums).
constexpr int FIN_COLS = 16, FIN_LINES = 64, FIN_BATCH = 8;

template <int NACC>
__global__ void __launch_bounds__(FIN_COLS * FIN_LINES) edge_finish_kernel(EdgeFinishArgs a) {
  __shared__ float sums[4][FIN_LINES][FIN_COLS + 1];
  const int tx = threadIdx.x % FIN_COLS, ty = threadIdx.x / FIN_COLS;
  const int H = a.H, col = (int)blockIdx.x * FIN_COLS + tx, c = min(col, H - 1);
  const bool in = col < H;
  const int64_t step = (int64_t)NACC * H;
  const float w = a.w_post ? load_param(a.w_post, a.p_bf16, c) : 1.0f;
  const float b0 = a.b_post ? load_param(a.b_post, a.p_bf16, c) : 0.0f;
  int share = FIN_LINES;  // lines to a row of the gate
  while (share > 1 && share * a.groups > FIN_LINES) share >>= 1;
  const int line = ty % share;
  float dw = 0.0f, db = 0.0f, t1 = 0.0f, t0 = 0.0f;
  for (int64_t g0 = 0; g0 < a.groups; g0 += FIN_LINES / share) {
    const int64_t g = g0 + ty / share;
    float s[4] = {};
    if (g < a.groups) {
      const float* slice = a.part + g * a.chunks * step + c;
      for (int b = line; b < a.chunks; b += FIN_BATCH * share) {
        float v[FIN_BATCH][NACC];
#pragma unroll
        for (int k = 0; k < FIN_BATCH; ++k)
#pragma unroll
          for (int j = 0; j < NACC; ++j) v[k][j] = slice[min(b + k * share, a.chunks - 1) * step + (int64_t)j * H];
#pragma unroll
        for (int k = 0; k < FIN_BATCH; ++k)
#pragma unroll
          for (int j = 0; j < NACC; ++j) s[j] += b + k * share < a.chunks ? v[k][j] : 0.0f;
      }
    }
    t1 += s[1];
    t0 += s[3];
    float s1 = s[0], s0 = s[2];
    if (share > 1) {  // uniform; then there is one pass over the groups
      sums[0][ty][tx] = s1;
      sums[1][ty][tx] = s0;
      __syncthreads();
      s1 = s0 = 0.0f;
      if (line == 0)
        for (int k = 0; k < share; ++k) {
          s1 += sums[0][ty + k][tx];
          s0 += sums[1][ty + k][tx];
        }
      __syncthreads();
    }
    if (line == 0 && g < a.groups) {
      const float gate = a.gate ? load_param(a.gate, a.p_bf16, g * a.ld_gate + c) : 1.0f;
      dw = __builtin_fmaf(gate, s1, dw);
      db = __builtin_fmaf(gate, s0, db);
      if (a.dgate && in) a.dgate[g * H + col] = w * s1 + b0 * s0;
    }
  }
  sums[0][ty][tx] = t1;
  sums[1][ty][tx] = t0;
  sums[2][ty][tx] = dw;
  sums[3][ty][tx] = db;
  __syncthreads();
  if (ty >= 4 || !in) return;
  float* out = ty == 0 ? a.dw_pre : ty == 1 ? a.db_pre : ty == 2 ? a.dw_post : a.db_post;
  if (!out) return;
  float t = 0.0f;
#pragma unroll
  for (int k = 0; k < FIN_LINES; ++k) t += sums[ty][k][tx];
  out[col] = t;
}

}  // namespace

EdgeShape edge_bwd_shape(int H, bool full) {
  if (H <= 256) return full ? EDGE_1x1 : EDGE_ANY_1x1;
  if (H <= 512) return full ? EDGE_1x2 : EDGE_ANY_1x2;
  if (H <= 1024) return full ? EDGE_4x1 : EDGE_ANY_4x1;
  if (H <= 4096) return !full ? EDGE_ANY_8x2 : H <= 2048 ? EDGE_4x2 : EDGE_8x2;
  return !full ? EDGE_ANY_WIDE : H <= 8192 ? EDGE_16x2 : EDGE_WIDE;
}

EdgeBwdPlan plan_edge_bwd(int64_t M, int H, int64_t gate_rows, bool layer) {
  EdgeBwdPlan p{};
  p.n_acc = layer ? EDGE_ACC_LAYER : EDGE_ACC_RMS;
  if (M < 1) return p;
  gate_rows = std::min(gate_rows, M);
  p.groups = (M + gate_rows - 1) / gate_rows;
  // As many workgroups as the 256 CUs hold at once (a workgroup walks several
  // rows), so that all of them end together.  A wide row's slice is that of several
  // workgroups.  (The cut does not depend on whether the rows are FULL, so that the
  // workspace does not.)
  const int64_t target = H <= 2048 ? 768 : H <= 4096 ? 512 : 256;
  // Rows that a workgroup takes at least: those it holds at once, and up to four while
  // there is a workgroup for every CU, which keeps the slices below the data.
  const int64_t least = std::max<int64_t>(H <= 512 ? 4 : 1, std::min<int64_t>(4, M / 256));
  const int64_t chunks = std::max<int64_t>(1, std::min(target / p.groups, (gate_rows + least - 1) / least));
  p.chunk_rows = (gate_rows + chunks - 1) / chunks;
  p.chunks = (int)((gate_rows + p.chunk_rows - 1) / p.chunk_rows);
  p.part_bytes = size_t(p.groups) * p.chunks * p.n_acc * H * 4;
  p.part_bytes = (p.part_bytes + 15) / 16 * 16;
  p.ws_bytes = p.part_bytes + (edge_bwd_wide(H) ? size_t(M) * 8 * 4 : 0);  // with a wide row's terms
  return p;
}

hipError_t launch_edge_bwd_rms(const EdgeBwdArgs& a, int64_t blocks, int y_type, int r_type, bool full, hipStream_t s) {
  return edge::launch_types<false>(a, blocks, y_type, r_type, full, s);
}

hipError_t launch_edge_bwd(const EdgeBwdArgs& a, const EdgeBwdPlan& p, int y_type, int r_type, bool full, hipStream_t s) {
  const int64_t blocks = p.groups * p.chunks;
  if (a.M < 1 || a.H < 8) return hipErrorInvalidValue;
  if (!block_grid_ok(blocks, 1024)) return hipErrorInvalidConfiguration;
  return p.n_acc == EDGE_ACC_LAYER ? launch_edge_bwd_layer(a, blocks, y_type, r_type, full, s)
                                   : launch_edge_bwd_rms(a, blocks, y_type, r_type, full, s);
}

hipError_t launch_edge_finish(const EdgeFinishArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.H + FIN_COLS - 1) / FIN_COLS)), block(FIN_COLS * FIN_LINES);
  return a.n_acc == EDGE_ACC_LAYER ? launch_kernel(edge_finish_kernel<EDGE_ACC_LAYER>, grid, block, s, a)
                                   : launch_kernel(edge_finish_kernel<EDGE_ACC_RMS>, grid, block, s, a);
}

}  // namespace tpmlp
