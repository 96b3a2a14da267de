// The edge's backward with RMSNorm or no norm on its sides (block_edge_bwd.h), the
// cut of the rows into workgroups, and the kernel that finishes the column sums.

#include "block_edge_bwd.h"

#include <algorithm>

namespace tpmlp {
namespace {

// One workgroup finishes 32 columns: 32 lanes side by side on a row of the
// partial sums, 32 of them down the slices.  For few gate rows the 32 go over the
// slices of one gate row after another; for many (32 or more) each takes whole
// gate rows, which then need no exchange between lanes.
__global__ void __launch_bounds__(1024) edge_finish_kernel(EdgeFinishArgs a) {
  __shared__ float sums[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int col = (int)blockIdx.x * 32 + tx, H = a.H;
  const bool in = col < H;
  const int64_t blocks = a.groups * a.chunks, step = (int64_t)a.n_acc * H;
  const float* base = a.part + col;
  const bool layer = a.n_acc == EDGE_ACC_LAYER;

  // Sum of v over the 32 lanes of a column, on every one of them.
  auto column = [&](float v) {
    __syncthreads();
    sums[ty][tx] = v;
    __syncthreads();
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) t += sums[k][tx];
    return t;
  };

  if (a.dw_pre || a.db_pre) {
    float t1 = 0.0f, t0 = 0.0f;
    for (int64_t b = ty; in && b < blocks; b += 32) {
      t1 += base[b * step + H];
      if (layer) t0 += base[b * step + 3 * (int64_t)H];
    }
    t1 = column(t1);
    t0 = column(t0);
    if (in && ty == 0) {
      if (a.dw_pre) a.dw_pre[col] = t1;
      if (a.db_pre) a.db_pre[col] = t0;
    }
  }
  if (!a.dw_post && !a.db_post && !a.dgate) return;
  const float w = in && a.w_post ? load_param(a.w_post, a.p_bf16, col) : 1.0f;
  const float b0 = in && a.b_post ? load_param(a.b_post, a.p_bf16, col) : 0.0f;
  float dw = 0.0f, db = 0.0f;
  if (a.groups >= 32) {
    for (int64_t g = ty; in && g < a.groups; g += 32) {
      float s1 = 0.0f, s0 = 0.0f;
      for (int c = 0; c < a.chunks; ++c) {
        s1 += base[(g * a.chunks + c) * step];
        if (layer) s0 += base[(g * a.chunks + c) * step + 2 * (int64_t)H];
      }
      const float gate = a.gate ? load_param(a.gate, a.p_bf16, g * a.ld_gate + col) : 1.0f;
      dw += gate * s1;
      db += gate * s0;
      if (a.dgate) a.dgate[g * H + col] = w * s1 + b0 * s0;
    }
  } else {
    for (int64_t g = 0; g < a.groups; ++g) {
      float s1 = 0.0f, s0 = 0.0f;
      for (int c = ty; in && c < a.chunks; c += 32) {
        s1 += base[(g * a.chunks + c) * step];
        if (layer) s0 += base[(g * a.chunks + c) * step + 2 * (int64_t)H];
      }
      s1 = column(s1);
      s0 = column(s0);
      if (in && ty == 0) {
        const float gate = a.gate ? load_param(a.gate, a.p_bf16, g * a.ld_gate + col) : 1.0f;
        dw += gate * s1;
        db += gate * s0;
        if (a.dgate) a.dgate[g * H + col] = w * s1 + b0 * s0;
      }
    }
  }
  dw = column(dw);
  db = column(db);
  if (in && ty == 0) {
    if (a.dw_post) a.dw_post[col] = dw;
    if (a.db_post) a.db_post[col] = db;
  }
}

}  // namespace

EdgeBwdPlan plan_edge_bwd(int64_t M, int H, int64_t gate_rows, bool layer) {
  EdgeBwdPlan p{};
  p.n_acc = layer ? EDGE_ACC_LAYER : EDGE_ACC_RMS;
  if (M < 1) return p;
  gate_rows = std::min(gate_rows, M);
  p.groups = (M + gate_rows - 1) / gate_rows;
  // Workgroups that fill the 256 CUs: a workgroup of four one-row waves or of four
  // waves to a row leaves room for several on a CU, one of 1024 threads does not.
  const int64_t target = H <= 4096 ? 1024 : H <= 8192 ? 512 : 256;
  const int64_t least = H <= 1024 ? 4 : 1;  // rows that a workgroup holds at once
  const int64_t chunks = std::max<int64_t>(1, std::min(target / p.groups, (gate_rows + least - 1) / least));
  p.chunk_rows = ((gate_rows + chunks - 1) / chunks + least - 1) / least * least;
  p.chunks = (int)((gate_rows + p.chunk_rows - 1) / p.chunk_rows);
  p.ws_bytes = size_t(p.groups) * p.chunks * p.n_acc * H * 4;
  return p;
}

hipError_t launch_edge_bwd_rms(const EdgeBwdArgs& a, int64_t blocks, int y_type, int r_type, hipStream_t s) {
  return edge::launch_types<false>(a, blocks, y_type, r_type, s);
}

hipError_t launch_edge_bwd(const EdgeBwdArgs& a, const EdgeBwdPlan& p, int y_type, int r_type, hipStream_t s) {
  const int64_t blocks = p.groups * p.chunks;
  if (a.M < 1 || blocks < 1 || blocks > INT32_MAX || a.H < 4) return hipErrorInvalidValue;
  return p.n_acc == EDGE_ACC_LAYER ? launch_edge_bwd_layer(a, blocks, y_type, r_type, s)
                                   : launch_edge_bwd_rms(a, blocks, y_type, r_type, s);
}

hipError_t launch_edge_finish(const EdgeFinishArgs& a, hipStream_t s) {
  return launch_kernel(edge_finish_kernel, dim3((unsigned)((a.H + 31) / 32)), dim3(1024), s, a);
}

}  // namespace tpmlp
