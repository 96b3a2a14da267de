// Internal declarations of the block operators: what stands around one MLP in a
// training or serving step (the block's edge, the expert route, gradient clipping).
// All of them move each value once and compute a few operations on it, so HBM
// bandwidth bounds the large calls and launch latency the small ones.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/tpmlp.h"
#include "common.h"

namespace tpmlp {

// Launches that read and write more than this mark their rows' accesses as
// non-temporal: half of the Infinity Cache's 256 MB, since what stands before and after
// a call wants room there too.  Above it nothing is lost: 2048 x 20480 edge forward
// (420 MB) 94 -> 76 us, 32768 x 3584 backward (2.6 GB) 488 -> 467, 2048 x 4096 backward
// of float32 (160 MB) 48.8 -> 42.9, and 32768 x 512 forward (235 MB) between a kernel that
// writes y and one that reads x 70.4 -> 67.8 for the three.  Below it those lose: 8192 x
// 1024 forward (117 MB) 35.4 -> 37.7 for the three, 4096 x 1024 (59 MB) 10.3 -> 11.3.
constexpr int64_t BLOCK_NT_BYTES = int64_t(128) << 20;

// A launch holds fewer than 2^32 threads along a dimension: rows of one launch of up
// to 1024 threads a row, and whether a grid stays below.
constexpr int64_t BLOCK_LAUNCH_ROWS = int64_t(1) << 21;
inline bool block_grid_ok(int64_t blocks, int64_t threads) { return blocks > 0 && blocks <= (int64_t(1) << 32) / threads - 1; }

// ---------------------------------------------------------------------------
// The edge between two blocks (block_edge.hip, block_edge_bwd.hip)
// ---------------------------------------------------------------------------
struct EdgeFwdArgs {
  const void *y, *r;
  void* r_out;   // nullable
  uint16_t* x;   // nullable
  const void *w_post, *b_post, *gate, *w_pre, *b_pre;  // nullable
  int64_t ld_y, ld_r, ld_r_out, ld_x, ld_gate;
  int64_t M, gate_rows, first_row;  // rows first_row .. M - 1, up to a launch's
  int H, post, pre, p_bf16, nt;
  float alpha, eps;
  // Output in 8 bits: x holds codes (rows of ld_x bytes), scales a float32 a row, or,
  // with scale_mx, H / 32 powers of two a row (rows of ld_scales).
  void* scales;
  int64_t ld_scales;
  int scale_mx;
};

struct EdgeBwdArgs {
  const void *y, *r, *dr_out, *dx;  // dr_out, dx nullable
  void* dr;
  uint16_t* dy;
  const void *w_post, *gate, *w_pre;
  float* part;   // [groups * chunks][acc][H] column sums of each workgroup's rows, or null
  float* terms;  // [M][8] what the second sweep of a wide row needs, or null
  int64_t ld_y, ld_r, ld_dr_out, ld_dx, ld_dr, ld_dy, ld_gate;
  int64_t M, gate_rows, first_row;  // first_row: of the wide form's first kernel
  int chunks;  // workgroups per gate group
  int H, post, pre, p_bf16, dx_bf16, nt;
  float alpha, eps;
};

struct EdgeFinishArgs {
  const float* part;
  const void *w_post, *b_post, *gate;
  float *dw_post, *db_post, *dgate, *dw_pre, *db_pre;  // nullable
  int64_t groups, ld_gate;
  int chunks, n_acc, H, p_bf16;
};

// The edge's column sums: which of them a workgroup keeps, in this order.
//   S1 = sum d yh, T1 = sum dx xh; with a LayerNorm also S0 = sum d, T0 = sum dx.
constexpr int EDGE_ACC_RMS = 2, EDGE_ACC_LAYER = 4;

// The backward's row forms, waves x chunks a lane (WIDE: two kernels); ANY: rows that
// are not FULL.
enum EdgeShape : int {
  EDGE_1x1, EDGE_1x2, EDGE_4x1, EDGE_4x2, EDGE_8x2, EDGE_16x2, EDGE_WIDE,
  EDGE_ANY_1x1, EDGE_ANY_1x2, EDGE_ANY_4x1, EDGE_ANY_8x2, EDGE_ANY_WIDE
};
EdgeShape edge_bwd_shape(int H, bool full);
// Whether rows of H elements may take the WIDE form, which needs workspace.
inline bool edge_bwd_wide(int H) { return H > 4096; }

// How the backward's rows are cut: a function of the sizes alone, so the
// workspace query and the launch agree.
struct EdgeBwdPlan {
  int64_t groups, chunk_rows;
  int chunks, n_acc;
  size_t part_bytes, ws_bytes;  // the column sums; with them a wide row's terms
};
EdgeBwdPlan plan_edge_bwd(int64_t M, int H, int64_t gate_rows, bool layer);

// y_type -1: no y.  full: H is a multiple of 4 and every row of every matrix and
// vector starts at a multiple of four elements.
hipError_t launch_edge_fwd(EdgeFwdArgs a, int y_type, int r_type, bool full, hipStream_t s);
hipError_t launch_edge_fwd_fp8(EdgeFwdArgs a, int y_type, int r_type, bool full, hipStream_t s);
hipError_t launch_edge_bwd(const EdgeBwdArgs& a, const EdgeBwdPlan& p, int y_type, int r_type, bool full, hipStream_t s);
hipError_t launch_edge_finish(const EdgeFinishArgs& a, hipStream_t s);

// ---------------------------------------------------------------------------
// The expert route (block_route.hip)
// ---------------------------------------------------------------------------
struct RouteSortArgs {
  const void* ids;
  int ids64;
  int64_t pairs, rows;
  int E, align, capacity;
  int32_t *counts, *offsets, *row_of, *src_of;
  int32_t* hist;     // [blocks][E], unused by the one-workgroup form
  int blocks;
  int64_t per_block;  // pairs of one workgroup
};
hipError_t launch_route_sort(const RouteSortArgs& a, hipStream_t s);
// Pairs of one workgroup of the sort and the workgroups that cover `pairs`.
int64_t route_sort_blocks(int64_t pairs, int64_t* per_block);

struct RouteDispatchArgs {
  const uint16_t* x;
  uint16_t* xs;
  const int32_t *row_of, *src_of;
  int64_t T, rows, ld_x, ld_xs;
  int K, H;
  int segments, pad_blocks, pad_rows, lanes;
};
// full: H is a multiple of eight and every row starts at a multiple of eight elements
// (dispatch), of four both (combine and its gradient); nt: non-temporal.
hipError_t launch_route_dispatch(RouteDispatchArgs a, bool full, bool nt, hipStream_t s);

struct RouteCombineArgs {
  const void* zs;
  void* y;
  const float* w;  // nullable: 1
  const int32_t* row_of;
  int64_t T, rows, ld_zs, ld_y;
  int K, H;
};
hipError_t launch_route_combine(const RouteCombineArgs& a, int z_type, int y_type, bool full, bool nt, hipStream_t s);

struct RouteCombineBwdArgs {
  const void *dy, *zs;  // zs nullable with dw
  uint16_t* dzs;
  float* dw;
  const float* w;
  const int32_t *row_of, *src_of;
  int64_t T, rows, ld_dy, ld_zs, ld_dzs;
  int K, H;
  int pad_blocks, pad_rows;
};
hipError_t launch_route_combine_bwd(const RouteCombineBwdArgs& a, int dy_type, int z_type, bool full, bool nt, hipStream_t s);

// ---------------------------------------------------------------------------
// Gradient norm and clipping (block_clip.hip)
// ---------------------------------------------------------------------------
// Tensors of one launch: the table travels in the kernel's arguments, which
// keeps a call free of host-to-device copies (and so capturable); 29 bytes a
// tensor stay below the 4 KiB that every launch path takes.
constexpr int CLIP_TENSORS = 128;
constexpr int64_t CLIP_CHUNK = 16384;  // elements of one unit of work
constexpr int CLIP_BLOCKS = 2048;        // most workgroups (and partial sums) of a summing launch
constexpr int CLIP_SCALE_BLOCKS = 8192;  // and of a scaling one, which has no partials
constexpr uint32_t CLIP_KEEP = 4096;     // last chunks of a launch that the first pass reads so as to stay in the cache

struct ClipArgs {
  const void* in[CLIP_TENSORS];
  void* out[CLIP_TENSORS];
  int64_t size[CLIP_TENSORS];       // elements; bit 62 set: bf16
  uint32_t first[CLIP_TENSORS];       // first chunk of each tensor; past the last one, `chunks`
  uint32_t eighth[CLIP_TENSORS / 8];  // every eighth of these
  uint32_t chunks;                    // of all tensors
  double* part;       // sumsq launches: one partial per workgroup; clip launches: n_part partials
  int n_part;
  float scale, max_norm;
  float* norm;        // nullable
};
static_assert(sizeof(ClipArgs) <= 4096, "kernel arguments stay below 4 KiB");

hipError_t launch_clip_sumsq(const ClipArgs& a, int blocks, hipStream_t s);
hipError_t launch_clip_total(const double* part, int n, double* total, hipStream_t s);
hipError_t launch_clip_scale(const ClipArgs& a, int blocks, hipStream_t s);

}  // namespace tpmlp
