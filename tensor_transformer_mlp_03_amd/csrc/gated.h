// Internal declarations of the gated block's operators: the gated MLP (glu.hip), dropout
// with the residual's addition (drop.hip), the edge with an 8-bit output
// (block_edge_fp8.hip) and products with 4-bit weights (fp4.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/tpmlp.h"
#include "common.h"

namespace tpmlp {

// ---------------------------------------------------------------------------
// The gated MLP (glu.hip)
// ---------------------------------------------------------------------------
struct GluSplitArgs {
  const float* part;   // splits slices of [M][2 F], n elements each
  int splits, act;
  int64_t M, F;
  uint16_t* h;         // [M][F]
  uint16_t* p;         // [M][2 F] or null
};
struct DGluSplitArgs {
  const float* part;   // splits slices of [M][F]
  int splits, act;
  int64_t M, F, ldt;
  const void* p;       // [M][2 F] bf16, or float32
  uint16_t* dp;        // [M][2 F]
  uint16_t* ht;        // [F][ldt], columns M .. roundup8(M) - 1 zero
};

// A few tokens' products (glu_tokens.hip): out = slices along K of x w, [slice][M][N].
constexpr int GLU_TOKENS_LDS = 8192;  // floats of x that a workgroup holds
struct GluTokensArgs {
  const uint16_t* x;     // [M][K] bf16, or
  const float* slices;   // n_slices of P [M][2 K]: x = act(P_g) * P_u
  uint16_t* p_save;      // with slices: their sum in bf16, or null
  const uint16_t* w;     // [K][N] bf16
  float* out;
  int64_t M, N, K;
  int n_slices, act, rows;
};
struct GluTokensPlan {
  int rows, slices;  // rows of K a wave, slices of K
};
bool glu_tokens(int64_t M, int64_t H, int64_t F);  // whether M tokens take these kernels
GluTokensPlan plan_glu_tokens(int64_t M, int64_t N, int64_t K);
hipError_t launch_glu_tokens(const GluTokensArgs& a, const GluTokensPlan& p, hipStream_t s);

// ---------------------------------------------------------------------------
// Dropout with a bias, added to the residual stream (drop.hip)
// ---------------------------------------------------------------------------
struct DropArgs {
  const void *y, *r, *bias;  // r and bias nullable; y is the gradient in the backward
  void* out;
  const uint64_t* state;     // {seed, step}
  float* part;               // backward with the bias's gradient: [chunks][H] column sums
  int64_t M, ld_y, ld_r, ld_out, first_row, chunk_rows;
  uint32_t site, drop;       // a number below `drop` drops the element
  int H, groups, bias_bf16, nt;  // groups of eight columns
  float scale;
};
struct DropSumArgs {
  const float* part;
  float* db;
  int64_t chunks;
  int H;
};
// How the backward with the bias's gradient cuts the rows: a function of the sizes alone.
struct DropPlan {
  int64_t chunks, chunk_rows;
  size_t ws_bytes;
};
DropPlan plan_drop(int64_t M, int64_t H);
// full: H is a multiple of 8 and every row starts at a multiple of eight elements.
hipError_t launch_drop(DropArgs a, int y_type, int out_type, bool full, hipStream_t s);
hipError_t launch_drop_bias(const DropArgs& a, const DropPlan& p, float* db, int y_type, int out_type, bool full, hipStream_t s);

// ---------------------------------------------------------------------------
// Products with 4-bit weights (fp4.hip)
// ---------------------------------------------------------------------------
constexpr int64_t FP4_LAUNCH_TILES = 4096;  // tiles of 16 tokens of one launch

struct Fp4Args {
  const void* x;        // [M][ld_x] bf16, or E4M3 codes
  const void* x_scale;  // float32 [M], or [M][K / 32] powers of two
  const void* w;        // packed codes and scales (fp4_pack_kernel)
  void* y;
  int64_t M, ld_x, ld_y;
  int N, K, act, gated, x_kind, y_bf16, y_vec;
};
int64_t fp4_packed_bytes(int64_t N, int64_t K, bool gated);
hipError_t launch_fp4(const Fp4Args& a, hipStream_t s);

struct Fp4PackArgs {
  const uint8_t *codes, *scales;  // [N or 2 N][K / 2], [N or 2 N][K / 32]
  void* packed;
  int N, K, gated;
};
hipError_t launch_fp4_pack(const Fp4PackArgs& a, hipStream_t s);

struct Fp4QuantArgs {
  const uint16_t* w;  // [K][ld] bf16 (N contiguous)
  uint8_t *codes, *scales;
  int64_t ld;
  int K, N;
};
hipError_t launch_fp4_quantize(const Fp4QuantArgs& a, hipStream_t s);

}  // namespace tpmlp
