// How the MLP's products are planned and launched (tpmlp.hip), for the calls that are
// made of such products.
#pragma once

#include "common.h"

namespace tpmlp {

constexpr int64_t MAX_DIM = int64_t(1) << 23;  // largest size of a product's matrices
constexpr int NUM_CU = 256;  // MI355X compute units, used to size split-K
constexpr size_t WS_ALIGN = 256;
inline size_t align_up(size_t x) { return (x + WS_ALIGN - 1) / WS_ALIGN * WS_ALIGN; }
inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

struct GemmPlan {
  TileCfg tile;
  int splits;
  int k_split;
  // Hybrid plan (n_full > 0): output columns [0, n_full) are whole waves of
  // unsplit 256 x 256 tiles with the product's own epilogue; only the tail
  // columns [n_full, N) are split along K (splits, k_split) and reduced.
  int n_full = 0;
  double seconds = 0;  // by the planner's model
};

// The model's rates of one CU on a tile, its bandwidth for split-K slices and its launch.
constexpr double CU_RATE_256 = 4.3e12;      // flop/s per CU, 256x256 tile
constexpr double CU_RATE_256x128 = 3.8e12;  // flop/s per CU, 256x128 tile (half the MFMAs per load)
constexpr double CU_RATE_128 = 3.3e12;      // flop/s per CU, 128x128 tile (a quarter)
constexpr double SPLIT_BW = 4.0e12;         // bytes/s for the slices' write and re-read
constexpr double LAUNCH_S = 5e-6;

// The plan of C[M,N] over K; hybrid: its columns may be cut as above.  Slices along K hold at
// least min_slice of it.
GemmPlan plan_gemm(int64_t M, int64_t N, int64_t K, bool hybrid = true, int64_t min_slice = 512);

// Bytes of a plan's float32 split-K slices.
inline size_t part_bytes(const GemmPlan& p, int64_t M, int64_t N) {
  return p.splits > 1 ? size_t(p.splits) * M * (N - p.n_full) * 4 : 0;
}

// Whether the forward's weights, and dP for dA, are transposed first.
bool transpose_weights(int64_t M, int64_t H, int64_t F);
bool transpose_dp(int64_t M, int64_t H, int64_t F);

GemmArgs gemm_args(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t M, int64_t N, int64_t K,
                   const GemmPlan& p, void* out, int64_t ldo);

// One product with its epilogue, recorded under timing kind `kind` (negative: not
// recorded).  Split along K, the slices go to `part` as float32 and the reduction
// applies the epilogue.
hipError_t run_gemm(int kind, Layout la, Layout lb, Epi epi, const void* a, int64_t lda, const void* b, int64_t ldb,
                    int64_t M, int64_t N, int64_t K, const GemmPlan& p, void* out, uint16_t* out2, const uint16_t* aux,
                    float* part, hipStream_t s, int64_t ldo = 0, int64_t ldt = 0);

// A bf16 product of a launch of several (gemm_group.hip), on 128 x 128 tiles: C[M,N] = A B with A
// K-contiguous, out with rows of N.  Item 0 has B K-contiguous, the others N-contiguous.  Split along K
// (k_split below K; float32), an item's slices lie one after the other in out, and
// launch_group_sum adds them up into outs[i] (null: item i was not split).
struct GroupItem {
  const uint16_t *a, *b;
  int64_t lda, ldb;
  int M, N, K, k_split;
  void* out;
  int tiles_m, tiles_n;
};
constexpr int GROUP_ITEMS = 3;
// A product with both operands K-contiguous on 128 x 128 tiles, EPI_F32, or EPI_DGLU or EPI_DGLU32 with act, and
// the transpose out[C][ld_out] of in[R][C] (zeros past R) in one launch.
hipError_t launch_gemm_transpose(const GemmArgs& g, int splits, Epi base, int act, const uint16_t* in, uint16_t* out, int64_t R,
                                 int64_t C, int64_t ld_out, hipStream_t s);

hipError_t launch_gemm_group(const GroupItem (&item)[GROUP_ITEMS], bool bf16_0, bool bf16_1, hipStream_t s);
hipError_t launch_group_sum(const GroupItem (&item)[GROUP_ITEMS], void* const (&outs)[GROUP_ITEMS], bool bf16_0, bool bf16_1,
                            hipStream_t s);

}  // namespace tpmlp
