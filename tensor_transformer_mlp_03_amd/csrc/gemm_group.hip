// Launches of the gated MLP's backward that hold several things, for sizes at which each by itself
// leaves most CUs idle: dh beside the transpose of X (gemm_transpose_kernel), then the three
// products behind the activation (gemm_group_kernel):
//
//   dX = dP A^T            first in the grid: its K, 2 F, is the longest; may be split along K
//   dB = h^T dZ, dA = X^T dP   K is the tokens; both read B N-contiguous
//
// A workgroup takes one 128 x 128 tile of one of them (the body is gemm_x16.h).  What bounds
// them is the latency of a tile's K steps, 0.6 us each, and of a launch, not bandwidth or
// matrix rate: 1001 tokens by 1000 x 1368 are 64 + 88 + 176 tiles of 43 and twice 16 steps.

#include "../../include/tpmlp.h"
#include "gemm_kernel.h"
#include "product.h"
#include "transpose.h"

namespace tpmlp {
namespace {

struct GroupArgs {
  GroupItem item[GROUP_ITEMS];
  int end[GROUP_ITEMS];  // workgroups of items 0 .. i
};

__device__ __forceinline__ GemmArgs widen_item(const GroupItem& p) {
  GemmArgs g;
  g.a = p.a;
  g.b = p.b;
  g.lda = p.lda;
  g.ldb = p.ldb;
  g.M = p.M;
  g.N = p.N;
  g.K = p.K;
  g.k_split = p.k_split;
  g.out = p.out;
  g.out2 = nullptr;
  g.aux = nullptr;
  g.ldo = g.ldt = p.N;
  g.split_stride = (int64_t)p.M * p.N;
  g.tiles_m = p.tiles_m;
  g.tiles_n = p.tiles_n;
  g.amax_a = g.amax_b = nullptr;
  g.amax_out = nullptr;
  g.amax_gelu = 0;
  g.batch = 0;
  return g;
}

template <int EPI0, int EPI1>
__global__ void __launch_bounds__(256) gemm_group_kernel(GroupArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  using namespace kern;
  constexpr int BM = 128, BN = 128, F8 = 0;
  __shared__ __attribute__((aligned(1024))) char smem[LDS_BYTES];
  const int block = blockIdx.x;
  if (block < a.end[0]) {
    constexpr int LB = KC, EPI = EPI0;
    const GemmArgs args_in = widen_item(a.item[0]);
    const int bid = block, nblocks = a.end[0];
#include "gemm_x16.h"
  } else {
    constexpr int LB = MC, EPI = EPI1;
    const int i = block < a.end[1] ? 1 : 2, first = a.end[i - 1];
    const GemmArgs args_in = widen_item(a.item[i]);
    const int bid = block - first, nblocks = a.end[i] - first;
#include "gemm_x16.h"
  }
#endif
}

// dh = dZ B^T (or its slices along K) with the transpose of X in the workgroups behind it, each on
// a CU that the product leaves idle.
struct WithTransposeArgs {
  GemmArgs g;
  TransposeArgs t;
  int tiles;  // workgroups of the product
};

template <int EPI>
__global__ void __launch_bounds__(256) gemm_transpose_kernel(WithTransposeArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  using namespace kern;
  constexpr int LB = KC, BM = 128, BN = 128, F8 = 0;
  __shared__ __attribute__((aligned(1024))) char smem[LDS_BYTES];
  const int bid = blockIdx.x, nblocks = a.tiles;
  if (bid < nblocks) {
    const GemmArgs& args_in = a.g;
#include "gemm_x16.h"
  } else {
    transpose_tile<true>(a.t, bid - nblocks);
  }
#endif
}

}  // namespace

hipError_t launch_gemm_transpose(const GemmArgs& g, int splits, int act, const uint16_t* in, uint16_t* out, int64_t R, int64_t C,
                                 int64_t ld_out, hipStream_t s) {
  WithTransposeArgs a;
  a.g = g;
  a.tiles = g.tiles_m * g.tiles_n * splits;
  const int blocks = plan_transpose(a.t, in, out, nullptr, nullptr, R, C, C, ld_out);
  if (blocks == 0 || g.batch > 1) return hipErrorInvalidValue;
  void (*k)(WithTransposeArgs) = nullptr;
  switch (act) {
    case TPMLP_ACT_NONE: k = gemm_transpose_kernel<EPI_F32>; break;
    case TPMLP_ACT_SILU: k = gemm_transpose_kernel<EPI_DGLU + TPMLP_ACT_SILU>; break;
    case TPMLP_ACT_GELU: k = gemm_transpose_kernel<EPI_DGLU + TPMLP_ACT_GELU>; break;
    case TPMLP_ACT_RELU: k = gemm_transpose_kernel<EPI_DGLU + TPMLP_ACT_RELU>; break;
    default: k = gemm_transpose_kernel<EPI_DGLU + TPMLP_ACT_SIGMOID>; break;
  }
  return launch_kernel(k, dim3(a.tiles + blocks), dim3(256), s, a);
}

hipError_t launch_gemm_group(const GroupItem (&item)[GROUP_ITEMS], bool bf16_0, bool bf16_1, hipStream_t s) {
  GroupArgs a;
  int end = 0;
  for (int i = 0; i < GROUP_ITEMS; ++i) {
    const int splits = ceil_div(item[i].K, item[i].k_split);
    if (splits > 1 && (i > 0 || bf16_0)) return hipErrorInvalidValue;
    a.item[i] = item[i];
    a.end[i] = end += item[i].tiles_m * item[i].tiles_n * splits;
  }
  void (*k)(GroupArgs) = bf16_0 ? (bf16_1 ? gemm_group_kernel<EPI_BF16, EPI_BF16> : gemm_group_kernel<EPI_BF16, EPI_F32>)
                                : (bf16_1 ? gemm_group_kernel<EPI_F32, EPI_BF16> : gemm_group_kernel<EPI_F32, EPI_F32>);
  return launch_kernel(k, dim3(end), dim3(256), s, a);
}

}  // namespace tpmlp
