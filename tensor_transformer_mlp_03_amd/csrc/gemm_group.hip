// Launches of the gated MLP's backward that hold several things, for sizes at which each by itself
// leaves most CUs idle: dh beside the transpose of X (gemm_transpose_kernel), then the three
// products behind the activation (gemm_group_kernel):
//
//   dX = dP A^T                K is 2 F
//   dB = h^T dZ, dA = X^T dP   K is the tokens; both read B N-contiguous
//
// The longest K is first in the grid; each may be split along it, and one more launch adds up
// the slices.
//
// A workgroup takes one 128 x 128 tile of one of them (the body is gemm_x16.h).  What bounds
// them is the latency of a tile's K steps, 0.6 us each, and of a launch, not bandwidth or
// matrix rate: 1001 tokens by 1000 x 1368 are 64 + 88 + 176 tiles of 43 and twice 16 steps.

#include "../../include/tpmlp.h"
#include "gemm_kernel.h"
#include "product.h"
#include "transpose.h"

#include <algorithm>

namespace tpmlp {
namespace {

struct GroupArgs {
  GroupItem item[GROUP_ITEMS];
  int start[GROUP_ITEMS], count[GROUP_ITEMS];  // workgroups of an item
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
  if (block >= a.start[0] && block < a.start[0] + a.count[0]) {
    constexpr int LB = KC, EPI = EPI0;
    const GemmArgs args_in = widen_item(a.item[0]);
    const int bid = block - a.start[0], nblocks = a.count[0];
#include "gemm_x16.h"
  } else {
    constexpr int LB = MC, EPI = EPI1;
    const int i = block < a.start[2] ? 1 : 2;  // dB's before dA's
    const GemmArgs args_in = widen_item(a.item[i]);
    const int bid = block - a.start[i], nblocks = a.count[i];
#include "gemm_x16.h"
  }
#endif
}

// The slices' sums of the items that were split, in order, four elements a thread.
struct GroupSum {
  const float* part;
  void* out;
  int64_t n4;  // of a slice
  int splits, bf16, blocks;
};
struct GroupSumArgs {
  GroupSum item[GROUP_ITEMS];
};

__global__ void __launch_bounds__(256) group_sum_kernel(GroupSumArgs a) {
  int block = blockIdx.x, i = 0;
  while (i < GROUP_ITEMS - 1 && block >= a.item[i].blocks) block -= a.item[i++].blocks;
  const GroupSum g = a.item[i];
  const int64_t at = (int64_t)block * 256 + threadIdx.x;
  if (at >= g.n4) return;
  const f32x4_t* p = reinterpret_cast<const f32x4_t*>(g.part) + at;
  f32x4_t s = p[0];
#pragma unroll 4
  for (int k = 1; k < g.splits; ++k) s += p[k * g.n4];
  if (g.bf16) {
    u16x4_t v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = f32_to_bf16(s[e]);
    reinterpret_cast<u16x4_t*>(g.out)[at] = v;
  } else {
    reinterpret_cast<f32x4_t*>(g.out)[at] = s;
  }
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

template <int BASE>
auto with_act(int act) -> void (*)(WithTransposeArgs) {
  switch (act) {
    case TPMLP_ACT_SILU: return gemm_transpose_kernel<BASE + TPMLP_ACT_SILU>;
    case TPMLP_ACT_GELU: return gemm_transpose_kernel<BASE + TPMLP_ACT_GELU>;
    case TPMLP_ACT_RELU: return gemm_transpose_kernel<BASE + TPMLP_ACT_RELU>;
    default: return gemm_transpose_kernel<BASE + TPMLP_ACT_SIGMOID>;
  }
}

}  // namespace

hipError_t launch_gemm_transpose(const GemmArgs& g, int splits, Epi base, int act, const uint16_t* in, uint16_t* out, int64_t R,
                                 int64_t C, int64_t ld_out, hipStream_t s) {
  WithTransposeArgs a;
  a.g = g;
  a.tiles = g.tiles_m * g.tiles_n * splits;
  const int blocks = plan_transpose(a.t, in, out, nullptr, nullptr, R, C, C, ld_out);
  if (blocks == 0 || g.batch > 1) return hipErrorInvalidValue;
  void (*k)(WithTransposeArgs) = base == EPI_DGLU     ? with_act<EPI_DGLU>(act)
                                 : base == EPI_DGLU32 ? with_act<EPI_DGLU32>(act)
                                                      : gemm_transpose_kernel<EPI_F32>;
  return launch_kernel(k, dim3(a.tiles + blocks), dim3(256), s, a);
}

hipError_t launch_group_sum(const GroupItem (&item)[GROUP_ITEMS], void* const (&outs)[GROUP_ITEMS], bool bf16_0, bool bf16_1,
                            hipStream_t s) {
  GroupSumArgs a;
  int blocks = 0;
  for (int i = 0; i < GROUP_ITEMS; ++i) {
    const int64_t n4 = (int64_t)item[i].M * item[i].N / 4;  // N is a multiple of 8
    a.item[i] = {static_cast<const float*>(item[i].out), outs[i], n4, ceil_div(item[i].K, item[i].k_split), i ? bf16_1 : bf16_0,
                 outs[i] ? ceil_div(n4, 256) : 0};
    blocks += a.item[i].blocks;
  }
  return launch_kernel(group_sum_kernel, dim3(blocks), dim3(256), s, a);
}

hipError_t launch_gemm_group(const GroupItem (&item)[GROUP_ITEMS], bool bf16_0, bool bf16_1, hipStream_t s) {
  GroupArgs a;
  for (int i = 0; i < GROUP_ITEMS; ++i) {
    const int splits = ceil_div(item[i].K, item[i].k_split);
    if (splits > 1 && (i > 0 ? bf16_1 : bf16_0)) return hipErrorInvalidValue;
    a.item[i] = item[i];
    a.count[i] = item[i].tiles_m * item[i].tiles_n * splits;
  }
  // the item with the longest K first
  const bool dx_first = std::min(item[0].K, item[0].k_split) >= std::min(item[1].K, item[1].k_split);
  a.start[0] = dx_first ? 0 : a.count[1] + a.count[2];
  a.start[1] = dx_first ? a.count[0] : 0;
  a.start[2] = a.start[1] + a.count[1];
  const int end = a.count[0] + a.count[1] + a.count[2];
  void (*k)(GroupArgs) = bf16_0 ? (bf16_1 ? gemm_group_kernel<EPI_BF16, EPI_BF16> : gemm_group_kernel<EPI_BF16, EPI_F32>)
                                : (bf16_1 ? gemm_group_kernel<EPI_F32, EPI_BF16> : gemm_group_kernel<EPI_F32, EPI_F32>);
  return launch_kernel(k, dim3(end), dim3(256), s, a);
}

}  // namespace tpmlp
