// The instantiations of the GEMM kernel (gemm_kernel.h) for the MLP's products, and
// their launches by tile, operand layout and epilogue.

#include "gemm_kernel.h"

namespace tpmlp {

namespace {

template <int BM, int BN, int LB, int EPI, int F8 = 0>
hipError_t launch_one(const GemmArgs& a, int splits, hipStream_t s) {
  if (a.batch > 1 && (splits != 1 || a.batch > MAX_BATCH)) return hipErrorInvalidValue;
  const int blocks = a.tiles_m * a.tiles_n * splits * (a.batch > 1 ? a.batch : 1);
  return launch_kernel(kern::gemm_x16_kernel<LB, EPI, BM, BN, F8>, dim3(blocks), dim3(256), s, a);
}

// FP8 products: (fmt_a, fmt_b) in {(0, 0), (1, 0), (0, 1)} with the epilogues the
// FP8 path uses for each.
template <int BM, int BN>
hipError_t dispatch_fp8(int fa, int fb, Epi epi, const GemmArgs& a, int splits, hipStream_t s) {
  if (fa == 0 && fb == 0) {
    switch (epi) {
      case EPI_BF16: return launch_one<BM, BN, KC, EPI_BF16, 1>(a, splits, s);
      case EPI_F32: return launch_one<BM, BN, KC, EPI_F32, 1>(a, splits, s);
      case EPI_F32_ACC: return launch_one<BM, BN, KC, EPI_F32_ACC, 1>(a, splits, s);
      default: break;
    }
  } else if (fa == 1 && fb == 0) {
    switch (epi) {
      case EPI_DGELU: return launch_one<BM, BN, KC, EPI_DGELU, 2>(a, splits, s);
      case EPI_F32: return launch_one<BM, BN, KC, EPI_F32, 2>(a, splits, s);
      case EPI_F32_ACC: return launch_one<BM, BN, KC, EPI_F32_ACC, 2>(a, splits, s);
      default: break;
    }
  } else if (fa == 0 && fb == 1) {
    if (epi == EPI_F32) return launch_one<BM, BN, KC, EPI_F32, 3>(a, splits, s);
  }
  return hipErrorInvalidValue;
}

// Every product reads A K-contiguous; B is K- or N-contiguous.
template <int BM, int BN>
hipError_t dispatch_layout(Layout la, Layout lb, Epi epi, const GemmArgs& a, int splits, hipStream_t s) {
  if (la != KC) return hipErrorInvalidValue;
  if constexpr (BN == 128) {  // paired products: no split-K, no batch
    if (epi == EPI_F32_PAIR || epi == EPI_F32_ACC_PAIR) {
      if (splits != 1 || a.batch > 1) return hipErrorInvalidValue;
      if (lb == MC)
        return epi == EPI_F32_PAIR ? launch_one<BM, BN, MC, EPI_F32_PAIR>(a, 1, s)
                                   : launch_one<BM, BN, MC, EPI_F32_ACC_PAIR>(a, 1, s);
      return epi == EPI_F32_PAIR ? launch_one<BM, BN, KC, EPI_F32_PAIR>(a, 1, s)
                                 : launch_one<BM, BN, KC, EPI_F32_ACC_PAIR>(a, 1, s);
    }
  }
  if (lb == MC) {
    switch (epi) {
      case EPI_GELU: return launch_one<BM, BN, MC, EPI_GELU>(a, splits, s);
      case EPI_F32: return launch_one<BM, BN, MC, EPI_F32>(a, splits, s);
      case EPI_F32_ACC: return launch_one<BM, BN, MC, EPI_F32_ACC>(a, splits, s);
      case EPI_BF16: return launch_one<BM, BN, MC, EPI_BF16>(a, splits, s);
      default: break;
    }
  } else {
    switch (epi) {
      case EPI_DGELU: return launch_one<BM, BN, KC, EPI_DGELU>(a, splits, s);
      case EPI_F32: return launch_one<BM, BN, KC, EPI_F32>(a, splits, s);
      case EPI_F32_ACC: return launch_one<BM, BN, KC, EPI_F32_ACC>(a, splits, s);
      case EPI_GELU: return launch_one<BM, BN, KC, EPI_GELU>(a, splits, s);
      case EPI_BF16: return launch_one<BM, BN, KC, EPI_BF16>(a, splits, s);
      default: break;
    }
  }
  return hipErrorInvalidValue;
}

}  // namespace

int tile_bm(TileCfg t) { return t == TILE_128x128 ? 128 : 256; }
int tile_bn(TileCfg t) { return t == TILE_256x256 ? 256 : 128; }

hipError_t launch_gemm_fp8(TileCfg tile, int fmt_a, int fmt_b, Epi epi, const GemmArgs& args, int splits,
                           hipStream_t stream) {
  // The kernel counts K, leading dimensions and K slices in 16-bit units: an FP8
  // row of K bytes is K/2 of them, and a K step of 64 units is 128 FP8 values.
  if ((args.K | args.lda | args.ldb | args.k_split) & 15) return hipErrorInvalidValue;
  GemmArgs g = args;
  g.K /= 2;
  g.lda /= 2;
  g.ldb /= 2;
  g.k_split /= 2;
  switch (tile) {
    case TILE_256x256: return dispatch_fp8<256, 256>(fmt_a, fmt_b, epi, g, splits, stream);
    case TILE_128x128: return dispatch_fp8<128, 128>(fmt_a, fmt_b, epi, g, splits, stream);
    case TILE_256x128: return dispatch_fp8<256, 128>(fmt_a, fmt_b, epi, g, splits, stream);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_gemm(TileCfg tile, Layout la, Layout lb, Epi epi, const GemmArgs& args, int splits,
                       hipStream_t stream) {
  switch (tile) {
    case TILE_256x256: return dispatch_layout<256, 256>(la, lb, epi, args, splits, stream);
    case TILE_128x128: return dispatch_layout<128, 128>(la, lb, epi, args, splits, stream);
    case TILE_256x128: return dispatch_layout<256, 128>(la, lb, epi, args, splits, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tpmlp
