// The GEMM kernel (gemm_kernel.h) for the gated MLP's two products with an activation:
//
//   forward   [P_g | P_u] = X [A_g | A_u],  h = act(P_g) * P_u     EPI_GLU
//   backward  dh = dZ B^T, dP_g = dh u act'(g), dP_u = dh act(g)    EPI_DGLU, with h^T for dB
//             the same from a P in float32, made again              EPI_DGLU32
//
// One launch makes both projections, the activation and the product of its two sides: a
// tile takes gate and up columns in blocks of 32, so the pair meets in one wave's
// staged rows and the pre-activations leave the chip only where the backward wants them.

#include "../../include/tpmlp.h"
#include "gemm_kernel.h"

namespace tpmlp {
namespace {

template <int BM, int BN, int LB, int EPI>
hipError_t launch_one(const GemmArgs& a, hipStream_t s) {
  return launch_kernel(kern::gemm_x16_kernel<LB, EPI, BM, BN, 0>, dim3(a.tiles_m * a.tiles_n), dim3(256), s, a);
}

template <int BM, int BN, int LB, int BASE>
hipError_t with_act(int act, const GemmArgs& a, hipStream_t s) {
  switch (act) {
    case TPMLP_ACT_SILU: return launch_one<BM, BN, LB, BASE + TPMLP_ACT_SILU>(a, s);
    case TPMLP_ACT_GELU: return launch_one<BM, BN, LB, BASE + TPMLP_ACT_GELU>(a, s);
    case TPMLP_ACT_RELU: return launch_one<BM, BN, LB, BASE + TPMLP_ACT_RELU>(a, s);
    case TPMLP_ACT_SIGMOID: return launch_one<BM, BN, LB, BASE + TPMLP_ACT_SIGMOID>(a, s);
    default: return hipErrorInvalidValue;
  }
}

template <int BM, int BN>
hipError_t with_layout(Layout lb, Epi base, int act, const GemmArgs& a, hipStream_t s) {
  if (base == EPI_DGLU) return lb == KC ? with_act<BM, BN, KC, EPI_DGLU>(act, a, s) : hipErrorInvalidValue;
  if (base == EPI_DGLU32) return lb == KC ? with_act<BM, BN, KC, EPI_DGLU32>(act, a, s) : hipErrorInvalidValue;
  if (base != EPI_GLU) return hipErrorInvalidValue;
  return lb == KC ? with_act<BM, BN, KC, EPI_GLU>(act, a, s) : with_act<BM, BN, MC, EPI_GLU>(act, a, s);
}

}  // namespace

hipError_t launch_gemm_glu(TileCfg tile, Layout lb, Epi base, int act, const GemmArgs& args, hipStream_t stream) {
  if (args.batch > 1 || args.k_split < args.K) return hipErrorInvalidValue;
  switch (tile) {
    case TILE_256x256: return with_layout<256, 256>(lb, base, act, args, stream);
    case TILE_128x128: return with_layout<128, 128>(lb, base, act, args, stream);
    case TILE_256x128: return with_layout<256, 128>(lb, base, act, args, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tpmlp
