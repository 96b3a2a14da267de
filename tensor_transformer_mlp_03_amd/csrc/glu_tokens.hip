// The gated MLP's forward for a few tokens, whose time is the reading of the weights:
//
//   1. [P_g | P_u] = X A, in slices along K                         (glu_tokens_kernel)
//   2. h = act(P_g) * P_u from the slices' sums, Z = h B in slices       (the same, GATED)
//   3. Z = the slices' sum                                     (the split products' reduction)
//
// The weights lie with their columns contiguous.  A wave reads four rows of 128 columns an
// instruction, 16 bytes a lane, and multiplies with one float32 multiply-add a weight and token,
// which stays below the time of the reading for the few tokens that come here (a matrix
// instruction would need the columns transposed).  The waves of a workgroup take runs of rows;
// their sums meet in LDS.  Slices along K give every CU a workgroup; one of the second
// product computes the h of its rows itself, which saves a launch.
//
// One token by 4096 x 2048 (50 MB) 19.4 us: 8 + 6 + 2.5 on the GPU; 20480 x 10240
// (1.26 GB) 214 us, 5.9 TB/s.  The second product in one slice, 64
// workgroups of 64 columns that write Z, took 9.4 us for 6 + 2.5: each has to make all of h.

#include "block_dev.h"
#include "gated.h"
#include "product.h"

#include <algorithm>

namespace tpmlp {
namespace {

[[maybe_unused]] constexpr int LOADS = 8;  // of a step of a wave
constexpr int WAVES = 8, COLS = 128, LANES = COLS / 8, RPI = 64 / LANES, STEP = LOADS * RPI;  // lanes of a row, rows of a load, of a step

__device__ __forceinline__ float act_of(float x, int act) {
  switch (act) {  // uniform
    case TPMLP_ACT_SILU: return act_f32<TPMLP_ACT_SILU>(x);
    case TPMLP_ACT_GELU: return act_f32<TPMLP_ACT_GELU>(x);
    case TPMLP_ACT_RELU: return act_f32<TPMLP_ACT_RELU>(x);
    default: return act_f32<TPMLP_ACT_SIGMOID>(x);
  }
}

}  // namespace

namespace kern {

// MT: tokens, padded to a power of two.  x [M][K] bf16; GATED: x is h, from the slices of P.
template <int MT, bool GATED>
__global__ void __launch_bounds__(64 * WAVES) glu_tokens_kernel(GluTokensArgs a) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ float xs[GLU_TOKENS_LDS];             // [row of the workgroup][MT]
  __shared__ float sums[WAVES][MT][COLS];
  const int lane = threadIdx.x & 63, c = 8 * (lane & (LANES - 1)), rq = lane / LANES;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * COLS;
  const int block_rows = WAVES * a.rows;
  const int64_t k0 = (int64_t)blockIdx.y * block_rows;
  const int rows = (int)min((int64_t)block_rows, a.K - k0);

  // The wave's run of rows, a step at a time.
  const int first = wave * a.rows, last = min(rows, first + a.rows);
  const bool in_n = n0 + c < a.N;  // N is a multiple of 8
  u32x4 w[2][LOADS];
  auto load = [&](int b, int r0) {
    // a descriptor at the step's first row keeps offsets in 31 bits; rows past the run read zeros
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(a.w + (k0 + min(r0, rows - 1)) * a.N + n0), (short)0, 0x7FFFFFF0, 0x00020000);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int r = RPI * i + rq;
      const bool ok = in_n && r0 + r < last;
      w[b][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, ok ? (uint32_t)((r * a.N + c) * 2) : 0x7FFFFFF0u, 0, 2));
    }
  };
  load(0, first);

  // x of the workgroup's rows in float32, zeros for the tokens that pad MT
  for (int i = threadIdx.x; i < rows * MT; i += 64 * WAVES) {
    const int m = i / rows, r = i - m * rows;  // neighbouring threads read neighbouring rows
    float v = 0.0f;
    if (m < a.M) {
      if constexpr (GATED) {
        // eight slices' loads are in flight together; past the last one it is read again and left out
        const float* p = a.slices + (int64_t)m * 2 * a.K + k0 + r;
        float g = 0.0f, u = 0.0f;
        for (int s0 = 0; s0 < a.n_slices; s0 += 8) {
          float gs[8], us[8];
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            const float* q = p + min(s0 + s, a.n_slices - 1) * (a.M * 2 * a.K);
            gs[s] = q[0];
            us[s] = q[a.K];
          }
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            g += s0 + s < a.n_slices ? gs[s] : 0.0f;
            u += s0 + s < a.n_slices ? us[s] : 0.0f;
          }
        }
        v = act_of(g, a.act) * u;  // h stays float32 here
        if (a.p_save && blockIdx.x == 0) {
          a.p_save[(int64_t)m * 2 * a.K + k0 + r] = f32_to_bf16(g);
          a.p_save[(int64_t)m * 2 * a.K + a.K + k0 + r] = f32_to_bf16(u);
        }
      } else {
        v = bf16_to_f32(a.x[m * a.K + k0 + r]);
      }
    }
    xs[r * MT + m] = v;
  }
  __syncthreads();

  float acc[MT][8];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[m][e] = 0.0f;
  auto add = [&](int b, int r0) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int r = min(r0 + RPI * i + rq, rows - 1);  // past the run the weights are zeros
      float x[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) x[m] = xs[r * MT + m];
      if (r0 + RPI * i + rq >= last)
#pragma unroll
        for (int m = 0; m < MT; ++m) x[m] = 0.0f;  // an infinite x times those zeros would be NaN
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = __builtin_bit_cast(float, e & 1 ? w[b][i][e >> 1] & 0xFFFF0000u : w[b][i][e >> 1] << 16);
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m][e] = __builtin_fmaf(x[m], v, acc[m][e]);
      }
    }
  };
  for (int r0 = first; r0 < last; r0 += 2 * STEP) {
    load(1, r0 + STEP);
    __builtin_amdgcn_sched_barrier(0);
    add(0, r0);
    load(0, r0 + 2 * STEP);
    __builtin_amdgcn_sched_barrier(0);
    if (r0 + STEP < last) add(1, r0 + STEP);
  }

  // The wave's row groups, then its part of the workgroup's sum.
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t v = __builtin_bit_cast(uint32_t, acc[m][e]);
      const auto h = __builtin_amdgcn_permlane16_swap(v, v, false, false);
      const uint32_t h0 = h[0], h1 = h[1];
      const uint32_t t = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, h0) + __builtin_bit_cast(float, h1));
      const auto g = __builtin_amdgcn_permlane32_swap(t, t, false, false);
      const uint32_t g0 = g[0], g1 = g[1];
      acc[m][e] = __builtin_bit_cast(float, g0) + __builtin_bit_cast(float, g1);
    }
  if (rq == 0)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      *reinterpret_cast<f32x4*>(&sums[wave][m][c]) = f32x4{acc[m][0], acc[m][1], acc[m][2], acc[m][3]};
      *reinterpret_cast<f32x4*>(&sums[wave][m][c + 4]) = f32x4{acc[m][4], acc[m][5], acc[m][6], acc[m][7]};
    }
  __syncthreads();
  for (int i = threadIdx.x; i < MT * COLS; i += 64 * WAVES) {
    const int m = i / COLS, n = i % COLS;
    if (m >= a.M || n0 + n >= a.N) continue;
    float s = sums[0][m][n];
#pragma unroll
    for (int k = 1; k < WAVES; ++k) s += sums[k][m][n];
    a.out[((int64_t)blockIdx.y * a.M + m) * a.N + n0 + n] = s;
  }
#else
  (void)a;
#endif
}

}  // namespace kern

namespace {

template <bool GATED>
hipError_t launch_tokens(const GluTokensArgs& a, int slices, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + COLS - 1) / COLS), (unsigned)slices);
  void (*k)(GluTokensArgs) = a.M == 1 ? kern::glu_tokens_kernel<1, GATED> : a.M == 2 ? kern::glu_tokens_kernel<2, GATED> : kern::glu_tokens_kernel<4, GATED>;
  return launch_kernel(k, grid, dim3(64 * WAVES), s, a);
}

}  // namespace

// Two tokens, or four where the weights' reading is short against the launches: four by 4096 x 2048
// 24 us against 25 with the GEMM kernel, by 20480 x 10240 280 against 257; two 20 and 238.
bool glu_tokens(int64_t M, int64_t H, int64_t F) { return M <= 2 || (M <= 4 && H * F <= int64_t(1) << 24); }

// Slices of a [K][N] weight, x within the LDS: four workgroups on every CU where a wave has two
// steps or more (20480 x 10240 by one token 243 us with one a CU, 222 with two, 214 with four), else of
// one step each up to a workgroup a CU.
GluTokensPlan plan_glu_tokens(int64_t M, int64_t N, int64_t K) {
  const int mt = M == 1 ? 1 : M == 2 ? 2 : 4;
  const int64_t groups = (N + COLS - 1) / COLS, most = GLU_TOKENS_LDS / mt / WAVES / STEP * STEP;  // rows of a wave
  auto rows_for = [&](int64_t blocks) {
    const int64_t slices = (blocks + groups - 1) / groups, rows = (K + slices * WAVES - 1) / (slices * WAVES);
    return std::min(most, (rows + STEP - 1) / STEP * STEP);
  };
  const int64_t rows = std::max(rows_for(4 * NUM_CU), std::min<int64_t>(2 * STEP, rows_for(NUM_CU)));
  GluTokensPlan p;
  p.rows = (int)rows;
  p.slices = (int)((K + rows * WAVES - 1) / (rows * WAVES));
  return p;
}

hipError_t launch_glu_tokens(const GluTokensArgs& a, const GluTokensPlan& p, hipStream_t s) {
  if (a.M < 1 || a.M > 4) return hipErrorInvalidValue;
  GluTokensArgs b = a;
  b.rows = p.rows;
  return a.slices ? launch_tokens<true>(b, p.slices, s) : launch_tokens<false>(b, p.slices, s);
}

}  // namespace tpmlp
