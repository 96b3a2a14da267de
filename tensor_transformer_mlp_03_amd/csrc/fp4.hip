// Products of few tokens with 4-bit weights:
//
//   Y = act(X W^T), or, gated, Y = act(X W_g^T) * (X W_u^T) with W = [W_g; W_u]
//
// W[n, k] is an E2M1 code (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives; two a byte, the
// lower k in the low half) times a power of two for every 32 values along K (a byte e: 2^(e
// - 127)).  X is bf16, or E4M3 with a float32 scale a token or such a power of two for
// every 32 values.
//
// A wave multiplies 16 rows of W (several such tiles) with 16 tokens (several tiles too),
// 128 k at a time: lane l reads 16 bytes, 32 weights, of row l % 16 at 32 (l / 16), 1 KiB an
// instruction, with no repacking of W.  They become bf16, exactly, by
// v_cvt_scalef32_pk_bf16_fp4 with the block's scale (one instruction for two weights), as
// E4M3 values of X do by v_cvt_scalef32_pk_bf16_fp8, and four v_mfma_f32_16x16x32_bf16
// follow.  (v_mfma_scale_f32_16x16x128_f8f6f4 takes the codes and scales as they are, but
// aligns its products to the largest with too few bits for a float32 sum: on codes of
// the whole E4M3 range it was off by 2^-15 of the magnitude.)
// The waves of a workgroup share its rows and split K; their float32 sums meet in LDS, in
// the order of K, where the activation follows.

#include "block_dev.h"
#include "gated.h"

#include <algorithm>

namespace tpmlp {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
[[maybe_unused]] constexpr uint32_t OOB = 0x7FFFFFF0u;  // an offset past the descriptor: the load returns 0

// 2^(e - 127) as a float: 2^-127 is subnormal, and 255 (not a number) is infinity here,
// which the conversions turn into NaN.
__device__ __forceinline__ float power(uint32_t e) { return __builtin_bit_cast(float, e ? e << 23 : 0x00400000u); }

__device__ __forceinline__ bf16x8_t join(bf16x2_t a, bf16x2_t b, bf16x2_t c, bf16x2_t d) {
  return bf16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ float act_of(float x, int act) {
  switch (act) {  // uniform
    case TPMLP_ACT_SILU: return act_f32<TPMLP_ACT_SILU>(x);
    case TPMLP_ACT_GELU: return act_f32<TPMLP_ACT_GELU>(x);
    case TPMLP_ACT_RELU: return act_f32<TPMLP_ACT_RELU>(x);
    case TPMLP_ACT_SIGMOID: return act_f32<TPMLP_ACT_SIGMOID>(x);
    default: return x;
  }
}

}  // namespace

namespace kern {

// NT tiles of 16 rows of W (gated: NT / 2 of gate rows, then the same pairs' up rows) by MT
// tiles of 16 tokens a wave; WK waves split K.
template <bool X8, int NT, int MT, int WK, bool GATED>
__global__ void __launch_bounds__(64 * WK) fp4_kernel(Fp4Args a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NO = GATED ? NT / 2 : NT;  // tiles of outputs
  __shared__ f32x4 sums[WK][NT][64];
  const int lane = threadIdx.x & 63, i = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * (16 * NO);
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
  const int K = a.K, K2 = K / 2, KS = K / 32;

  auto rsrc = [](const void* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)OOB, 0x00020000);
  };
  // Descriptors at the workgroup's first row of each half of W, so that offsets stay in 31 bits.
  __amdgpu_buffer_rsrc_t rw[GATED ? 2 : 1], rs[GATED ? 2 : 1];
#pragma unroll
  for (int h = 0; h < (GATED ? 2 : 1); ++h) {
    const int64_t row = n0 + (h ? (int64_t)a.N : 0);
    rw[h] = rsrc(a.w + row * K2);
    rs[h] = rsrc(a.w_scale + row * KS);
  }
  uint32_t w_off[NT], s_off[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = 16 * (t % NO) + i;
    w_off[t] = n0 + r < a.N ? (uint32_t)(r * K2 + 16 * q) : OOB;
    s_off[t] = n0 + r < a.N ? (uint32_t)(r * KS + q) : OOB;
  }
  const __amdgpu_buffer_rsrc_t rx = rsrc(static_cast<const char*>(a.x) + m0 * a.ld_x * (X8 ? 1 : 2));
  const __amdgpu_buffer_rsrc_t rxs = rsrc(static_cast<const uint8_t*>(a.x_scale) + (X8 && a.x_mx ? m0 * KS : 0));
  uint32_t x_off[MT], xs_off[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int r = 16 * t + i;
    x_off[t] = m0 + r < a.M ? (uint32_t)((r * a.ld_x + 32 * q) * (X8 ? 1 : 2)) : OOB;
    xs_off[t] = m0 + r < a.M ? (uint32_t)(r * KS + q) : OOB;
  }

  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[m][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  const int blocks = (K + 127) / 128, per = (blocks + WK - 1) / WK;
  const int last = min(blocks, (wave + 1) * per);
  for (int kb = wave * per; kb < last; ++kb) {
    const bool in = 128 * kb + 32 * q < K;  // K is a multiple of 32: a lane's weights are in or out together
    u32x4 w[NT];
    uint32_t s[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int h = GATED && t >= NO ? 1 : 0;
      w[t] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw[h], in ? w_off[t] + 64 * kb : OOB, 0, 0));
      s[t] = __builtin_amdgcn_raw_buffer_load_b8(rs[h], in ? s_off[t] + 4 * kb : OOB, 0, 0);
    }
    bf16x8_t x[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const bool ok = in && x_off[m] != OOB;
      if constexpr (X8) {
        const uint32_t o = x_off[m] + 128 * kb;
        const u32x4 lo = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, ok ? o : OOB, 0, 0));
        const u32x4 hi = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, ok ? o + 16 : OOB, 0, 0));
        const float scale = a.x_mx ? power(__builtin_amdgcn_raw_buffer_load_b8(rxs, ok ? xs_off[m] + 4 * kb : OOB, 0, 0)) : 1.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4& v = j < 2 ? lo : hi;
          x[m][j] = join(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v[2 * (j & 1)], scale, false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v[2 * (j & 1)], scale, true),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v[2 * (j & 1) + 1], scale, false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)v[2 * (j & 1) + 1], scale, true));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[m][j] = __builtin_bit_cast(bf16x8_t, __builtin_amdgcn_raw_buffer_load_b128(rx, ok ? x_off[m] + 256 * kb + 16 * j : OOB, 0, 0));
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float scale = power(s[t]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x8_t wt = join(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[t][j], scale, 0),
                                 __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[t][j], scale, 1),
                                 __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[t][j], scale, 2),
                                 __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[t][j], scale, 3));
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wt, x[m][j], acc[m][t], 0, 0, 0);
      }
    }
  }

  // Register e of a tile holds W row 4 (l / 16) + e by token l % 16.
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int t = 0; t < NT; ++t) sums[wave][t][lane] = acc[m][t];
    __syncthreads();
    for (int item = threadIdx.x; item < NO * 64; item += 64 * WK) {
      const int t = item >> 6, l = item & 63;
      f32x4 v = sums[0][t][l], u = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 1; k < WK; ++k) v += sums[k][t][l];
      if constexpr (GATED) {
        u = sums[0][NO + t][l];
#pragma unroll
        for (int k = 1; k < WK; ++k) u += sums[k][NO + t][l];
      }
      const int64_t token = m0 + 16 * m + (l & 15);
      const int n = n0 + 16 * t + 4 * (l >> 4);
      if (token >= a.M || n >= a.N) continue;
      if (X8 && !a.x_mx) {
        const float xs = static_cast<const float*>(a.x_scale)[token];
        v *= xs;
        u *= xs;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = act_of(v[e], a.act) * (GATED ? u[e] : 1.0f);
      const int64_t o = token * a.ld_y + n;
      if (a.y_bf16) {
        uint16_t* y = static_cast<uint16_t*>(a.y) + o;
        if (a.y_vec) put(y, v);
        else
          for (int e = 0; e < 4; ++e)
            if (n + e < a.N) put1(y + e, v[e]);
      } else {
        float* y = static_cast<float*>(a.y) + o;
        if (a.y_vec) put(y, v);
        else
          for (int e = 0; e < 4; ++e)
            if (n + e < a.N) y[e] = v[e];
      }
    }
    __syncthreads();
  }
#else
  (void)a;
#endif
}

}  // namespace kern

namespace {

template <bool X8, int NT, int MT, int WK>
hipError_t launch_form(Fp4Args a, hipStream_t s) {
  const int per = 16 * (a.gated ? NT / 2 : NT);
  const int64_t M = a.M, most = int64_t(32768) * 16 * MT;  // tokens of one launch
  for (int64_t m = 0; m < M; m += most) {
    Fp4Args b = a;
    b.M = std::min(most, M - m);
    b.x = static_cast<const char*>(a.x) + m * a.ld_x * (X8 ? 1 : 2);
    if (X8) b.x_scale = static_cast<const char*>(a.x_scale) + m * (a.x_mx ? a.K / 32 : 4);
    b.y = static_cast<char*>(a.y) + m * a.ld_y * (a.y_bf16 ? 2 : 4);
    const dim3 grid((unsigned)((b.N + per - 1) / per), (unsigned)((b.M + 16 * MT - 1) / (16 * MT)));
    const hipError_t e = launch_kernel(a.gated ? kern::fp4_kernel<X8, NT, MT, WK, true> : kern::fp4_kernel<X8, NT, MT, WK, false>,
                                       grid, dim3(64 * WK), s, b);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool X8>
hipError_t launch_x(const Fp4Args& a, hipStream_t s) {
  if (a.M <= 16) return launch_form<X8, 2, 1, 8>(a, s);
  if (a.M <= 32) return launch_form<X8, 2, 2, 8>(a, s);
  return launch_form<X8, 4, 4, 8>(a, s);
}

// Weights [K][N] in bf16 to codes and scales: a lane takes the 32 values of one column.
__global__ void __launch_bounds__(256) fp4_quantize_kernel(Fp4QuantArgs a) {
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t g = blockIdx.y + (int64_t)blockIdx.z * 32768;
  if (n >= a.N || g >= a.K / 32) return;
  float v[32], amax = 0.0f;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[i] = bf16_to_f32(a.w[(g * 32 + i) * a.ld + n]);
    amax = fmaxf(amax, fabsf(v[i]));
    finite &= fabsf(v[i]) < __builtin_inff();
  }
  // The smallest power of two with amax <= 6 times it: amax = m 2^e, 6 = 1.5 * 2^2.
  const uint32_t bits = __builtin_bit_cast(uint32_t, amax);
  const int e = (int)(bits >> 23) - 127 - ((bits & 0x7FFFFFu) > 0x400000u ? 1 : 2);
  const int code = amax == 0.0f ? 127 : min(254, max(0, e + 127));
  const float inv = __builtin_bit_cast(float, code == 254 ? 0x00400000u : (uint32_t)(254 - code) << 23);
  uint32_t word[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float x = fabsf(v[i]) * inv;
    // to nearest, ties to the even code
    uint32_t c = (x > 0.25f) + (x >= 0.75f) + (x > 1.25f) + (x >= 1.75f) + (x > 2.5f) + (x >= 3.5f) + (x > 5.0f);
    c |= __builtin_bit_cast(uint32_t, v[i]) >> 31 << 3;
    word[i >> 3] |= c << (4 * (i & 7));
  }
  *reinterpret_cast<u32x4*>(a.codes + n * (a.K / 2) + g * 16) = u32x4{word[0], word[1], word[2], word[3]};
  a.scales[n * (a.K / 32) + g] = finite ? (uint8_t)code : 255;  // 255: not a number
}

}  // namespace

hipError_t launch_fp4(const Fp4Args& a, bool x_bf16, hipStream_t s) {
  return x_bf16 ? launch_x<false>(a, s) : launch_x<true>(a, s);
}

hipError_t launch_fp4_quantize(const Fp4QuantArgs& a, hipStream_t s) {
  const unsigned g = (unsigned)(a.K / 32);
  const dim3 grid((unsigned)((a.N + 255) / 256), std::min(g, 32768u), (g + 32767) / 32768);
  return launch_kernel(fp4_quantize_kernel, grid, dim3(256), s, a);
}

}  // namespace tpmlp
