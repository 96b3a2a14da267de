// Products of few tokens with 4-bit weights:
//
//   Y = act(X W^T), or, gated, Y = act(X W_g^T) * (X W_u^T) with W = [W_g; W_u]
//
// W[n, k] is an E2M1 code (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives) times a power of
// two for every 32 values along K (a byte e: 2^(e - 127)).  X is bf16, or E4M3 with a
// float32 scale a token or such a power of two for every 32 values.
//
// Layout.  A wave multiplies 16 rows of W (several such tiles) with 16 tokens (several
// tiles too), 128 k at a time: lane l holds 32 weights of row l % 16, eight from each 32 j + 8 (l /
// 16) on, j < 4, in 16 bytes.  In a row-major W the 64 lanes of such a load lie in 16 rows, 64 accesses where
// 1 KiB of neighbours takes 16: 20480 x 20480 weights by one token took 64 us, whatever
// the tiles, the prefetch or the order of K.  So W is packed once into these blocks of 1
// KiB, padded with zeros, and its scales into a word a row for every 128 k.  X, which every
// workgroup reads whole, is loaded along its rows and turned in LDS, a wave for itself (packed by a
// launch before, 16 tokens by 4096 x 2048 gated took 9.7 us, so 7.1; 64 by 10240 x 20480
// 44.6 and 40.8).  E4M3 values times a power of two are exact in bf16 from 2^-124 to 2^119 (bytes
// 3 to 246): of four significant bits, from bf16's least value 2^-133 to below 2^128.  Smaller ones
// round to multiples of 2^-133, larger ones are infinite.
//
// The weights become bf16 by v_cvt_scalef32_pk_bf16_fp4 with the block's scale (one
// instruction for two weights), exactly up to 2^125 (byte 252; 6 times 2^126 is past bf16); four
// v_mfma_f32_16x16x32_bf16 follow.
// (v_mfma_scale_f32_16x16x128_f8f6f4 takes the codes and scales as they are, but aligns its
// products to the largest with too few bits for a float32 sum: on codes of the whole E4M3
// range it was off by 2^-15 of the magnitude.)  The waves of a workgroup share its rows and
// split K; their float32 sums meet in LDS, where the activation follows.

#include "block_dev.h"
#include "gated.h"

#include <algorithm>

namespace tpmlp {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

constexpr int X_MX_SHORT = 3;  // TPMLP_X_E4M3_MX with K below 128

// 2^(e - 127) as a float, e byte j of a word: 2^-127 is subnormal, and 255 (not a number) is
// infinity here, which the conversions turn into NaN.
__device__ __forceinline__ float power(uint32_t word, int j) {
  const uint32_t e = (j == 3 ? word >> 1 : word << (23 - 8 * j)) & 0x7F800000u;
  return __builtin_bit_cast(float, max(e, 0x00400000u));
}

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

#if defined(__HIP_DEVICE_COMPILE__)
// Eight E4M3 values times a scale, in bf16.
__device__ __forceinline__ bf16x8_t from_e4m3(uint32_t lo, uint32_t hi, float scale) {
  return join(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, scale, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, scale, true),
              __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, scale, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, scale, true));
}
#endif

}  // namespace

namespace kern {

// NT tiles of 16 rows of W (gated: NT / 2 of gate rows, then the same pairs' up rows) by MT
// tiles of 16 tokens a wave; the WK waves take the blocks of 128 k in turn.  D blocks'
// loads are in flight at a time.  KIND: a tpmlp_x, or X_MX_SHORT.
template <int KIND, int NT, int MT, int WK, int D, bool GATED>
__global__ void __launch_bounds__(64 * WK) fp4_kernel(Fp4Args a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int NO = GATED ? NT / 2 : NT;  // tiles of outputs
  constexpr bool MX = KIND == TPMLP_X_E4M3_MX || KIND == X_MX_SHORT;
  constexpr int XV = KIND == TPMLP_X_BF16 ? 4 : 2;  // loads of 16 bytes a lane, for a tile of tokens and 128 k
  constexpr int REGIONS = MT > 1 ? 2 : 1;           // of a wave's staged X
  union Shared {
    u32x4 x[WK][REGIONS][64 * XV];
    f32x4 sums[WK][NT][64];
  };
  __shared__ Shared shared;
  auto& sums = shared.sums;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles = (a.N + 15) / 16, t0 = blockIdx.x * NO;  // tiles of outputs: of all, first of the workgroup's
  const int64_t mt0 = (int64_t)blockIdx.y * MT;
  const int blocks = (a.K + 127) / 128;

  // A tile past the last one is read as the last one and not stored.
  const u32x4* w[NT];
  const uint32_t* ws[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t tile = min(t0 + t % NO, tiles - 1) + (t >= NO ? (int64_t)tiles : 0);
    w[t] = static_cast<const u32x4*>(a.w) + tile * blocks * 64 + lane;
    ws[t] = reinterpret_cast<const uint32_t*>(static_cast<const u32x4*>(a.w) + (GATED ? 2 : 1) * (int64_t)tiles * blocks * 64) +
            tile * blocks * 16 + (lane & 15);
  }

  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[m][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  u32x4 wv[D][NT], xv[D][MT][XV];
  uint32_t sv[D][NT], xs[D][MT];
  // Past the last block its data are read again, so that no load stands behind a branch and the
  // compiler knows which are in flight.  A token or k outside X is read as the last one's.
  auto load = [&](int d, int kb) {
    kb = min(kb, blocks - 1);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      wv[d][t] = __builtin_nontemporal_load(w[t] + (int64_t)kb * 64);
      sv[d][t] = ws[t][(int64_t)kb * 16];
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int64_t first = (mt0 + m) * 16;
#pragma unroll
      for (int v = 0; v < XV; ++v) {
        if constexpr (KIND == TPMLP_X_BF16) {
          const int64_t token = min(first + (lane >> 2), a.M - 1);
          const int k8 = min(16 * kb + 4 * v + (lane & 3), a.K / 8 - 1);
          xv[d][m][v] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(a.x) + token * a.ld_x + 8 * k8);
        } else {
          const int64_t token = min(first + 8 * v + (lane >> 3), a.M - 1);
          const int k16 = min(8 * kb + (lane & 7), a.K / 16 - 1);
          xv[d][m][v] = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(a.x) + token * a.ld_x + 16 * k16);
        }
      }
      if constexpr (MX) {
        const uint8_t* p = static_cast<const uint8_t*>(a.x_scale) + min(first + (lane & 15), a.M - 1) * (a.K / 32);
        if constexpr (KIND == X_MX_SHORT) {
          xs[d][m] = p[0] | p[min(1, a.K / 32 - 1)] << 8 | p[min(2, a.K / 32 - 1)] << 16;
        } else {  // at any byte; shifted where it would pass the row's end
          const int at = min(4 * kb, a.K / 32 - 4);
          uint32_t word;
          __builtin_memcpy(&word, p + at, 4);
          xs[d][m] = word;
        }
      }
    }
  };
  // X of a block and tile of tokens: from the order of loads, neighbours along a token's row, to that of
  // the matrix instructions, through LDS; 16-byte chunks are swizzled by the token against bank
  // conflicts, of which some are left: 0.59 of the LDS's active cycles at 16 tokens of bf16, 0.42 at 64 of E4M3.
  auto tokens = [&](int d, int m, int kb, bf16x8_t (&f)[4]) {
    u32x4* region = shared.x[wave][m % REGIONS];
    const int token = lane & 15, g = lane >> 4;
    if constexpr (KIND == TPMLP_X_BF16) {
#pragma unroll
      for (int v = 0; v < 4; ++v) region[64 * v + (lane & ~3) + ((lane & 3) ^ (lane >> 4))] = xv[d][m][v];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = __builtin_bit_cast(bf16x8_t, region[64 * j + 4 * token + (g ^ (token >> 2))]);
    } else {
#pragma unroll
      for (int v = 0; v < 2; ++v) region[64 * v + (lane & ~7) + ((lane & 7) ^ (lane >> 3))] = xv[d][m][v];
      uint32_t scales = 0x7F7F7F7Fu;
      if constexpr (KIND == X_MX_SHORT) scales = xs[d][m];
      else if constexpr (MX) scales = xs[d][m] >> 8 * max(0, 4 * kb - (a.K / 32 - 4));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x2 c = reinterpret_cast<const u32x2*>(region)[2 * (8 * token + ((2 * j + (g >> 1)) ^ (token & 7))) + (g & 1)];
        f[j] = from_e4m3(c[0], c[1], MX ? power(scales, j) : 1.0f);
      }
    }
    if (kb == blocks - 1 && a.K % 128)  // W's zeros there times infinity were no zeros
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (128 * kb + 32 * j >= a.K) f[j] = __builtin_bit_cast(bf16x8_t, u32x4{0, 0, 0, 0});
  };
  auto multiply = [&](int d, int kb) {
    bf16x8_t x[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m) tokens(d, m, kb, x[m]);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float scale = power(sv[d][t], j);
        const bf16x8_t b = join(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(wv[d][t][j], scale, 0), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(wv[d][t][j], scale, 1),
                                __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(wv[d][t][j], scale, 2), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(wv[d][t][j], scale, 3));
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, x[m][j], acc[m][t], 0, 0, 0);
      }
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, wave + d * WK);
  int kb = wave;
  for (; kb + (D - 1) * WK < blocks; kb += D * WK) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      multiply(d, kb + d * WK);
      load(d, kb + (d + D) * WK);
      __builtin_amdgcn_sched_barrier(0);  // the loads stay where they are issued
    }
  }
#pragma unroll
  for (int d = 0; d < D - 1; ++d)
    if (kb + d * WK < blocks) multiply(d, kb + d * WK);

  __syncthreads();  // the staged X and the sums share their place

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
      const int64_t token = (mt0 + m) * 16 + (l & 15);
      const int n = 16 * (t0 + t) + 4 * (l >> 4);
      if (token >= a.M || n >= a.N) continue;
      if (a.x_kind == TPMLP_X_E4M3_ROW) {
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

template <int KIND, int NT, int MT, int WK, int D>
hipError_t launch_form(const Fp4Args& a, hipStream_t s) {
  const int tiles = (a.N + 15) / 16, per = a.gated ? NT / 2 : NT;
  const dim3 grid((unsigned)((tiles + per - 1) / per), (unsigned)((a.M + 16 * MT - 1) / (16 * MT)));
  if constexpr (NT % 2 == 0)
    if (a.gated) return launch_kernel(kern::fp4_kernel<KIND, NT, MT, WK, D, true>, grid, dim3(64 * WK), s, a);
  return launch_kernel(kern::fp4_kernel<KIND, NT, MT, WK, D, false>, grid, dim3(64 * WK), s, a);
}

// Tiles of W rows a workgroup (gated: of gate and up rows together).  A CU's time is W's 1 KiB a tile
// and block of 128 k, and X's 4 KiB a token tile, each read by every workgroup, which costs about
// FP4_X_COST tiles of W; the CU that has most workgroups ends last.  (20480 x 20480 gated by 16
// tokens: 640 pairs of tiles; 3 workgroups of one pair on a CU 63 us, 2 of two 61, 1 of three 44.5.
// 64 by 10240 x 20480: 5 of two tiles 78 us, 2 of four 65, 1 of five 41, 1 of six 50.)
constexpr int FP4_X_COST = 3;
int fp4_tiles(const Fp4Args& a, int mt, int most) {
  const int tiles = (a.N + 15) / 16, step = a.gated ? 2 : 1;
  int best = step;
  int64_t least = INT64_MAX;
  for (int nt = step; nt <= most; nt += step) {
    const int64_t groups = (tiles + nt / step - 1) / (nt / step), busiest = (groups + 255) / 256;
    const int64_t cost = busiest * (nt + FP4_X_COST * mt);
    if (cost < least) {
      least = cost;
      best = nt;
    }
  }
  return best;
}

template <int KIND, int MT, int D, int MOST>
hipError_t launch_tiles(const Fp4Args& a, hipStream_t s) {
  const int nt = fp4_tiles(a, MT, MOST);
  switch (nt) {
    case 1: return launch_form<KIND, 1, MT, 8, D>(a, s);
    case 2: return launch_form<KIND, 2, MT, 8, D>(a, s);
    case 3: return launch_form<KIND, 3, MT, 8, D>(a, s);
    default: break;
  }
  if constexpr (MOST >= 5) {
    if (nt == 5) return launch_form<KIND, 5, MT, 8, D>(a, s);
    // Six by four tiles do not fit the registers of eight waves (64 tokens by 20480 x 10240
    // gated 112 us, with four waves and two blocks in flight 78).
    if (nt == 6) return launch_form<KIND, 6, MT, (MT > 3 ? 4 : 8), (MT > 3 ? 2 : D)>(a, s);
  }
  return launch_form<KIND, 4, MT, 8, D>(a, s);
}

template <int KIND>
hipError_t launch_kind(const Fp4Args& a, hipStream_t s) {
  const int64_t tiles = (a.M + 15) / 16;
  if (tiles == 1) return launch_tiles<KIND, 1, 2, 6>(a, s);
  if (tiles == 2) return launch_tiles<KIND, 2, 2, 6>(a, s);
  if (tiles == 3) return launch_tiles<KIND, 3, 1, 6>(a, s);
  return launch_tiles<KIND, 4, 1, 6>(a, s);
}

hipError_t launch_part(const Fp4Args& a, hipStream_t s) {
  if (a.x_kind == TPMLP_X_E4M3_MX && a.K < 128) return launch_form<X_MX_SHORT, 2, 1, 8, 1>(a, s);
  switch (a.x_kind) {
    case TPMLP_X_BF16: return launch_kind<TPMLP_X_BF16>(a, s);
    case TPMLP_X_E4M3_ROW: return launch_kind<TPMLP_X_E4M3_ROW>(a, s);
    default: return launch_kind<TPMLP_X_E4M3_MX>(a, s);
  }
}

// Codes and scales into the blocks that the product reads, [tile][block of 128 k][lane] 16 bytes, then a
// byte each, zeros times one past the rows' and K's end: a thread writes a lane's.
__global__ void __launch_bounds__(256) fp4_pack_kernel(Fp4PackArgs a) {
  const int tiles = (a.N + 15) / 16, blocks = (a.K + 127) / 128;
  const int64_t total = (int64_t)(a.gated ? 2 : 1) * tiles * blocks * 64;
  u32x4* codes = static_cast<u32x4*>(a.packed);
  uint8_t* scales = reinterpret_cast<uint8_t*>(codes + total);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int lane = (int)(i & 63), g = lane >> 4;
    const int64_t tile = (i >> 6) / blocks;
    const int first = 4 * (int)((i >> 6) - tile * blocks);  // block of 32
    const int n = 16 * (int)(tile % tiles) + (lane & 15);
    const int64_t at = (n + (tile >= tiles ? (int64_t)a.N : 0)) * (a.K / 32) + first;
    u32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = n < a.N && first + j < a.K / 32 ? reinterpret_cast<const uint32_t*>(a.codes)[(at + j) * 4 + g] : 0;
    codes[i] = v;
    scales[(i >> 6) * 64 + 4 * (lane & 15) + g] = n < a.N && first + g < a.K / 32 ? a.scales[at + g] : 127;
  }
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

int64_t fp4_packed_bytes(int64_t N, int64_t K, bool gated) {
  const int64_t tiles = (N + 15) / 16 * (gated ? 2 : 1), blocks = (K + 127) / 128;
  return tiles * blocks * (1024 + 64);
}

hipError_t launch_fp4(const Fp4Args& a, hipStream_t s) {
  // Launches of so many tokens that their tiles fit a grid.
  const int64_t M = a.M, most = FP4_LAUNCH_TILES * 16;
  const int xs = a.x_kind == TPMLP_X_BF16 ? 2 : 1, per = a.x_kind == TPMLP_X_E4M3_MX ? a.K / 32 : 4;
  for (int64_t m = 0; m < M; m += most) {
    Fp4Args b = a;
    b.M = std::min(most, M - m);
    b.x = static_cast<const char*>(a.x) + m * a.ld_x * xs;
    if (a.x_scale) b.x_scale = static_cast<const char*>(a.x_scale) + m * per;
    b.y = static_cast<char*>(a.y) + m * a.ld_y * (a.y_bf16 ? 2 : 4);
    const hipError_t e = launch_part(b, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_fp4_pack(const Fp4PackArgs& a, hipStream_t s) {
  const int64_t threads = fp4_packed_bytes(a.N, a.K, a.gated != 0) / 17;
  return launch_kernel(fp4_pack_kernel, dim3((unsigned)std::min<int64_t>(8192, (threads + 255) / 256)), dim3(256), s, a);
}

hipError_t launch_fp4_quantize(const Fp4QuantArgs& a, hipStream_t s) {
  const unsigned g = (unsigned)(a.K / 32);
  const dim3 grid((unsigned)((a.N + 255) / 256), std::min(g, 32768u), (g + 32767) / 32768);
  return launch_kernel(fp4_quantize_kernel, grid, dim3(256), s, a);
}

}  // namespace tpmlp
