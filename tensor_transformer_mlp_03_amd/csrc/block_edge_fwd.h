// The edge between two blocks, forward: the row kernel, whose x is bf16 (block_edge.hip)
// or E4M3 with scales (block_edge_fp8.hip).
#pragma once

#include "block_dev.h"

namespace tpmlp {
namespace {

// Statistics of a row held in registers: its mean (0 for RMSNorm) and
// 1 / sqrt(mean of squares about it + eps).
template <int W, int NV, bool FULL>
__device__ __forceinline__ void row_stats(const f32x4 (&v)[NV], int kind, int lane, int H, float eps, float* slot, int wave,
                                          float& mean, float& rstd) {
  const float inv = 1.0f / (float)H;
  mean = 0.0f;
  float q[1] = {0.0f};
  if (kind == TPMLP_NORM_LAYER) {
    float s[1] = {0.0f};
#pragma unroll
    for (int p = 0; p < NV; ++p) s[0] += (v[p][0] + v[p][1]) + (v[p][2] + v[p][3]);
    row_sum<W>(s, slot, wave);
    mean = s[0] * inv;
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const int i = 4 * (p * 64 * W + lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float c = (FULL ? i < H : i + e < H) ? v[p][e] - mean : 0.0f;
        q[0] = __builtin_fmaf(c, c, q[0]);
      }
    }
  } else {  // zeros past the row's end add nothing
#pragma unroll
    for (int p = 0; p < NV; ++p)
#pragma unroll
      for (int e = 0; e < 4; ++e) q[0] = __builtin_fmaf(v[p][e], v[p][e], q[0]);
  }
  row_sum<W>(q, slot + W, wave);
  rstd = 1.0f / sqrtf(__builtin_fmaf(q[0], inv, eps));
}

// The row's x as E4M3 codes and scales, from its float32 values: one scale a row, amax /
// 448 (float32, 1 for a row of zeros, at least 2^-126 so that its reciprocal is finite),
// or one power of two for every 32 values, the smallest with amax <= 448 times it.  The
// largest value is so at most 448 codes high and nothing saturates.  Codes are those of x
// times the scale's reciprocal: exact for powers of two, a float32 rounding more for a row's, less
// than a division costs.  NaN keeps its code.
__device__ __forceinline__ uint32_t e4m3x4(f32x4 v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {  // comparisons: a NaN passes
    v[e] = v[e] > FP8_E4M3_MAX ? FP8_E4M3_MAX : v[e];
    v[e] = v[e] < -FP8_E4M3_MAX ? -FP8_E4M3_MAX : v[e];
  }
  int c = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], c, true);
}

template <int W, int NV, bool FULL, bool NT>
__device__ __forceinline__ void store_fp8(const EdgeFwdArgs& a, const f32x4 (&x)[NV], int64_t row, int lane, float* slot, int wave) {
  const int H = a.H;
  uint8_t* codes = reinterpret_cast<uint8_t*>(a.x) + row * a.ld_x;
  auto amax4 = [](f32x4 v) { return fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))); };
  auto put4 = [&](int p, float inv) {
    const int i = 4 * (p * 64 * W + lane);
    const uint32_t c = e4m3x4(x[p] * inv);
    if (FULL) {
      if (i < H) {
        uint32_t* to = reinterpret_cast<uint32_t*>(codes + i);
        if (NT) __builtin_nontemporal_store(c, to);
        else *to = c;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < H) codes[i + e] = (uint8_t)(c >> (8 * e));
    }
  };
  if (a.scale_mx) {
    uint8_t* scales = static_cast<uint8_t*>(a.scales) + row * a.ld_scales;
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      const float m = max8(fmaxf(0.0f, amax4(x[p])));  // eight lanes hold the 32 values of a scale; 0 if all are NaN
      const uint32_t b = __builtin_bit_cast(uint32_t, m);
      // m = f 2^(e - 127), 448 = 1.75 * 2^8
      const int e = (int)(b >> 23) - ((b & 0x7FFFFFu) > 0x600000u ? 7 : 8);
      const int code = m == 0.0f ? 127 : max(0, e);
      const int i = 4 * (p * 64 * W + lane);
      if ((lane & 7) == 0 && i < H) scales[i >> 5] = (uint8_t)code;
      put4(p, __builtin_bit_cast(float, (uint32_t)(254 - code) << 23));
    }
  } else {
    float m = 0.0f;
#pragma unroll
    for (int p = 0; p < NV; ++p) m = fmaxf(m, amax4(x[p]));
    m = row_max<W>(m, slot, wave);
    const float scale = m == 0.0f ? 1.0f : fmaxf(m / FP8_E4M3_MAX, 1.17549435e-38f);
    if (lane == 0) static_cast<float*>(a.scales)[row] = scale;
    const float inv = 1.0f / scale;
#pragma unroll
    for (int p = 0; p < NV; ++p) put4(p, inv);
  }
}

// Rows up to four chunks a lane have their parameters loaded with the row, so that no
// load waits behind a sum (one token 4.9 -> 3.8 us); wider ones would lose a resident
// workgroup to the registers.
template <class YT, class RT, class PT, bool HAS_Y, int W, int NV, bool FULL, bool NT, bool OUT8 = false>
__global__ void __launch_bounds__(W == 1 ? 256 : 64 * W, W == 16 && NV <= 5 ? 8 : 1) edge_fwd_kernel(EdgeFwdArgs a) {
  constexpr bool EARLY = NV <= 4 && W < 16;
  __shared__ float slots[(OUT8 ? 5 : 4) * W];
  const int lane = W == 1 ? threadIdx.x & 63 : threadIdx.x;  // of the row
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = a.first_row + (W == 1 ? (int64_t)blockIdx.x * 4 + wave : (int64_t)blockIdx.x);
  if (row >= a.M) return;  // W == 1 only, where no barrier follows
  const int H = a.H;
  auto at = [&](int p) { return 4 * (p * 64 * W + lane); };
  const bool post = HAS_Y && a.post != TPMLP_NORM_NONE, gated = HAS_Y && a.gate;
  const Row<PT, FULL> w_post(a.w_post, 0, H), b_post(a.b_post, 0, H), w_pre(a.w_pre, 0, H), b_pre(a.b_pre, 0, H);
  const Row<PT, FULL> gate(a.gate, gated ? (row / a.gate_rows) * a.ld_gate : 0, H);
  typedef typename Row<PT, FULL>::raw praw;
  auto value = [&](praw v, int p) { return Row<PT, FULL>::widen_raw(v, at(p), H); };

  f32x4 r[NV], y[NV];
  praw wp[NV], g[NV], wn[NV];
  const Row<RT, FULL, NT> rr(a.r, row * a.ld_r, H);
  const Row<YT, FULL, NT> yr(a.y, row * a.ld_y, H);
  typename Row<RT, FULL, NT>::raw r0[NV];
  typename Row<YT, FULL, NT>::raw y0[NV];
  if (HAS_Y)
#pragma unroll
    for (int p = 0; p < NV; ++p) y0[p] = yr.load_raw(at(p));
#pragma unroll
  for (int p = 0; p < NV; ++p) r0[p] = rr.load_raw(at(p));
  if (EARLY) {
    if (post)
#pragma unroll
      for (int p = 0; p < NV; ++p) wp[p] = w_post.load_raw(at(p));
    if (gated)
#pragma unroll
      for (int p = 0; p < NV; ++p) g[p] = gate.load_raw(at(p));
    if (a.x)
#pragma unroll
      for (int p = 0; p < NV; ++p) wn[p] = w_pre.load_raw(at(p));
  }
#pragma unroll
  for (int p = 0; p < NV; ++p) {
    if (HAS_Y) y[p] = Row<YT, FULL, NT>::widen_raw(y0[p], at(p), H);
    r[p] = Row<RT, FULL, NT>::widen_raw(r0[p], at(p), H);
  }
  if (HAS_Y) {
    float mean = 0.0f, rstd = 1.0f;
    if (post) row_stats<W, NV, FULL>(y, a.post, lane, H, a.eps, slots, wave, mean, rstd);
#pragma unroll
    for (int p = 0; p < NV; ++p) {
      f32x4 n = y[p];
      if (post) {
        n = (n - mean) * rstd * (EARLY ? value(wp[p], p) : w_post.load(at(p)));
        if (a.b_post) n += b_post.load(at(p));
      }
      if (gated) n *= EARLY ? value(g[p], p) : gate.load(at(p));
      r[p] = r[p] * a.alpha + n;
    }
  } else {
#pragma unroll
    for (int p = 0; p < NV; ++p) r[p] *= a.alpha;
  }
  if (a.r_out) {
    const Row<RT, FULL, NT> ro(a.r_out, row * a.ld_r_out, H);
#pragma unroll
    for (int p = 0; p < NV; ++p) ro.store(at(p), r[p]);
  }
  if (a.x) {
    praw bn[NV];
    if (EARLY && a.b_pre)
#pragma unroll
      for (int p = 0; p < NV; ++p) bn[p] = b_pre.load_raw(at(p));
    float mean, rstd;
    row_stats<W, NV, FULL>(r, a.pre, lane, H, a.eps, slots + 2 * W, wave, mean, rstd);
    if constexpr (OUT8) {
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        f32x4 n = (r[p] - mean) * rstd * (EARLY ? value(wn[p], p) : w_pre.load(at(p)));
        if (a.b_pre) n += EARLY ? value(bn[p], p) : b_pre.load(at(p));
        r[p] = n;
      }
      store_fp8<W, NV, FULL, NT>(a, r, row, lane, slots + 4 * W, wave);
    } else {
      const Row<BF16, FULL, NT> xr(a.x, row * a.ld_x, H);
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        f32x4 n = (r[p] - mean) * rstd * (EARLY ? value(wn[p], p) : w_pre.load(at(p)));
        if (a.b_pre) n += EARLY ? value(bn[p], p) : b_pre.load(at(p));
        xr.store(at(p), n);
      }
    }
  }
}

}  // namespace
}  // namespace tpmlp
