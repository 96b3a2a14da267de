// The gated MLP, Z = h B with h = act(P_g) * P_u and [P_g | P_u] = X [A_g | A_u], and its
// gradients, on the MLP's GEMM kernel (gemm_kernel.h, gemm_glu.hip):
//
//   forward   h, P = X A       gated product      6 M H F flops in all
//             Z = h B
//   backward  P = X A          where it was not kept
//             dh = dZ B^T      with dP_g = dh u act'(g), dP_u = dh act(g), h^T
//             dB = h^T dZ,  dA = X^T dP,  dX = dP A^T          12 M H F
//
// with g = P_g, u = P_u.  h and dP are bf16 between the products, which is what the matrix
// instructions take, as the plain MLP's G and dP are, and so is a kept P, for its bytes; every sum
// is float32.  A P that the backward makes again stays float32: in bf16 it would double the gradients'
// error.  A few tokens' forward (glu_tokens.hip), which multiplies without those instructions, keeps h
// in float32.  Tokens need not be a multiple of 8: X^T and h^T, whose
// rows are the tokens, are padded with zeros, and rows past the last token are masked in
// the loads of the other operands.

#include "checks.h"
#include "epilogue.h"
#include "gated.h"
#include "product.h"

namespace tpmlp {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint16_t u16x4_t __attribute__((ext_vector_type(4)));
typedef uint16_t u16x8_t __attribute__((ext_vector_type(8)));

int64_t up8(int64_t x) { return (x + 7) / 8 * 8; }

// ---------------------------------------------------------------------------
// The gated product split along K: the slices' sum with the epilogue of EPI_GLU
// ---------------------------------------------------------------------------
template <int ACT>
__global__ void __launch_bounds__(256) glu_split_kernel(GluSplitArgs a) {
  const int64_t n4 = a.M * a.F / 4, plane = 2 * a.M * a.F, stride = (int64_t)gridDim.x * blockDim.x;
  const uint32_t f4 = (uint32_t)(a.F / 4);
  for (int64_t j = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; j < n4; j += stride) {
    const int64_t row = (uint64_t)j / f4, col = 4 * ((uint64_t)j % f4);
    const float* pg = a.part + row * 2 * a.F + col;
    f32x4_t g = *reinterpret_cast<const f32x4_t*>(pg), u = *reinterpret_cast<const f32x4_t*>(pg + a.F);
#pragma unroll 4
    for (int i = 1; i < a.splits; ++i) {
      g += *reinterpret_cast<const f32x4_t*>(pg + i * plane);
      u += *reinterpret_cast<const f32x4_t*>(pg + i * plane + a.F);
    }
    u16x4_t h, bg, bu;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h[e] = f32_to_bf16(act_f32<ACT>(g[e]) * u[e]);
      bg[e] = f32_to_bf16(g[e]);
      bu[e] = f32_to_bf16(u[e]);
    }
    *reinterpret_cast<u16x4_t*>(a.h + row * a.F + col) = h;
    if (a.p) {
      *reinterpret_cast<u16x4_t*>(a.p + row * 2 * a.F + col) = bg;
      *reinterpret_cast<u16x4_t*>(a.p + row * 2 * a.F + a.F + col) = bu;
    }
  }
}

// Eight values of P.
__device__ __forceinline__ void eight(const uint16_t* p, float (&v)[8]) {
  const u16x8_t b = *reinterpret_cast<const u16x8_t*>(p);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = bf16_to_f32(b[e]);
}
__device__ __forceinline__ void eight(const float* p, float (&v)[8]) {
  const f32x4_t a = *reinterpret_cast<const f32x4_t*>(p), b = *reinterpret_cast<const f32x4_t*>(p + 4);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = e < 4 ? a[e & 3] : b[e & 3];
}

// ---------------------------------------------------------------------------
// dh split along K: the slices' sum with the epilogue of EPI_DGLU.  One 64 x 64 tile a
// workgroup: a thread finishes eight columns of two rows, then, through LDS, 16 rows of
// one column of h^T.
// ---------------------------------------------------------------------------
template <int ACT, class PT>
__global__ void __launch_bounds__(256) dglu_split_kernel(DGluSplitArgs a) {
  __shared__ uint16_t s_h[64][72];  // 8 elements of padding a row
  const int64_t tiles_n = (a.F + 63) / 64;
  const int64_t m0 = (blockIdx.x / tiles_n) * 64, n0 = (blockIdx.x % tiles_n) * 64;
  const int t = threadIdx.x;
  const int64_t plane = a.M * a.F;
  const int rq = t >> 3, c = 8 * (t & 7);
  const int64_t col = n0 + c;
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    const int r = rq + 32 * v;
    const int64_t row = m0 + r;
    u16x8_t h = {0, 0, 0, 0, 0, 0, 0, 0};
    if (row < a.M && col < a.F) {  // F % 8 == 0: eight columns in or out together
      const float* x = a.part + row * a.F + col;
      f32x4_t s0 = *reinterpret_cast<const f32x4_t*>(x), s1 = *reinterpret_cast<const f32x4_t*>(x + 4);
#pragma unroll 4  // loads in flight together: 16 slices 7.2 us without
      for (int i = 1; i < a.splits; ++i) {
        s0 += *reinterpret_cast<const f32x4_t*>(x + i * plane);
        s1 += *reinterpret_cast<const f32x4_t*>(x + i * plane + 4);
      }
      const int64_t o = row * 2 * a.F + col;
      float gs[8], us[8];
      eight(static_cast<const PT*>(a.p) + o, gs);
      eight(static_cast<const PT*>(a.p) + o + a.F, us);
      u16x8_t dg, du;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float dh = e < 4 ? s0[e & 3] : s1[e & 3];
        float f, df;
        act_grad_f32<ACT>(gs[e], f, df);
        dg[e] = f32_to_bf16(dh * us[e] * df);
        du[e] = f32_to_bf16(dh * f);
        h[e] = f32_to_bf16(f * us[e]);
      }
      *reinterpret_cast<u16x8_t*>(a.dp + o) = dg;
      *reinterpret_cast<u16x8_t*>(a.dp + o + a.F) = du;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s_h[r][c + e] = h[e];
  }
  __syncthreads();
  const int ct = t >> 2, r0 = 16 * (t & 3);
  if (n0 + ct < a.F)
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int64_t row = m0 + r0 + 8 * v;
      if (row >= a.M) continue;
      u16x8_t hv;
#pragma unroll
      for (int e = 0; e < 8; ++e) hv[e] = s_h[r0 + 8 * v + e][ct];
      *reinterpret_cast<u16x8_t*>(a.ht + (n0 + ct) * a.ldt + row) = hv;
    }
}

struct ZeroArgs {
  void* p;
  int64_t n;  // bytes, a multiple of 16
};
__global__ void __launch_bounds__(256) glu_zero_kernel(ZeroArgs a) {
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 16; i < a.n; i += (int64_t)gridDim.x * 4096) *reinterpret_cast<f32x4_t*>(static_cast<char*>(a.p) + i) = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
}
hipError_t zero(void* p, int64_t bytes, hipStream_t s) {
  return launch_kernel(glu_zero_kernel, dim3((unsigned)std::min<int64_t>(2048, (bytes + 4095) / 4096)), dim3(256), s, ZeroArgs{p, bytes});
}

template <class A, class K1, class K2, class K3, class K4>
hipError_t launch_act(int act, int64_t blocks, const A& a, hipStream_t s, K1 silu, K2 gelu, K3 relu, K4 sigmoid) {
  void (*k)(A) = act == TPMLP_ACT_SILU ? silu : act == TPMLP_ACT_GELU ? gelu : act == TPMLP_ACT_RELU ? relu : sigmoid;
  return launch_kernel(k, dim3((unsigned)blocks), dim3(256), s, a);
}
#define BY_ACT(kernel, ...)                                                     \
  kernel<TPMLP_ACT_SILU __VA_ARGS__>, kernel<TPMLP_ACT_GELU __VA_ARGS__>, \
      kernel<TPMLP_ACT_RELU __VA_ARGS__>, kernel<TPMLP_ACT_SIGMOID __VA_ARGS__>

// ---------------------------------------------------------------------------
// Plans: functions of the sizes alone
// ---------------------------------------------------------------------------
// The forward's products in slices of 256 of K or more: 5 tokens by 1104 x 800 19.2 us with 512, 16.7
// so, 100 by 2048 x 1024 22.2 and 21.2, 64 by 4096 x 2048 28.1 and 29.1.  (The
// backward's lose by it: 64 by 4096 x 2048 50.7 and 54.6.)
constexpr int64_t FWD_SLICE = 256;

struct GluFwdPlan {
  bool tokens;  // a few tokens' kernels, with the slices of P at off_h and of Z at off_part
  GluTokensPlan t1, t2;
  GemmPlan g1, g2;
  bool wt;  // the products read A^T and B^T from the workspace
  size_t off_h, off_At, off_Bt, off_part, total;
};

GluFwdPlan plan_glu_fwd(int64_t M, int64_t H, int64_t F) {
  GluFwdPlan p{};
  p.tokens = glu_tokens(M, H, F);
  if (p.tokens) {
    p.t1 = plan_glu_tokens(M, 2 * F, H);
    p.t2 = plan_glu_tokens(M, H, F);
    p.off_part = align_up(size_t(p.t1.slices) * M * F * 8);
    p.total = p.off_part + align_up(size_t(p.t2.slices) * M * H * 4);
    return p;
  }
  p.g1 = plan_gemm(M, 2 * F, H, false, FWD_SLICE);
  p.g2 = plan_gemm(M, H, F, true, FWD_SLICE);
  p.wt = transpose_weights(M, H, F);
  p.off_h = 0;
  p.off_At = align_up(size_t(M) * F * 2);
  p.off_Bt = p.off_At + (p.wt ? align_up(size_t(H) * F * 4) : 0);
  p.off_part = p.off_Bt + (p.wt ? align_up(size_t(H) * F * 2) : 0);
  p.total = p.off_part + align_up(std::max(part_bytes(p.g1, M, 2 * F), part_bytes(p.g2, M, H)));
  return p;
}

// The products behind the activation in one launch (gemm_group.hip), each split along K or not, and one
// launch that adds the slices up: taken when the model gives it less time than three
// products.  The makespan is that of workgroups handed to free CUs in their order, the longest
// first.  A backward of 2048 tokens by 512 x 2048 67 -> 45 us, of 180 by 1104 x 800 38 -> 28, of
// 4305 by 64 x 408, where dB and dA are split, 44 -> 23; where it is not taken, one token by 4096
// x 2048, whose 1568 tiles have a K step each, 46 us, together 49.
constexpr int GROUP_TILE_STEPS = 3;  // what a tile takes beside its K steps, in steps: first loads and epilogue
constexpr int GROUP_MIN_STEPS = 8;   // of a slice

struct GroupPlan {
  bool on = false;
  int s_dx = 1, s_dw = 1;  // slices along K of dX, of dB and dA each
  int k_dx = 0, k_dw = 0;  // a slice's K
};

double group_steps(int64_t n0, int64_t k0, int64_t n1, int64_t k1) {
  const int64_t q = n0 / NUM_CU, r = n0 % NUM_CU;  // r CUs take one more of the first
  const int64_t t0 = q * k0, t1 = r ? t0 + k0 : t0;
  if (n1 == 0) return (double)t1;
  auto done = [&](int64_t at) {
    return (NUM_CU - r) * std::max<int64_t>(0, (at - t0) / k1) + r * std::max<int64_t>(0, (at - t1) / k1);
  };
  int64_t lo = t0, hi = t1 + (n1 + NUM_CU - 1) / NUM_CU * k1;  // the first time at which all are done
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (done(mid) < n1) lo = mid + 1;
    else hi = mid;
  }
  return (double)std::max(lo, t1);
}

GroupPlan plan_group(int64_t M, int64_t H, int64_t F, const GemmPlan& gdb, const GemmPlan& gda, const GemmPlan& gdx) {
  GroupPlan p;
  const int64_t tm = ceil_div(M, 128), th = ceil_div(H, 128), tf = ceil_div(F, 128), t2f = ceil_div(2 * F, 128);
  const int64_t n0 = tm * th, n1 = tf * th + th * t2f, k0 = ceil_div(2 * F, TILE_BK), k1 = ceil_div(M, TILE_BK);
  if (n0 + n1 > 8 * NUM_CU) return p;  // larger tiles are faster
  const double step = 128.0 * 128 * 2 * TILE_BK / CU_RATE_128;
  double best = gdb.seconds + gda.seconds + gdx.seconds + 2 * LAUNCH_S;
  for (int sx : {1, 2, 3, 4, 6, 8, 12, 16}) {
    const int64_t kx = (k0 + sx - 1) / sx;
    if ((sx > 1 && kx < GROUP_MIN_STEPS) || ceil_div(k0, kx) != sx) continue;
    for (int sw : {1, 2, 4, 8, 16}) {
      const int64_t kw = (k1 + sw - 1) / sw;
      if ((sw > 1 && kw < GROUP_MIN_STEPS) || ceil_div(k1, kw) != sw) continue;
      double t = step * (kx >= kw ? group_steps(n0 * sx, kx + GROUP_TILE_STEPS, n1 * sw, kw + GROUP_TILE_STEPS)
                                  : group_steps(n1 * sw, kw + GROUP_TILE_STEPS, n0 * sx, kx + GROUP_TILE_STEPS));
      if (sx > 1 || sw > 1) t += ((sx > 1 ? double(sx) * M * H : 0) + (sw > 1 ? double(sw) * 3 * H * F : 0)) * 4 * 2 / SPLIT_BW + LAUNCH_S;
      if (t < best * (1 - 1e-9)) {
        best = t;
        p = GroupPlan{true, sx, sw, (int)(kx * TILE_BK), (int)(kw * TILE_BK)};
      }
    }
  }
  return p;
}

struct GluBwdPlan {
  GemmPlan g0, g1, gdb, gda, gdx;
  GroupPlan group;
  bool wt, tdp, tdz;  // the recomputed product reads A^T; dA reads dP^T; dB reads dZ^T
  bool xt_beside;     // X is transposed by the launch that makes dh
  size_t off_Xt, off_dZt, off_At, off_P, off_ht, off_dP, off_dPt, off_part, total;
};

GluBwdPlan plan_glu_bwd(int64_t M, int64_t H, int64_t F, bool recompute) {
  GluBwdPlan p;
  const int64_t M8 = up8(M);
  p.g0 = plan_gemm(M, 2 * F, H);
  p.g1 = plan_gemm(M, F, H, false);
  p.gdb = plan_gemm(F, H, M);
  p.gda = plan_gemm(H, 2 * F, M);
  p.gdx = plan_gemm(M, H, 2 * F);
  p.wt = recompute && transpose_weights(M, H, F);
  p.group = plan_group(M, H, F, p.gdb, p.gda, p.gdx);
  // dZ^T pays as dP^T does, by F instead of H: 2048 tokens by 4096 x 2048 without it save 6 us of
  // transposing and lose 4 in dB.  Either is a launch as well, which few tokens' products do not earn
  // (4.4e-17 s a multiply-add of dB, twice that of dA).
  const bool large = double(M) * H * F * 4.4e-17 * 2 > LAUNCH_S;
  p.tdp = !p.group.on && large && transpose_dp(M, H, F);
  p.tdz = !p.group.on && large && transpose_dp(M, F, H);
  // Where the workgroups of both fit the chip at once, the transpose is hidden: 300 tokens by 520 x
  // 264 20.7 us after it, 18.0 beside it; 1001 by 1000 x 1368 with P made again (bf16 then) 62.6 and 59.3.
  const int64_t tiles = (int64_t)ceil_div(M, 128) * ceil_div(F, 128) * p.g1.splits;
  p.xt_beside = !p.tdz && p.g1.tile == TILE_128x128 && tiles + (int64_t)ceil_div(M, 256) * ceil_div(H, 64) <= NUM_CU;
  const size_t mh = align_up(size_t(M8) * H * 2), mf = align_up(size_t(M8) * F * 2), m2f = align_up(size_t(M8) * F * 4);
  p.off_Xt = 0;
  p.off_dZt = mh;
  p.off_At = mh + (p.tdz ? mh : 0);
  p.off_P = p.off_At + (p.wt ? align_up(size_t(H) * F * 4) : 0);
  p.off_ht = p.off_P + (recompute ? 2 * m2f : 0);  // in float32
  p.off_dP = p.off_ht + mf;
  p.off_dPt = p.off_dP + m2f;
  p.off_part = p.off_dPt + (p.tdp ? m2f : 0);
  size_t part = std::max(recompute ? part_bytes(p.g0, M, 2 * F) : 0, part_bytes(p.g1, M, F));
  if (p.group.on)
    part = std::max(part, (p.group.s_dx > 1 ? size_t(p.group.s_dx) * M * H * 4 : 0) + (p.group.s_dw > 1 ? size_t(p.group.s_dw) * 3 * H * F * 4 : 0));
  else part = std::max({part, part_bytes(p.gdb, F, H), part_bytes(p.gda, H, 2 * F), part_bytes(p.gdx, M, H)});
  p.total = p.off_part + align_up(part);
  return p;
}

bool glu_sizes_ok(int64_t M, int64_t H, int64_t F) {
  return M >= 0 && M <= MAX_DIM && H > 0 && H <= MAX_DIM && H % 8 == 0 && F > 0 && F <= MAX_DIM / 2 && F % 8 == 0;
}

template <class T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

// ---------------------------------------------------------------------------
// The launches
// ---------------------------------------------------------------------------
hipError_t enqueue_glu_fwd(const uint16_t* X, const uint16_t* A, const uint16_t* B, void* Z, Epi z_epi, uint16_t* P, int act,
                           int64_t M, int64_t H, int64_t F, const GluFwdPlan& p, void* ws, hipStream_t s) {
  uint16_t *h = at<uint16_t>(ws, p.off_h), *At = at<uint16_t>(ws, p.off_At), *Bt = at<uint16_t>(ws, p.off_Bt);
  float* part = at<float>(ws, p.off_part);
  hipError_t e;
  if (p.tokens) {
    float* P_slices = at<float>(ws, p.off_h);
    if ((e = launch_glu_tokens({X, nullptr, nullptr, A, P_slices, M, 2 * F, H, 0, act, 0}, p.t1, s)) != hipSuccess) return e;
    if ((e = launch_glu_tokens({nullptr, P_slices, P, B, part, M, H, F, p.t1.slices, act, 0}, p.t2, s)) != hipSuccess) return e;
    return launch_splitk_epilogue(z_epi, part, p.t2.slices, M, H, Z, nullptr, nullptr, H, M, s);
  }
  if (p.wt) {
    if ((e = launch_transpose(A, H, 2 * F, 2 * F, At, s)) != hipSuccess) return e;
    if ((e = launch_transpose(B, F, H, H, Bt, s)) != hipSuccess) return e;
  }
  // h = act(P_g) P_u        X: [M][H], A: [H][2 F] or A^T [2 F][H]
  if (p.g1.splits == 1) {
    GemmArgs g = gemm_args(X, H, p.wt ? At : A, p.wt ? H : 2 * F, M, F, H, p.g1, h, F);
    g.tiles_n = ceil_div(F, tile_bn(p.g1.tile) / 2);
    g.out2 = P;
    g.ldt = 2 * F;
    e = launch_gemm_glu(p.g1.tile, p.wt ? KC : MC, EPI_GLU, act, g, s);
  } else {
    GemmArgs g = gemm_args(X, H, p.wt ? At : A, p.wt ? H : 2 * F, M, 2 * F, H, p.g1, part, 2 * F);
    e = launch_gemm(p.g1.tile, KC, p.wt ? KC : MC, EPI_F32, g, p.g1.splits, s);
    if (e != hipSuccess) return e;
    const GluSplitArgs a{part, p.g1.splits, act, M, F, h, P};
    e = launch_act(act, std::min<int64_t>(2048, (M * F / 4 + 255) / 256), a, s, BY_ACT(glu_split_kernel));
  }
  if (e != hipSuccess) return e;
  // Z = h B                 h: [M][F], B: [F][H] or B^T [H][F]
  return run_gemm(-1, KC, p.wt ? KC : MC, z_epi, h, F, p.wt ? Bt : B, p.wt ? F : H, M, H, F, p.g2, Z, nullptr, nullptr, part, s);
}

hipError_t enqueue_glu_bwd(const uint16_t* dZ, const uint16_t* X, const uint16_t* A, const uint16_t* B, const uint16_t* P, void* dX,
                           Epi x_epi, void* dA, void* dB, Epi w_epi, int act, int64_t M, int64_t H, int64_t F,
                           const GluBwdPlan& p, void* ws, hipStream_t s) {
  const int64_t M8 = up8(M);
  uint16_t *Xt = at<uint16_t>(ws, p.off_Xt), *dZt = at<uint16_t>(ws, p.off_dZt), *ht = at<uint16_t>(ws, p.off_ht);
  uint16_t* dP = at<uint16_t>(ws, p.off_dP);
  float* part = at<float>(ws, p.off_part);
  hipError_t e = hipSuccess;
  if (!p.xt_beside && (e = launch_transpose2(X, Xt, p.tdz ? dZ : nullptr, dZt, M, H, H, s, M8)) != hipSuccess) return e;
  const bool again = !P;
  const void* p_in = P;
  if (again) {
    float* Pw = at<float>(ws, p.off_P);
    uint16_t* At = at<uint16_t>(ws, p.off_At);
    if (p.wt && (e = launch_transpose(A, H, 2 * F, 2 * F, At, s)) != hipSuccess) return e;
    // X as aux: P is read by the next launch (2048 x 4096, F 4096 480 us without, 464 so)
    e = run_gemm(-1, KC, p.wt ? KC : MC, EPI_F32, X, H, p.wt ? At : A, p.wt ? H : 2 * F, M, 2 * F, H, p.g0, Pw, nullptr, X,
                 part, s);
    if (e != hipSuccess) return e;
    p_in = Pw;
  }
  // dh = dZ B^T -> dP [M][2 F], h^T [F][M8]       dZ: [M][H], B: [F][H] = [N][K]
  if (p.g1.splits == 1) {
    GemmArgs g = gemm_args(dZ, H, B, H, M, F, H, p.g1, dP, 2 * F);
    g.out2 = ht;
    g.aux = static_cast<const uint16_t*>(p_in);
    g.ldt = M8;
    const Epi base = again ? EPI_DGLU32 : EPI_DGLU;
    e = p.xt_beside ? launch_gemm_transpose(g, 1, base, act, X, Xt, M, H, M8, s) : launch_gemm_glu(p.g1.tile, KC, base, act, g, s);
  } else {
    GemmArgs g = gemm_args(dZ, H, B, H, M, F, H, p.g1, part, F);
    e = p.xt_beside ? launch_gemm_transpose(g, p.g1.splits, EPI_F32, TPMLP_ACT_NONE, X, Xt, M, H, M8, s)
                    : launch_gemm(p.g1.tile, KC, KC, EPI_F32, g, p.g1.splits, s);
    if (e != hipSuccess) return e;
    const DGluSplitArgs a{part, p.g1.splits, act, M, F, M8, p_in, dP, ht};
    const int64_t blocks = ((M + 63) / 64) * ((F + 63) / 64);
    e = again ? launch_act(act, blocks, a, s, BY_ACT(dglu_split_kernel, , float))
              : launch_act(act, blocks, a, s, BY_ACT(dglu_split_kernel, , uint16_t));
  }
  if (e != hipSuccess) return e;
  if (p.group.on) {
    const GroupPlan& q = p.group;
    const int m = (int)M, h = (int)H, f = (int)F;
    const int tm = ceil_div(M, 128), th = ceil_div(H, 128);
    float* part_dw = part + (q.s_dx > 1 ? q.s_dx * M * H : 0);
    const bool xs = q.s_dx > 1, ws_ = q.s_dw > 1;
    const GroupItem items[GROUP_ITEMS] = {
        {dP, A, 2 * F, 2 * F, m, h, 2 * f, q.k_dx, xs ? part : dX, tm, th},
        {ht, dZ, M8, H, f, h, m, q.k_dw, ws_ ? part_dw : dB, ceil_div(F, 128), th},
        {Xt, dP, M8, 2 * F, h, 2 * f, m, q.k_dw, ws_ ? part_dw + q.s_dw * F * H : dA, th, ceil_div(2 * F, 128)}};
    e = launch_gemm_group(items, !xs && x_epi == EPI_BF16, !ws_ && w_epi == EPI_BF16, s);
    if (e != hipSuccess || !(xs || ws_)) return e;
    void* const outs[GROUP_ITEMS] = {xs ? dX : nullptr, ws_ ? dB : nullptr, ws_ ? dA : nullptr};
    return launch_group_sum(items, outs, x_epi == EPI_BF16, w_epi == EPI_BF16, s);
  }
  // dB = h^T dZ             h^T: [F][M8], dZ: [M][H] (rows past M masked) or dZ^T [H][M8]
  if (p.tdz) e = run_gemm(-1, KC, KC, w_epi, ht, M8, dZt, M8, F, H, M8, p.gdb, dB, nullptr, nullptr, part, s);
  else e = run_gemm(-1, KC, MC, w_epi, ht, M8, dZ, H, F, H, M, p.gdb, dB, nullptr, nullptr, part, s);
  if (e != hipSuccess) return e;
  // dA = X^T dP             X^T: [H][M8], dP: [M][2 F] (rows past M masked) or dP^T [2 F][M8]
  if (p.tdp) {
    uint16_t* dPt = at<uint16_t>(ws, p.off_dPt);
    if ((e = launch_transpose(dP, M, 2 * F, 2 * F, dPt, s, M8)) != hipSuccess) return e;
    e = run_gemm(-1, KC, KC, w_epi, Xt, M8, dPt, M8, H, 2 * F, M8, p.gda, dA, nullptr, nullptr, part, s);
  } else {
    e = run_gemm(-1, KC, MC, w_epi, Xt, M8, dP, 2 * F, H, 2 * F, M, p.gda, dA, nullptr, nullptr, part, s);
  }
  if (e != hipSuccess) return e;
  // dX = dP A^T             dP: [M][2 F], A: [H][2 F] = [N][K]
  return run_gemm(-1, KC, KC, x_epi, dP, 2 * F, A, 2 * F, M, H, 2 * F, p.gdx, dX, nullptr, nullptr, part, s);
}

tpmlp_status check_glu(int act, int64_t M, int64_t H, int64_t F) {
  if (!glu_sizes_ok(M, H, F))
    return fail(TPMLP_ERR_SHAPE, "M outside 0 .. 2^23, or H or F not a positive multiple of 8 up to 2^23 (F: 2^22)");
  if (act < TPMLP_ACT_SILU || act > TPMLP_ACT_SIGMOID) return fail(TPMLP_ERR_SHAPE, "act must be a tpmlp_act other than TPMLP_ACT_NONE");
  return TPMLP_OK;
}

tpmlp_status check_ws(const void* ws, size_t ws_bytes, size_t need, const char* query) {
  if (!ws) return fail(TPMLP_ERR_NULL, "ws is NULL");
  if (!aligned16(ws)) return fail(TPMLP_ERR_ALIGN, "ws is not 16-byte aligned");
  if (ws_bytes < need) return fail(TPMLP_ERR_WORKSPACE, std::string("ws_bytes below ") + query);
  return TPMLP_OK;
}

}  // namespace
}  // namespace tpmlp

using namespace tpmlp;

extern "C" {

size_t tpmlp_glu_fwd_workspace_bytes(int64_t M, int64_t H, int64_t F) {
  return glu_sizes_ok(M, H, F) && M > 0 ? plan_glu_fwd(M, H, F).total : 0;
}

size_t tpmlp_glu_bwd_workspace_bytes(int64_t M, int64_t H, int64_t F, int recompute) {
  return glu_sizes_ok(M, H, F) && M > 0 ? plan_glu_bwd(M, H, F, recompute != 0).total : 0;
}

tpmlp_status tpmlp_glu_fwd(const tpmlp_bf16* X, const tpmlp_bf16* A, const tpmlp_bf16* B, void* Z, int z_type, tpmlp_bf16* P_save,
                           int act, int64_t M, int64_t H, int64_t F, void* ws, size_t ws_bytes, void* stream) {
  return guarded([&]() -> tpmlp_status {
    TRY(check_glu(act, M, H, F));
    if (!type_ok(z_type)) return fail(TPMLP_ERR_SHAPE, "z_type must be a tpmlp_dtype");
    if (M == 0) return TPMLP_OK;
    TRY(check_ptrs({{X, "X"}, {A, "A"}, {B, "B"}, {Z, "Z"}}));
    if (P_save && !aligned16(P_save)) return fail(TPMLP_ERR_ALIGN, "P_save is not 16-byte aligned");
    const GluFwdPlan plan = plan_glu_fwd(M, H, F);
    const size_t need = plan.total, mh = size_t(M) * H, mf = size_t(M) * F, hf = size_t(H) * F;
    TRY(check_ws(ws, ws_bytes, need, "tpmlp_glu_fwd_workspace_bytes"));
    TRY(check_alias({{Z, mh * size_of(z_type), "Z"}, {P_save, mf * 4, "P_save"}, {ws, need, "ws"}},
                    {{X, mh * 2, "X"}, {A, hf * 4, "A"}, {B, hf * 2, "B"}}));
    TRY(check_device());
    return launched(enqueue_glu_fwd(X, A, B, Z, z_type == TPMLP_BF16 ? EPI_BF16 : EPI_F32, P_save, act, M, H, F, plan, ws,
                                    stream_of(stream)),
                    "tpmlp_glu_fwd launch");
  });
}

tpmlp_status tpmlp_glu_bwd(const tpmlp_bf16* dZ, const tpmlp_bf16* X, const tpmlp_bf16* A, const tpmlp_bf16* B,
                           const tpmlp_bf16* P_saved, void* dX, int dx_type, void* dA, void* dB, int dw_type, int act, int64_t M,
                           int64_t H, int64_t F, void* ws, size_t ws_bytes, void* stream) {
  return guarded([&]() -> tpmlp_status {
    TRY(check_glu(act, M, H, F));
    if (!type_ok(dx_type) || !type_ok(dw_type)) return fail(TPMLP_ERR_SHAPE, "dx_type and dw_type must be a tpmlp_dtype");
    const size_t mh = size_t(M) * H, mf = size_t(M) * F, hf = size_t(H) * F;
    const size_t xs = size_of(dx_type), wsz = size_of(dw_type);
    TRY(check_ptrs({{dA, "dA"}, {dB, "dB"}}));
    GluBwdPlan plan;
    size_t need = 0;
    if (M > 0) {
      TRY(check_ptrs({{dZ, "dZ"}, {X, "X"}, {A, "A"}, {B, "B"}, {dX, "dX"}}));
      if (P_saved && !aligned16(P_saved)) return fail(TPMLP_ERR_ALIGN, "P_saved is not 16-byte aligned");
      plan = plan_glu_bwd(M, H, F, P_saved == nullptr);
      need = plan.total;
      TRY(check_ws(ws, ws_bytes, need, "tpmlp_glu_bwd_workspace_bytes"));
    }
    TRY(check_alias({{dX, mh * xs, "dX"}, {dA, hf * 2 * wsz, "dA"}, {dB, hf * wsz, "dB"}, {ws, need, "ws"}},
                    {{dZ, mh * 2, "dZ"}, {X, mh * 2, "X"}, {A, hf * 4, "A"}, {B, hf * 2, "B"}, {P_saved, mf * 4, "P_saved"}}));
    TRY(check_device());
    hipStream_t s = stream_of(stream);
    if (M == 0) {  // sums over no tokens
      TRY(launched(zero(dA, (int64_t)(hf * 2 * wsz), s), "tpmlp_glu_bwd launch"));
      return launched(zero(dB, (int64_t)(hf * wsz), s), "tpmlp_glu_bwd launch");
    }
    return launched(enqueue_glu_bwd(dZ, X, A, B, P_saved, dX, dx_type == TPMLP_BF16 ? EPI_BF16 : EPI_F32, dA, dB,
                                    dw_type == TPMLP_BF16 ? EPI_BF16 : EPI_F32, act, M, H, F, plan, ws, s),
                    "tpmlp_glu_bwd launch");
  });
}

}  // extern "C"
