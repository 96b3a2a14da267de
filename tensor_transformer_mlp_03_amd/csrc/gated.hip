// C entry points of dropout and of the products with 4-bit weights (include/tpmlp.h):
// argument checks, all before any HIP call, and launches.  (The gated MLP's are in glu.hip,
// the edge's in block.hip.)

#include "checks.h"
#include "gated.h"

#include <cmath>

namespace tpmlp {
namespace {

constexpr int64_t MAX_SIZE = int64_t(1) << 23;  // of a row

// A matrix that one output may be the same as: left out of the overlap check if it is.
Mat unless_same(const Mat& m, const Mat& out) {
  Mat o = m;
  if (m.p == out.p && m.ld == out.ld && m.elem == out.elem) o.p = nullptr;
  return o;
}

tpmlp_status check_drop(int64_t M, int64_t H, float p, const uint64_t* state, int64_t first_row, uint32_t* drop, float* scale) {
  if (M < 0 || M > MAX_TOKENS || H < 1 || H > MAX_SIZE) return fail(TPMLP_ERR_SHAPE, "M outside 0 .. 2^23 or H outside 1 .. 2^23");
  if (!(p >= 0.0f && p <= 1.0f)) return fail(TPMLP_ERR_SHAPE, "p must be from 0 to 1");
  if (first_row < 0 || first_row > (int64_t(1) << 32) - M) return fail(TPMLP_ERR_SHAPE, "first_row negative, or first_row + M above 2^32");
  if (!state) return fail(TPMLP_ERR_NULL, "state is NULL");
  if (reinterpret_cast<uintptr_t>(state) & 7) return fail(TPMLP_ERR_ALIGN, "state is not aligned to its elements");
  *drop = (uint32_t)std::lround((double)p * 65536.0);
  *scale = *drop < 65536u ? (float)(65536.0 / (65536u - *drop)) : 0.0f;
  return TPMLP_OK;
}

template <size_t NO, size_t NI>
bool all_eights(int64_t H, const Mat (&outs)[NO], const Mat (&ins)[NI]) {
  auto eights = [](const Mat& m) { return starts_at(m, 8); };
  return H % 8 == 0 && std::all_of(outs, outs + NO, eights) && std::all_of(ins, ins + NI, eights);
}

tpmlp_status dropout_fwd(const void* y, int y_type, int64_t ld_y, const void* bias, int bias_type, const void* r, int64_t ld_r,
                         void* out, int out_type, int64_t ld_out, int64_t M, int64_t H, float p, const uint64_t* state,
                         uint32_t site, int64_t first_row, void* stream) {
  DropArgs a{};
  TRY(check_drop(M, H, p, state, first_row, &a.drop, &a.scale));
  if (!type_ok(y_type) || !type_ok(out_type) || (bias && !type_ok(bias_type)))
    return fail(TPMLP_ERR_SHAPE, "y_type, out_type and bias_type must be a tpmlp_dtype");
  const Mat my{y, M, H, ld_or(ld_y, H), size_of(y_type), "y"}, mr{r, M, H, ld_or(ld_r, H), size_of(out_type), "r"};
  const Mat mo{out, M, H, ld_or(ld_out, H), size_of(out_type), "out"}, mb{bias, 1, H, H, size_of(bias_type), "bias"};
  TRY(check_mat(my));
  TRY(check_mat(mo));
  if (r) TRY(check_mat(mr));
  if (bias) TRY(check_mat(mb));
  const Mat outs[] = {mo}, ins[] = {unless_same(my, mo), unless_same(mr, mo), mb, {state, 1, 2, 2, 8, "state"}};
  TRY(check_overlaps(outs, ins));
  if (M == 0) return TPMLP_OK;
  TRY(check_device());
  a.y = y;
  a.r = r;
  a.bias = bias;
  a.out = out;
  a.state = state;
  a.M = M;
  a.ld_y = my.ld;
  a.ld_r = mr.ld;
  a.ld_out = mo.ld;
  a.first_row = first_row;
  a.site = site;
  a.H = (int)H;
  a.groups = (int)((H + 7) / 8);
  a.bias_bf16 = bias_type == TPMLP_BF16;
  const Mat rows[] = {my, mr, mb};
  a.nt = past_caches(outs, rows);
  return launched(launch_drop(a, y_type, out_type, all_eights(H, outs, rows), stream_of(stream)), "tpmlp_dropout_fwd launch");
}

tpmlp_status dropout_bwd(const void* dout, int out_type, int64_t ld_dout, void* dy, int y_type, int64_t ld_dy, float* db, int64_t M,
                         int64_t H, float p, const uint64_t* state, uint32_t site, int64_t first_row, void* ws, size_t ws_bytes,
                         void* stream) {
  DropArgs a{};
  TRY(check_drop(M, H, p, state, first_row, &a.drop, &a.scale));
  if (!type_ok(y_type) || !type_ok(out_type)) return fail(TPMLP_ERR_SHAPE, "y_type and out_type must be a tpmlp_dtype");
  const Mat mg{dout, M, H, ld_or(ld_dout, H), size_of(out_type), "dout"}, my{dy, M, H, ld_or(ld_dy, H), size_of(y_type), "dy"};
  TRY(check_mat(mg));
  TRY(check_mat(my));
  const DropPlan plan = plan_drop(M, H);
  const Mat mb{db, 1, H, H, 4, "db"};
  int64_t ws_n = 0;
  if (db) {
    TRY(check_mat(mb));
    if (!ws) return fail(TPMLP_ERR_NULL, "ws is NULL");
    if (reinterpret_cast<uintptr_t>(ws) & 15) return fail(TPMLP_ERR_ALIGN, "ws is not 16-byte aligned");
    if (ws_bytes < plan.ws_bytes) return fail(TPMLP_ERR_WORKSPACE, "ws_bytes below tpmlp_dropout_bwd_workspace_bytes");
    ws_n = (int64_t)plan.ws_bytes;
  }
  const Mat outs[] = {my, mb, {ws, 1, ws_n, ws_n, 1, "ws"}}, ins[] = {unless_same(mg, my), {state, 1, 2, 2, 8, "state"}};
  TRY(check_overlaps(outs, ins));
  if (db && overlap(mb, mg)) return fail(TPMLP_ERR_ALIAS, "db overlaps dout");
  if (db && overlap(outs[2], mg)) return fail(TPMLP_ERR_ALIAS, "ws overlaps dout");
  if (M == 0 && !db) return TPMLP_OK;
  TRY(check_device());
  a.y = dout;
  a.out = dy;
  a.state = state;
  a.M = M;
  a.ld_y = mg.ld;
  a.ld_out = my.ld;
  a.first_row = first_row;
  a.site = site;
  a.H = (int)H;
  a.groups = (int)((H + 7) / 8);
  const Mat rows_out[] = {my}, rows_in[] = {mg};
  a.nt = past_caches(rows_out, rows_in);
  const bool full = all_eights(H, rows_out, rows_in);
  if (!db) return launched(launch_drop(a, out_type, y_type, full, stream_of(stream)), "tpmlp_dropout_bwd launch");
  a.part = static_cast<float*>(ws);
  a.chunk_rows = plan.chunk_rows;
  return launched(launch_drop_bias(a, plan, db, out_type, y_type, full, stream_of(stream)), "tpmlp_dropout_bwd launch");
}

tpmlp_status check_fp4(int64_t N, int64_t K) {
  if (N < 1 || N > MAX_SIZE || K < 32 || K > MAX_SIZE || K % 32)
    return fail(TPMLP_ERR_SHAPE, "N outside 1 .. 2^23, or K not a positive multiple of 32 up to 2^23");
  return TPMLP_OK;
}

tpmlp_status fp4_quantize(const tpmlp_bf16* W, int64_t ld_w, int64_t K, int64_t N, uint8_t* codes, uint8_t* scales, void* stream) {
  TRY(check_fp4(N, K));
  const Mat mw{W, K, N, ld_or(ld_w, N), 2, "W"}, mc{codes, N, K / 2, K / 2, 1, "codes"}, ms{scales, N, K / 32, K / 32, 1, "scales"};
  TRY(check_mat(mw));
  TRY(check_mat(mc));
  TRY(check_mat(ms));
  if (!aligned16(codes)) return fail(TPMLP_ERR_ALIGN, "codes is not 16-byte aligned");
  const Mat outs[] = {mc, ms}, ins[] = {mw};
  TRY(check_overlaps(outs, ins));
  TRY(check_device());
  return launched(launch_fp4_quantize(Fp4QuantArgs{W, codes, scales, mw.ld, (int)K, (int)N}, stream_of(stream)),
                  "tpmlp_fp4_quantize launch");
}

Mat packed_mat(const void* p, int64_t N, int64_t K, int gated) {
  const int64_t n = fp4_packed_bytes(N, K, gated != 0);
  return Mat{p, 1, n, n, 1, "packed"};
}

// check_mat but for the length of a row, which may pass its limit.
tpmlp_status check_bytes(const Mat& m) {
  if (!m.p) return fail(TPMLP_ERR_NULL, std::string(m.name) + " is NULL");
  if (!aligned16(m.p)) return fail(TPMLP_ERR_ALIGN, std::string(m.name) + " is not 16-byte aligned");
  return TPMLP_OK;
}

tpmlp_status fp4_pack(const uint8_t* codes, const uint8_t* scales, void* packed, int gated, int64_t N, int64_t K, void* stream) {
  TRY(check_fp4(N, K));
  const int64_t rows = gated ? 2 * N : N;
  const Mat c{codes, rows, K / 2, K / 2, 1, "codes"}, sc{scales, rows, K / 32, K / 32, 1, "scales"}, p = packed_mat(packed, N, K, gated);
  TRY(check_mat(c));
  TRY(check_mat(sc));
  if (!aligned16(codes)) return fail(TPMLP_ERR_ALIGN, "codes is not 16-byte aligned");
  TRY(check_bytes(p));
  const Mat outs[] = {p}, ins[] = {c, sc};
  TRY(check_overlaps(outs, ins));
  TRY(check_device());
  return launched(launch_fp4_pack(Fp4PackArgs{codes, scales, packed, (int)N, (int)K, gated != 0}, stream_of(stream)),
                  "tpmlp_fp4_pack launch");
}

tpmlp_status fp4_fwd(const void* X, int x_kind, int64_t ld_x, const void* x_scales, const void* packed, void* Y, int y_type,
                     int64_t ld_y, int act, int gated, int64_t M, int64_t N, int64_t K, void* stream) {
  TRY(check_fp4(N, K));
  if (M < 0 || M > MAX_TOKENS) return fail(TPMLP_ERR_SHAPE, "M outside 0 .. 2^23");
  if (x_kind < TPMLP_X_BF16 || x_kind > TPMLP_X_E4M3_MX) return fail(TPMLP_ERR_SHAPE, "x_kind must be a tpmlp_x");
  if (act < TPMLP_ACT_NONE || act > TPMLP_ACT_SIGMOID) return fail(TPMLP_ERR_SHAPE, "act must be a tpmlp_act");
  if (!type_ok(y_type)) return fail(TPMLP_ERR_SHAPE, "y_type must be a tpmlp_dtype");
  const bool bf16 = x_kind == TPMLP_X_BF16, mx = x_kind == TPMLP_X_E4M3_MX;
  const Mat x{X, M, K, ld_or(ld_x, K), bf16 ? 2 : 1, "X"}, y{Y, M, N, ld_or(ld_y, N), size_of(y_type), "Y"};
  const Mat p = packed_mat(packed, N, K, gated);
  Mat xs{nullptr, 0, 1, 1, 1, "x_scales"};
  if (mx) xs = Mat{x_scales, M, K / 32, K / 32, 1, "x_scales"};
  else if (!bf16) xs = Mat{x_scales, M > 0 ? 1 : 0, M, M, 4, "x_scales"};
  else if (x_scales) return fail(TPMLP_ERR_SHAPE, "x_scales is given with a bf16 X");
  for (const Mat& m : {x, y, xs}) TRY(check_mat(m));
  TRY(check_bytes(p));
  if (!starts_at(x, bf16 ? 8 : 16)) return fail(TPMLP_ERR_ALIGN, "the rows of X do not start at multiples of 16 bytes");
  const Mat outs[] = {y}, ins[] = {x, xs, p};
  TRY(check_overlaps(outs, ins));
  if (M == 0) return TPMLP_OK;
  TRY(check_device());
  Fp4Args a{};
  a.x = X;
  a.x_scale = x_scales;
  a.w = packed;
  a.y = Y;
  a.M = M;
  a.ld_x = x.ld;
  a.ld_y = y.ld;
  a.N = (int)N;
  a.K = (int)K;
  a.act = act;
  a.gated = gated != 0;
  a.x_kind = x_kind;
  a.y_bf16 = y_type == TPMLP_BF16;
  a.y_vec = N % 4 == 0 && starts_at(y, 4);
  return launched(launch_fp4(a, stream_of(stream)), "tpmlp_fp4_fwd launch");
}

}  // namespace
}  // namespace tpmlp

using namespace tpmlp;

extern "C" {

tpmlp_status tpmlp_dropout_fwd(const void* y, int y_type, int64_t ld_y, const void* bias, int bias_type, const void* r,
                               int64_t ld_r, void* out, int out_type, int64_t ld_out, int64_t M, int64_t H, float p,
                               const uint64_t* state, uint32_t site, int64_t first_row, void* stream) {
  return guarded([&] {
    return dropout_fwd(y, y_type, ld_y, bias, bias_type, r, ld_r, out, out_type, ld_out, M, H, p, state, site, first_row, stream);
  });
}

size_t tpmlp_dropout_bwd_workspace_bytes(int64_t M, int64_t H) {
  return M < 0 || M > MAX_TOKENS || H < 1 || H > MAX_SIZE ? 0 : plan_drop(M, H).ws_bytes;
}

tpmlp_status tpmlp_dropout_bwd(const void* dout, int out_type, int64_t ld_dout, void* dy, int y_type, int64_t ld_dy, float* db,
                               int64_t M, int64_t H, float p, const uint64_t* state, uint32_t site, int64_t first_row, void* ws,
                               size_t ws_bytes, void* stream) {
  return guarded([&] {
    return dropout_bwd(dout, out_type, ld_dout, dy, y_type, ld_dy, db, M, H, p, state, site, first_row, ws, ws_bytes, stream);
  });
}

tpmlp_status tpmlp_fp4_quantize(const tpmlp_bf16* W, int64_t ld_w, int64_t K, int64_t N, uint8_t* codes, uint8_t* scales,
                                void* stream) {
  return guarded([&] { return fp4_quantize(W, ld_w, K, N, codes, scales, stream); });
}

size_t tpmlp_fp4_packed_bytes(int64_t N, int64_t K, int gated) {
  return N < 1 || N > MAX_SIZE || K < 32 || K > MAX_SIZE || K % 32 ? 0 : (size_t)fp4_packed_bytes(N, K, gated != 0);
}

tpmlp_status tpmlp_fp4_pack(const uint8_t* codes, const uint8_t* scales, void* packed, int gated, int64_t N, int64_t K,
                            void* stream) {
  return guarded([&] { return fp4_pack(codes, scales, packed, gated, N, K, stream); });
}

tpmlp_status tpmlp_fp4_fwd(const void* X, int x_kind, int64_t ld_x, const void* x_scales, const void* packed, void* Y,
                           int y_type, int64_t ld_y, int act, int gated, int64_t M, int64_t N, int64_t K, void* stream) {
  return guarded([&] { return fp4_fwd(X, x_kind, ld_x, x_scales, packed, Y, y_type, ld_y, act, gated, M, N, K, stream); });
}

}  // extern "C"
