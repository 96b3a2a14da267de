// C entry points of the block operators (include/tpmlp.h): argument checks, all
// before any HIP call, and launches.  Nothing thrown crosses the boundary.

#include "block.h"
#include "checks.h"

#include <algorithm>
#include <cmath>
#include <new>
#include <string>
#include <utility>
#include <vector>

namespace tpmlp {
namespace {

constexpr int64_t MAX_ROWS = INT32_MAX;           // of a sorted buffer
constexpr int64_t MAX_H = int64_t(1) << 23;
constexpr int64_t MAX_GATES = int64_t(1) << 21;   // rows of the gate: a workgroup of the backward each

// ---------------------------------------------------------------------------
// Edge
// ---------------------------------------------------------------------------
int64_t gate_rows_of(const tpmlp_edge& e) {
  return e.gate ? std::min(e.gate_rows, std::max<int64_t>(e.M, 1)) : std::max<int64_t>(e.M, 1);
}
int64_t gate_groups(const tpmlp_edge& e) { return e.gate ? (e.M + gate_rows_of(e) - 1) / gate_rows_of(e) : 0; }
bool has_layer(const tpmlp_edge& e) { return e.post == TPMLP_NORM_LAYER || e.pre == TPMLP_NORM_LAYER; }

tpmlp_status check_edge(const tpmlp_edge* e, bool has_y) {
  if (!e) return fail(TPMLP_ERR_NULL, "the edge is NULL");
  if (e->M < 0 || e->M > MAX_TOKENS) return fail(TPMLP_ERR_SHAPE, "M outside 0 .. 2^23");
  if (e->H < 8 || e->H > TPMLP_EDGE_MAX_H) return fail(TPMLP_ERR_SHAPE, "H outside 8 .. TPMLP_EDGE_MAX_H");
  for (int n : {e->post, e->pre})
    if (n < TPMLP_NORM_NONE || n > TPMLP_NORM_LAYER) return fail(TPMLP_ERR_SHAPE, "post and pre must be a tpmlp_norm");
  if (!type_ok(e->y_type) || !type_ok(e->r_type) || !type_ok(e->param_type))
    return fail(TPMLP_ERR_SHAPE, "y_type, r_type and param_type must be a tpmlp_dtype");
  if (!std::isfinite(e->alpha) || !std::isfinite(e->eps) || e->eps < 0.0f)
    return fail(TPMLP_ERR_SHAPE, "alpha and eps must be finite, eps at least 0");
  if (!has_y && (e->post != TPMLP_NORM_NONE || e->gate)) return fail(TPMLP_ERR_NULL, "y is NULL, but it has a norm or a gate");
  const int ps = size_of(e->param_type);
  const struct {
    const void *w, *b;
    int norm;
    const char *wn, *bn;
  } sides[2] = {{e->w_post, e->b_post, e->post, "w_post", "b_post"}, {e->w_pre, e->b_pre, e->pre, "w_pre", "b_pre"}};
  for (auto& s : sides) {
    if (s.norm == TPMLP_NORM_NONE && s.w) return fail(TPMLP_ERR_SHAPE, std::string(s.wn) + " is given without a norm");
    if (s.norm != TPMLP_NORM_LAYER && s.b) return fail(TPMLP_ERR_SHAPE, std::string(s.bn) + " is given without a LayerNorm");
    if (s.norm != TPMLP_NORM_NONE) TRY(check_mat({s.w, 1, e->H, e->H, ps, s.wn}));
    if (s.b) TRY(check_mat({s.b, 1, e->H, e->H, ps, s.bn}));
  }
  if (e->gate) {
    if (e->gate_rows < 1) return fail(TPMLP_ERR_SHAPE, "gate_rows must be positive");
    if (gate_groups(*e) > MAX_GATES) return fail(TPMLP_ERR_SHAPE, "gate_rows gives a gate of more than 2^21 rows");
    TRY(check_mat({e->gate, gate_groups(*e), e->H, ld_or(e->ld_gate, e->H), ps, "gate"}));
  }
  return TPMLP_OK;
}

// The edge's parameters as inputs of the overlap check.
#define EDGE_PARAMS(e)                                                                                  \
  {(e).w_post, 1, (e).H, (e).H, size_of((e).param_type), "w_post"},                                     \
      {(e).b_post, 1, (e).H, (e).H, size_of((e).param_type), "b_post"},                                 \
      {(e).w_pre, 1, (e).H, (e).H, size_of((e).param_type), "w_pre"},                                   \
      {(e).b_pre, 1, (e).H, (e).H, size_of((e).param_type), "b_pre"}, {                                 \
    (e).gate, gate_groups(e), (e).H, ld_or((e).ld_gate, (e).H), size_of((e).param_type), "gate"         \
  }

// The forward's output in 8 bits: codes in place of x, with scales.
struct EdgeCodes {
  uint8_t* codes;
  int64_t ld;
  void* scales;
  int64_t ld_scales;
  int kind;
};

tpmlp_status edge_fwd(const tpmlp_edge* e, const void* y, int64_t ld_y, const void* r, int64_t ld_r, void* r_out,
                      int64_t ld_r_out, tpmlp_bf16* x, int64_t ld_x, const EdgeCodes* c, void* stream) {
  const bool has_y = y != nullptr || (e && e->M == 0);
  TRY(check_edge(e, has_y));
  const int64_t M = e->M, H = e->H;
  const int ys = size_of(e->y_type), rs = size_of(e->r_type);
  if (e->pre == TPMLP_NORM_NONE && x) return fail(TPMLP_ERR_SHAPE, "x is given without a norm before the next block");
  Mat mx{x, M, H, ld_or(ld_x, H), 2, "x"}, ms{nullptr, 0, 1, 1, 1, "scales"};
  if (c) {
    if (e->pre == TPMLP_NORM_NONE) return fail(TPMLP_ERR_SHAPE, "codes need a norm before the next block");
    if (c->kind != TPMLP_SCALE_ROW && c->kind != TPMLP_SCALE_MX) return fail(TPMLP_ERR_SHAPE, "scale_kind must be a tpmlp_scale");
    if (c->kind == TPMLP_SCALE_MX && H % 32) return fail(TPMLP_ERR_SHAPE, "H must be a multiple of 32 with TPMLP_SCALE_MX");
    if (c->kind == TPMLP_SCALE_ROW && c->ld_scales) return fail(TPMLP_ERR_SHAPE, "ld_scales must be 0 with TPMLP_SCALE_ROW");
    mx = Mat{c->codes, M, H, ld_or(c->ld, H), 1, "codes"};
    if (c->kind == TPMLP_SCALE_MX) ms = Mat{c->scales, M, H / 32, ld_or(c->ld_scales, H / 32), 1, "scales"};
    else ms = Mat{c->scales, M > 0 ? 1 : 0, M, M, 4, "scales"};
    TRY(check_mat(ms));
  }
  const Mat my{y, M, H, ld_or(ld_y, H), ys, "y"}, mr{r, M, H, ld_or(ld_r, H), rs, "r"};
  const Mat mo{r_out, M, H, ld_or(ld_r_out, H), rs, "r_out"};
  TRY(check_mat(mr));
  if (y) TRY(check_mat(my));
  if (r_out || e->pre == TPMLP_NORM_NONE) TRY(check_mat(mo));
  if (e->pre != TPMLP_NORM_NONE) TRY(check_mat(mx));
  const Mat outs[] = {mo, mx, ms}, ins[] = {mr, my, EDGE_PARAMS(*e)};
  TRY(check_overlaps(outs, ins, 0, 0));
  if (M == 0) return TPMLP_OK;
  TRY(check_device());
  EdgeFwdArgs a{};
  a.y = y;
  a.r = r;
  a.r_out = r_out;
  a.x = c ? reinterpret_cast<uint16_t*>(c->codes) : x;
  a.w_post = e->w_post;
  a.b_post = e->b_post;
  a.gate = e->gate;
  a.w_pre = e->w_pre;
  a.b_pre = e->b_pre;
  a.ld_y = my.ld;
  a.ld_r = mr.ld;
  a.ld_r_out = mo.ld;
  a.ld_x = mx.ld;
  a.ld_gate = ld_or(e->ld_gate, H);
  a.M = M;
  a.gate_rows = gate_rows_of(*e);
  a.H = (int)H;
  a.post = e->post;
  a.pre = e->pre;
  a.p_bf16 = e->param_type == TPMLP_BF16;
  a.alpha = e->alpha;
  a.eps = e->eps;
  const int y_type = y ? e->y_type : -1;
  if (c) {
    a.scales = c->scales;
    a.ld_scales = ms.ld;
    a.scale_mx = c->kind == TPMLP_SCALE_MX;
    a.nt = past_caches(outs, ins);
    const Mat rows[] = {mo, mx};
    return launched(launch_edge_fwd_fp8(a, y_type, e->r_type, all_quads(H, rows, ins), stream_of(stream)), "tpmlp_edge_fwd_fp8 launch");
  }
  const Mat rows[] = {mo, mx};
  a.nt = past_caches(rows, ins);
  return launched(launch_edge_fwd(a, y_type, e->r_type, all_quads(H, rows, ins), stream_of(stream)), "tpmlp_edge_fwd launch");
}

tpmlp_status edge_bwd(const tpmlp_edge* e, const void* y, int64_t ld_y, const void* r_out, int64_t ld_r_out,
                      const void* dr_out, int64_t ld_dr_out, const void* dx, int dx_type, int64_t ld_dx, void* dr,
                      int64_t ld_dr, tpmlp_bf16* dy, int64_t ld_dy, float* dw_post, float* db_post, float* dw_pre,
                      float* db_pre, float* dgate, void* ws, size_t ws_bytes, void* stream) {
  const bool has_y = y != nullptr || (e && e->M == 0);
  TRY(check_edge(e, has_y));
  const int64_t M = e->M, H = e->H;
  const bool pre = e->pre != TPMLP_NORM_NONE;
  const int ys = size_of(e->y_type), rs = size_of(e->r_type);
  if (pre && !type_ok(dx_type)) return fail(TPMLP_ERR_SHAPE, "dx_type must be a tpmlp_dtype");
  if (!pre && (dx || r_out)) return fail(TPMLP_ERR_SHAPE, "dx or r_out is given without a norm before the next block");
  if (!y && M > 0 && dy) return fail(TPMLP_ERR_SHAPE, "dy is given without y");
  if (dw_post && !e->w_post) return fail(TPMLP_ERR_SHAPE, "dw_post is given without w_post");
  if (db_post && !e->b_post) return fail(TPMLP_ERR_SHAPE, "db_post is given without b_post");
  if (dw_pre && !e->w_pre) return fail(TPMLP_ERR_SHAPE, "dw_pre is given without w_pre");
  if (db_pre && !e->b_pre) return fail(TPMLP_ERR_SHAPE, "db_pre is given without b_pre");
  if (dgate && !e->gate) return fail(TPMLP_ERR_SHAPE, "dgate is given without a gate");
  const Mat my{y, M, H, ld_or(ld_y, H), ys, "y"}, mr{r_out, M, H, ld_or(ld_r_out, H), rs, "r_out"};
  const Mat mdo{dr_out, M, H, ld_or(ld_dr_out, H), rs, "dr_out"};
  const Mat mdx{dx, M, H, ld_or(ld_dx, H), size_of(dx_type), "dx"};
  const Mat mdr{dr, M, H, ld_or(ld_dr, H), rs, "dr"}, mdy{dy, M, H, ld_or(ld_dy, H), 2, "dy"};
  TRY(check_mat(mdr));
  if (y) {
    TRY(check_mat(my));
    TRY(check_mat(mdy));
  }
  if (pre) {
    TRY(check_mat(mr));
    TRY(check_mat(mdx));
  }
  if (dr_out || !pre) TRY(check_mat(mdo));
  const Mat g[] = {{dw_post, 1, H, H, 4, "dw_post"},
                   {db_post, 1, H, H, 4, "db_post"},
                   {dw_pre, 1, H, H, 4, "dw_pre"},
                   {db_pre, 1, H, H, 4, "db_pre"},
                   {dgate, gate_groups(*e), H, H, 4, "dgate"}};
  bool any = false;
  for (const Mat& m : g) {
    TRY(check_mat({m.p, 0, H, H, 4, m.name}));
    any |= m.p != nullptr;
  }
  const EdgeBwdPlan plan = plan_edge_bwd(M, (int)H, gate_rows_of(*e), has_layer(*e));
  const bool use_ws = (any || edge_bwd_wide((int)H)) && plan.ws_bytes;
  if (use_ws) {
    if (!ws) return fail(TPMLP_ERR_NULL, "ws is NULL");
    if (reinterpret_cast<uintptr_t>(ws) & 15) return fail(TPMLP_ERR_ALIGN, "ws is not 16-byte aligned");
    if (ws_bytes < plan.ws_bytes) return fail(TPMLP_ERR_WORKSPACE, "ws_bytes below tpmlp_edge_bwd_workspace_bytes");
  }
  const int64_t ws_n = use_ws ? (int64_t)(plan.ws_bytes / 4) : 0;
  const Mat outs[] = {mdr, mdy, g[0], g[1], g[2], g[3], g[4], {ws, 1, ws_n, ws_n, 4, "ws"}};
  const Mat ins[] = {mdo, my, mr, mdx, EDGE_PARAMS(*e)};
  TRY(check_overlaps(outs, ins, 0, 0));
  if (M == 0 && !any) return TPMLP_OK;
  TRY(check_device());
  hipStream_t s = stream_of(stream);
  if (M > 0) {
    EdgeBwdArgs a{};
    a.y = y;
    a.r = r_out;
    a.dr_out = dr_out;
    a.dx = dx;
    a.dr = dr;
    a.dy = dy;
    a.w_post = e->w_post;
    a.gate = e->gate;
    a.w_pre = e->w_pre;
    a.part = any ? static_cast<float*>(ws) : nullptr;
    a.terms = edge_bwd_wide((int)H) ? reinterpret_cast<float*>(static_cast<char*>(ws) + plan.part_bytes) : nullptr;
    a.ld_y = my.ld;
    a.ld_r = mr.ld;
    a.ld_dr_out = mdo.ld;
    a.ld_dx = mdx.ld;
    a.ld_dr = mdr.ld;
    a.ld_dy = mdy.ld;
    a.ld_gate = ld_or(e->ld_gate, H);
    a.M = M;
    a.gate_rows = gate_rows_of(*e);
    a.chunks = plan.chunks;
    a.H = (int)H;
    a.post = e->post;
    a.pre = e->pre;
    a.p_bf16 = e->param_type == TPMLP_BF16;
    a.dx_bf16 = dx_type == TPMLP_BF16;
    a.alpha = e->alpha;
    a.eps = e->eps;
    a.nt = past_caches(outs, ins);
    TRY(launched(launch_edge_bwd(a, plan, y ? e->y_type : -1, e->r_type, all_quads(H, outs, ins), s), "tpmlp_edge_bwd launch"));
  }
  if (!any) return TPMLP_OK;
  EdgeFinishArgs f{};
  f.part = static_cast<const float*>(ws);
  f.w_post = e->w_post;
  f.b_post = e->b_post;
  f.gate = e->gate;
  f.dw_post = dw_post;
  f.db_post = db_post;
  f.dgate = dgate;
  f.dw_pre = dw_pre;
  f.db_pre = db_pre;
  f.groups = plan.groups;
  f.ld_gate = ld_or(e->ld_gate, H);
  f.chunks = plan.chunks;
  f.n_acc = plan.n_acc;
  f.H = (int)H;
  f.p_bf16 = e->param_type == TPMLP_BF16;
  return launched(launch_edge_finish(f, s), "tpmlp_edge_bwd launch");
}

// ---------------------------------------------------------------------------
// Route
// ---------------------------------------------------------------------------
bool pairs_ok(int64_t T, int K) {
  return T >= 0 && T <= MAX_TOKENS && K >= 1 && K <= TPMLP_ROUTE_MAX_CHOICES;
}

tpmlp_status check_route(int64_t T, int K, int64_t H, int64_t rows) {
  if (!pairs_ok(T, K)) return fail(TPMLP_ERR_SHAPE, "T outside 0 .. 2^23 or K outside 1 .. TPMLP_ROUTE_MAX_CHOICES");
  if (H < 8 || H > MAX_H) return fail(TPMLP_ERR_SHAPE, "H outside 8 .. 2^23");
  if (rows < 0 || rows > MAX_ROWS) return fail(TPMLP_ERR_SHAPE, "rows outside 0 .. 2^31 - 1");
  return TPMLP_OK;
}

tpmlp_status route_sort(const void* ids, int id_bits, int64_t T, int K, int E, int align, int capacity, int32_t* counts,
                        int32_t* offsets, int32_t* row_of, int32_t* src_of, void* ws, size_t ws_bytes, void* stream) {
  if (id_bits != 32 && id_bits != 64) return fail(TPMLP_ERR_SHAPE, "id_bits must be 32 or 64");
  const int64_t rows = tpmlp_route_rows(T, K, E, align, capacity);
  if (rows < 0)
    return fail(TPMLP_ERR_SHAPE, "T, K, E, align or capacity out of range (tpmlp_route_rows), or capacity not a multiple of align");
  const int64_t pairs = T * K;
  const size_t need = tpmlp_route_workspace_bytes(T, K, E);
  const Mat outs[] = {{counts, 1, E, E, 4, "counts"},
                      {offsets, 1, E + 1, E + 1, 4, "offsets"},
                      {row_of, 1, pairs, pairs, 4, "row_of"},
                      {src_of, 1, rows, rows, 4, "src_of"},
                      {ws, 1, (int64_t)need, (int64_t)need, 4, "ws"}};
  const Mat ins[] = {{ids, 1, pairs, pairs, id_bits / 8, "ids"}};
  for (const Mat& m : outs) TRY(check_mat({m.p, m.cols ? 1 : 0, m.cols, m.cols, m.elem, m.name}));
  TRY(check_mat(ins[0]));
  if (ws_bytes < need) return fail(TPMLP_ERR_WORKSPACE, "ws_bytes below tpmlp_route_workspace_bytes");
  const Mat outs_b[] = {outs[0], outs[1], outs[2], outs[3], {ws, 1, (int64_t)need, (int64_t)need, 1, "ws"}};
  TRY(check_overlaps(outs_b, ins));
  TRY(check_device());
  RouteSortArgs a{};
  a.ids = ids;
  a.ids64 = id_bits == 64;
  a.pairs = pairs;
  a.rows = rows;
  a.E = E;
  a.align = align;
  a.capacity = capacity;
  a.counts = counts;
  a.offsets = offsets;
  a.row_of = row_of;
  a.src_of = src_of;
  a.hist = static_cast<int32_t*>(ws);
  a.blocks = (int)route_sort_blocks(pairs, &a.per_block);
  return launched(launch_route_sort(a, stream_of(stream)), "tpmlp_route_sort launch");
}

tpmlp_status route_dispatch(const tpmlp_bf16* X, int64_t ld_x, const int32_t* row_of, const int32_t* src_of, int64_t T,
                            int K, int64_t H, int64_t rows, tpmlp_bf16* Xs, int64_t ld_xs, void* stream) {
  TRY(check_route(T, K, H, rows));
  const Mat outs[] = {{Xs, rows, H, ld_or(ld_xs, H), 2, "Xs"}};
  const Mat ins[] = {{X, T, H, ld_or(ld_x, H), 2, "X"},
                     {row_of, 1, T * K, T * K, 4, "row_of"},
                     {src_of, 1, rows, rows, 4, "src_of"}};
  TRY(check_mat(outs[0]));
  for (const Mat& m : ins) TRY(check_mat(m));
  TRY(check_overlaps(outs, ins));
  if (rows == 0) return TPMLP_OK;
  TRY(check_device());
  RouteDispatchArgs a{};
  a.x = X;
  a.xs = Xs;
  a.row_of = row_of;
  a.src_of = src_of;
  a.T = T;
  a.rows = rows;
  a.ld_x = ins[0].ld;
  a.ld_xs = outs[0].ld;
  a.K = K;
  a.H = (int)H;
  return launched(launch_route_dispatch(a, H % 8 == 0 && starts_at(outs[0], 8) && starts_at(ins[0], 8),
                                        past_caches(outs, ins), stream_of(stream)), "tpmlp_route_dispatch launch");
}

tpmlp_status route_combine(const void* Zs, int z_type, int64_t ld_zs, const int32_t* row_of, const float* w, int64_t T,
                           int K, int64_t H, int64_t rows, void* Y, int y_type, int64_t ld_y, void* stream) {
  TRY(check_route(T, K, H, rows));
  if (!type_ok(z_type) || !type_ok(y_type)) return fail(TPMLP_ERR_SHAPE, "z_type and y_type must be a tpmlp_dtype");
  const Mat outs[] = {{Y, T, H, ld_or(ld_y, H), size_of(y_type), "Y"}};
  const Mat ins[] = {{Zs, rows, H, ld_or(ld_zs, H), size_of(z_type), "Zs"},
                     {row_of, 1, T * K, T * K, 4, "row_of"},
                     {w, w ? 1 : 0, T * K, T * K, 4, "w"}};
  TRY(check_mat(outs[0]));
  for (const Mat& m : ins) TRY(check_mat(m));
  TRY(check_overlaps(outs, ins));
  if (T == 0) return TPMLP_OK;
  TRY(check_device());
  RouteCombineArgs a{};
  a.zs = Zs;
  a.y = Y;
  a.w = w;
  a.row_of = row_of;
  a.T = T;
  a.rows = rows;
  a.ld_zs = ins[0].ld;
  a.ld_y = outs[0].ld;
  a.K = K;
  a.H = (int)H;
  return launched(launch_route_combine(a, z_type, y_type, H % 4 == 0 && quads(outs[0]) && quads(ins[0]),
                                       past_caches(outs, ins), stream_of(stream)), "tpmlp_route_combine launch");
}

tpmlp_status route_combine_bwd(const void* dY, int dy_type, int64_t ld_dy, const void* Zs, int z_type, int64_t ld_zs,
                               const int32_t* row_of, const int32_t* src_of, const float* w, int64_t T, int K, int64_t H,
                               int64_t rows, tpmlp_bf16* dZs, int64_t ld_dzs, float* dw, void* stream) {
  TRY(check_route(T, K, H, rows));
  if (!type_ok(dy_type) || !type_ok(z_type)) return fail(TPMLP_ERR_SHAPE, "dy_type and z_type must be a tpmlp_dtype");
  const bool want_z = rows > 0 && dZs, want_w = T > 0 && dw;
  if (rows > 0 && !dZs != !src_of) return fail(TPMLP_ERR_NULL, "dZs and src_of must be given together");
  if (rows > 0 && T > 0 && !dw != !Zs) return fail(TPMLP_ERR_NULL, "dw and Zs must be given together");
  if (rows > 0 && T > 0 && !dZs && !dw) return fail(TPMLP_ERR_NULL, "dZs and dw are NULL");
  const Mat outs[] = {{dZs, want_z ? rows : 0, H, ld_or(ld_dzs, H), 2, "dZs"}, {dw, want_w ? 1 : 0, T * K, T * K, 4, "dw"}};
  const Mat ins[] = {{dY, T, H, ld_or(ld_dy, H), size_of(dy_type), "dY"},
                     {Zs, want_w ? rows : 0, H, ld_or(ld_zs, H), size_of(z_type), "Zs"},
                     {row_of, 1, T * K, T * K, 4, "row_of"},
                     {src_of, want_z ? 1 : 0, rows, rows, 4, "src_of"},
                     {w, w ? 1 : 0, T * K, T * K, 4, "w"}};
  for (const Mat& m : outs) TRY(check_mat(m));
  for (const Mat& m : ins) TRY(check_mat(m));
  TRY(check_overlaps(outs, ins));
  if (!want_z && !want_w) return TPMLP_OK;
  TRY(check_device());
  RouteCombineBwdArgs a{};
  a.dy = dY;
  a.zs = Zs;
  a.dzs = want_z ? dZs : nullptr;
  a.dw = want_w ? dw : nullptr;
  a.w = w;
  a.row_of = row_of;
  a.src_of = src_of;
  a.T = T;
  a.rows = rows;
  a.ld_dy = ins[0].ld;
  a.ld_zs = ins[1].ld;
  a.ld_dzs = outs[0].ld;
  a.K = K;
  a.H = (int)H;
  return launched(launch_route_combine_bwd(a, dy_type, z_type, H % 4 == 0 && quads(outs[0]) && quads(ins[0]) && quads(ins[1]),
                                           past_caches(outs, ins), stream_of(stream)), "tpmlp_route_combine_bwd launch");
}

// ---------------------------------------------------------------------------
// Gradient norm and clipping
// ---------------------------------------------------------------------------
int64_t chunks_of(int64_t size) { return (size + CLIP_CHUNK - 1) / CLIP_CHUNK; }

// Workgroups of the launch that covers tensors [t0, t1).
int clip_blocks(const int64_t* sizes, int t0, int t1, int most = CLIP_BLOCKS) {
  int64_t c = 0;
  for (int t = t0; t < t1; ++t) c += chunks_of(sizes[t]);
  return (int)std::max<int64_t>(1, std::min<int64_t>(c, most));
}

// Calls f(first tensor, end, workgroups) for each launch.
template <class F>
tpmlp_status clip_launches(const int64_t* sizes, int n, F&& f) {
  for (int t0 = 0; t0 < n || t0 == 0; t0 += CLIP_TENSORS) {
    const int t1 = std::min(n, t0 + CLIP_TENSORS);
    TRY(f(t0, t1, clip_blocks(sizes, t0, t1)));
  }
  return TPMLP_OK;
}

bool sizes_ok(const int64_t* sizes, int n) {
  if (n < 0 || (n > 0 && !sizes)) return false;
  int64_t chunks = 0;
  for (int t = 0; t < n; ++t) {
    if (sizes[t] < 0 || sizes[t] > (int64_t(1) << 44)) return false;
    chunks += chunks_of(sizes[t]);
  }
  return chunks < INT32_MAX;
}

tpmlp_status check_grads(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* types, int n) {
  if (n < 0) return fail(TPMLP_ERR_SHAPE, "n is negative");
  if (n > 0 && (!grads || !sizes || !types)) return fail(TPMLP_ERR_NULL, "grads, sizes or types is NULL");
  if (!sizes_ok(sizes, n)) return fail(TPMLP_ERR_SHAPE, "a size is negative or the sizes are too large");
  for (int t = 0; t < n; ++t) {
    if (!type_ok(types[t])) return fail(TPMLP_ERR_SHAPE, "types[" + std::to_string(t) + "] is not a tpmlp_dtype");
    if (!sizes[t]) continue;
    const void* o = outs ? outs[t] : grads[t];
    if (!grads[t] || !o) return fail(TPMLP_ERR_NULL, (grads[t] ? "outs[" : "grads[") + std::to_string(t) + "] is NULL");
    const uintptr_t mask = size_of(types[t]) - 1, g = reinterpret_cast<uintptr_t>(grads[t]), u = reinterpret_cast<uintptr_t>(o);
    if ((g & mask) || (u & mask))
      return fail(TPMLP_ERR_ALIGN, ((g & mask) ? "grads[" : "outs[") + std::to_string(t) + "] is not aligned to its elements");
  }
  return TPMLP_OK;
}

// What is written must be disjoint from everything else, a tensor scaled in place from
// all but itself.  Written and read stretches in the order of their addresses: merged,
// none may begin before an earlier one ends if one of the two is written.  Tensors
// that were allocated one after another are in order already.
tpmlp_status check_grad_overlaps(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* types, int n) {
  struct Stretch {
    uintptr_t from, to;
    bool operator<(const Stretch& o) const { return from < o.from; }
  };
  std::vector<Stretch> written, read;
  written.reserve(n);
  if (outs) read.reserve(n);
  for (int t = 0; t < n; ++t) {
    if (!sizes[t]) continue;
    const uintptr_t bytes = uintptr_t(sizes[t]) * size_of(types[t]), g = reinterpret_cast<uintptr_t>(grads[t]);
    const uintptr_t o = outs ? reinterpret_cast<uintptr_t>(outs[t]) : g;
    written.push_back({o, o + bytes});
    if (o != g) read.push_back({g, g + bytes});
  }
  for (auto* v : {&written, &read})
    if (!std::is_sorted(v->begin(), v->end())) std::sort(v->begin(), v->end());
  uintptr_t written_to = 0, read_to = 0;
  size_t r = 0;
  for (const Stretch& w : written) {
    for (; r < read.size() && read[r].from <= w.from; ++r) {
      if (read[r].from < written_to) return fail(TPMLP_ERR_ALIAS, "an output overlaps another gradient");
      read_to = std::max(read_to, read[r].to);
    }
    if (w.from < read_to) return fail(TPMLP_ERR_ALIAS, "an output overlaps another gradient");
    if (w.from < written_to) return fail(TPMLP_ERR_ALIAS, "two outputs overlap");
    written_to = w.to;
  }
  if (r < read.size() && read[r].from < written_to) return fail(TPMLP_ERR_ALIAS, "an output overlaps another gradient");
  return TPMLP_OK;
}

// A buffer of the call beside the tensors (p NULL: absent).
struct Own {
  const void* p;
  size_t bytes;
  bool written;
  const char* name;
};

bool meet(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}

// The two are disjoint from each other if one is written, each from the outputs of a call
// that scales, and from the gradients if it is written.
tpmlp_status check_own(const void* const* grads, void* const* outs, bool scales, const int64_t* sizes, const int32_t* types,
                       int n, const Own (&own)[2]) {
  if ((own[0].written || own[1].written) && meet(own[0].p, own[0].bytes, own[1].p, own[1].bytes))
    return fail(TPMLP_ERR_ALIAS, std::string(own[0].name) + " overlaps " + own[1].name);
  for (int t = 0; t < n; ++t) {
    const size_t bytes = size_t(sizes[t]) * size_of(types[t]);
    const void* o = outs ? outs[t] : grads[t];
    for (const Own& b : own)
      if (bytes && ((b.written && meet(b.p, b.bytes, grads[t], bytes)) || (scales && meet(b.p, b.bytes, o, bytes))))
        return fail(TPMLP_ERR_ALIAS, std::string(b.name) + " overlaps gradient " + std::to_string(t) + " or its output");
  }
  return TPMLP_OK;
}

void fill_clip(ClipArgs& a, const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* types, int t0,
               int t1) {
  uint32_t chunk = 0;
  for (int t = t0; t < t1; ++t) {
    const int i = t - t0;
    a.in[i] = grads[t];
    a.out[i] = outs ? outs[t] : const_cast<void*>(grads[t]);
    a.size[i] = sizes[t] | (types[t] == TPMLP_BF16 ? int64_t(1) << 62 : 0);
    a.first[i] = chunk;
    chunk += (uint32_t)chunks_of(sizes[t]);
  }
  a.chunks = chunk;
  for (int i = t1 - t0; i < CLIP_TENSORS; ++i) a.first[i] = chunk;
  for (int k = 0; k < CLIP_TENSORS / 8; ++k) a.eighth[k] = a.first[8 * k];
}

// The partial sums of all launches into ws; *count of them.
tpmlp_status enqueue_sumsq(const void* const* grads, const int64_t* sizes, const int32_t* types, int n, double* ws,
                           int* count, hipStream_t s) {
  *count = 0;
  return clip_launches(sizes, n, [&](int t0, int t1, int blocks) {
    ClipArgs a{};
    fill_clip(a, grads, nullptr, sizes, types, t0, t1);
    a.part = ws + *count;
    *count += blocks;
    return launched(launch_clip_sumsq(a, blocks, s), "gradient norm launch");
  });
}

tpmlp_status enqueue_scale(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* types, int n,
                           const double* part, int n_part, float scale, float max_norm, float* norm, hipStream_t s) {
  return clip_launches(sizes, n, [&](int t0, int t1, int blocks) {
    ClipArgs a{};
    fill_clip(a, grads, outs, sizes, types, t0, t1);
    a.part = const_cast<double*>(part);
    a.n_part = n_part;
    a.scale = scale;
    a.max_norm = max_norm;
    a.norm = t0 == 0 ? norm : nullptr;
    blocks = clip_blocks(sizes, t0, t1, CLIP_SCALE_BLOCKS);
    return launched(launch_clip_scale(a, blocks, s), "gradient clipping launch");
  });
}

tpmlp_status check_ws(const int64_t* sizes, int n, void* ws, size_t ws_bytes) {
  if (!ws) return fail(TPMLP_ERR_NULL, "ws is NULL");
  if (reinterpret_cast<uintptr_t>(ws) & 15) return fail(TPMLP_ERR_ALIGN, "ws is not 16-byte aligned");
  if (ws_bytes < tpmlp_grad_workspace_bytes(sizes, n)) return fail(TPMLP_ERR_WORKSPACE, "ws_bytes below tpmlp_grad_workspace_bytes");
  return TPMLP_OK;
}

tpmlp_status check_factors(float scale, float max_norm, const float* norm) {
  if (!std::isfinite(scale)) return fail(TPMLP_ERR_SHAPE, "scale must be finite");
  if (!(max_norm > 0.0f)) return fail(TPMLP_ERR_SHAPE, "max_norm must be positive");
  if (reinterpret_cast<uintptr_t>(norm) & 3) return fail(TPMLP_ERR_ALIGN, "norm is not aligned to its elements");
  return TPMLP_OK;
}

}  // namespace
}  // namespace tpmlp

using namespace tpmlp;

extern "C" {

tpmlp_status tpmlp_edge_fwd(const tpmlp_edge* e, const void* y, int64_t ld_y, const void* r, int64_t ld_r, void* r_out,
                            int64_t ld_r_out, tpmlp_bf16* x, int64_t ld_x, void* stream) {
  return guarded([&] { return edge_fwd(e, y, ld_y, r, ld_r, r_out, ld_r_out, x, ld_x, nullptr, stream); });
}

tpmlp_status tpmlp_edge_fwd_fp8(const tpmlp_edge* e, const void* y, int64_t ld_y, const void* r, int64_t ld_r, void* r_out,
                                int64_t ld_r_out, uint8_t* codes, int64_t ld_codes, void* scales, int64_t ld_scales,
                                int scale_kind, void* stream) {
  return guarded([&] {
    const EdgeCodes c{codes, ld_codes, scales, ld_scales, scale_kind};
    return edge_fwd(e, y, ld_y, r, ld_r, r_out, ld_r_out, nullptr, 0, &c, stream);
  });
}

size_t tpmlp_edge_bwd_workspace_bytes(const tpmlp_edge* e) {
  if (!e || e->M < 1 || e->M > MAX_TOKENS || e->H < 8 || e->H > TPMLP_EDGE_MAX_H) return 0;
  if (e->gate && (e->gate_rows < 1 || gate_groups(*e) > MAX_GATES)) return 0;
  return plan_edge_bwd(e->M, (int)e->H, gate_rows_of(*e), has_layer(*e)).ws_bytes;
}

tpmlp_status tpmlp_edge_bwd(const tpmlp_edge* e, const void* y, int64_t ld_y, const void* r_out, int64_t ld_r_out,
                            const void* dr_out, int64_t ld_dr_out, const void* dx, int dx_type, int64_t ld_dx, void* dr,
                            int64_t ld_dr, tpmlp_bf16* dy, int64_t ld_dy, float* dw_post, float* db_post, float* dw_pre,
                            float* db_pre, float* dgate, void* ws, size_t ws_bytes, void* stream) {
  return guarded([&] {
    return edge_bwd(e, y, ld_y, r_out, ld_r_out, dr_out, ld_dr_out, dx, dx_type, ld_dx, dr, ld_dr, dy, ld_dy, dw_post,
                    db_post, dw_pre, db_pre, dgate, ws, ws_bytes, stream);
  });
}

int64_t tpmlp_route_rows(int64_t T, int K, int E, int align, int capacity) {
  if (!pairs_ok(T, K) || E < 1 || E > TPMLP_ROUTE_MAX_EXPERTS || align < 1 || capacity < 0 || capacity % align) return -1;
  const int64_t pairs = T * K;
  const int64_t rows = capacity ? int64_t(E) * capacity
                                : (pairs + std::min<int64_t>(E, pairs) * (align - 1)) / align * align;
  return rows <= MAX_ROWS ? rows : -1;
}

size_t tpmlp_route_workspace_bytes(int64_t T, int K, int E) {
  if (!pairs_ok(T, K) || E < 1 || E > TPMLP_ROUTE_MAX_EXPERTS) return 0;
  int64_t per = 0;
  const int64_t blocks = route_sort_blocks(T * K, &per);
  return blocks > 1 ? size_t(blocks) * E * 4 : 0;
}

tpmlp_status tpmlp_route_sort(const void* ids, int id_bits, int64_t T, int K, int E, int align, int capacity,
                              int32_t* counts, int32_t* offsets, int32_t* row_of, int32_t* src_of, void* ws,
                              size_t ws_bytes, void* stream) {
  return guarded(
      [&] { return route_sort(ids, id_bits, T, K, E, align, capacity, counts, offsets, row_of, src_of, ws, ws_bytes, stream); });
}

tpmlp_status tpmlp_route_dispatch(const tpmlp_bf16* X, int64_t ld_x, const int32_t* row_of, const int32_t* src_of,
                                  int64_t T, int K, int64_t H, int64_t rows, tpmlp_bf16* Xs, int64_t ld_xs, void* stream) {
  return guarded([&] { return route_dispatch(X, ld_x, row_of, src_of, T, K, H, rows, Xs, ld_xs, stream); });
}

tpmlp_status tpmlp_route_combine(const void* Zs, int z_type, int64_t ld_zs, const int32_t* row_of, const float* w,
                                 int64_t T, int K, int64_t H, int64_t rows, void* Y, int y_type, int64_t ld_y, void* stream) {
  return guarded([&] { return route_combine(Zs, z_type, ld_zs, row_of, w, T, K, H, rows, Y, y_type, ld_y, stream); });
}

tpmlp_status tpmlp_route_combine_bwd(const void* dY, int dy_type, int64_t ld_dy, const void* Zs, int z_type, int64_t ld_zs,
                                     const int32_t* row_of, const int32_t* src_of, const float* w, int64_t T, int K,
                                     int64_t H, int64_t rows, tpmlp_bf16* dZs, int64_t ld_dzs, float* dw, void* stream) {
  return guarded([&] {
    return route_combine_bwd(dY, dy_type, ld_dy, Zs, z_type, ld_zs, row_of, src_of, w, T, K, H, rows, dZs, ld_dzs, dw, stream);
  });
}

size_t tpmlp_grad_workspace_bytes(const int64_t* sizes, int n) {
  if (!sizes_ok(sizes, n)) return 0;
  size_t blocks = 0;
  for (int t0 = 0; t0 < n || t0 == 0; t0 += CLIP_TENSORS) blocks += clip_blocks(sizes, t0, std::min(n, t0 + CLIP_TENSORS));
  return blocks * sizeof(double) + sizeof(double);
}

tpmlp_status tpmlp_grad_sumsq(const void* const* grads, const int64_t* sizes, const int32_t* types, int n, double* sumsq,
                              void* ws, size_t ws_bytes, void* stream) {
  return guarded([&]() -> tpmlp_status {
    TRY(check_grads(grads, nullptr, sizes, types, n));
    if (!sumsq) return fail(TPMLP_ERR_NULL, "sumsq is NULL");
    if (reinterpret_cast<uintptr_t>(sumsq) & 7) return fail(TPMLP_ERR_ALIGN, "sumsq is not aligned to its elements");
    TRY(check_ws(sizes, n, ws, ws_bytes));
    TRY(check_own(grads, nullptr, false, sizes, types, n,
                  {{sumsq, sizeof(double), true, "sumsq"}, {ws, tpmlp_grad_workspace_bytes(sizes, n), true, "ws"}}));
    TRY(check_device());
    hipStream_t s = stream_of(stream);
    int count = 0;
    TRY(enqueue_sumsq(grads, sizes, types, n, static_cast<double*>(ws), &count, s));
    return launched(launch_clip_total(static_cast<double*>(ws), count, sumsq, s), "gradient norm launch");
  });
}

tpmlp_status tpmlp_grad_clip(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* types, int n,
                             const double* sumsq, float scale, float max_norm, float* norm, void* stream) {
  return guarded([&]() -> tpmlp_status {
    TRY(check_grads(grads, outs, sizes, types, n));
    TRY(check_grad_overlaps(grads, outs, sizes, types, n));
    if (!sumsq) return fail(TPMLP_ERR_NULL, "sumsq is NULL");
    if (reinterpret_cast<uintptr_t>(sumsq) & 7) return fail(TPMLP_ERR_ALIGN, "sumsq is not aligned to its elements");
    TRY(check_factors(scale, max_norm, norm));
    TRY(check_own(grads, outs, true, sizes, types, n,
                  {{norm, sizeof(float), true, "norm"}, {sumsq, sizeof(double), false, "sumsq"}}));
    TRY(check_device());
    return enqueue_scale(grads, outs, sizes, types, n, sumsq, 1, scale, max_norm, norm, stream_of(stream));
  });
}

tpmlp_status tpmlp_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* types,
                                  int n, float scale, float max_norm, float* norm, void* ws, size_t ws_bytes, void* stream) {
  return guarded([&]() -> tpmlp_status {
    TRY(check_grads(grads, outs, sizes, types, n));
    TRY(check_grad_overlaps(grads, outs, sizes, types, n));
    TRY(check_factors(scale, max_norm, norm));
    TRY(check_ws(sizes, n, ws, ws_bytes));
    TRY(check_own(grads, outs, true, sizes, types, n,
                  {{norm, sizeof(float), true, "norm"}, {ws, tpmlp_grad_workspace_bytes(sizes, n), true, "ws"}}));
    TRY(check_device());
    hipStream_t s = stream_of(stream);
    double* part = static_cast<double*>(ws);
    int count = 0;
    TRY(enqueue_sumsq(grads, sizes, types, n, part, &count, s));
    if (count > CLIP_BLOCKS) {  // several launches' partials: added once, not by every workgroup
      TRY(launched(launch_clip_total(part, count, part + count, s), "gradient norm launch"));
      part += count;
      count = 1;
    }
    return enqueue_scale(grads, outs, sizes, types, n, part, count, scale, max_norm, norm, s);
  });
}

}  // extern "C"
