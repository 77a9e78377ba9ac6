// C ABI of the row operators and the dense product: argument checks, workspace layout and
// the launches.  Every check runs on the host before any HIP call.
#include "api_checks.h"
#include "dense.h"

using namespace mvq;

namespace {

bool rows_dims_ok(int n_tokens, int top_k, int n_cols) {
  return n_tokens >= 0 && n_tokens <= MAX_T && top_k >= 1 && top_k <= MAX_K && n_cols >= 1 && n_cols <= MAX_COLS;
}

bool linear_dims_ok(const moe_vq_linear* L) {
  if (!L) return false;
  if (L->n_in < 1 || L->n_in > MAX_DIM || L->n_out < 1 || L->n_out > MAX_DIM) return false;
  if (L->n_groups < 1 || L->n_groups > MAX_E) return false;
  if (L->act < MOE_VQ_ACT_NONE || L->act > MOE_VQ_ACT_SWIGLU || !dtype_ok(L->dtype)) return false;
  if (L->act == MOE_VQ_ACT_SWIGLU && !(L->swiglu_limit >= 0.f && L->swiglu_limit <= 3.4e38f)) return false;
  return true;
}

// What both directions check before their own pointers.
int check_linear(const moe_vq_linear* L, int n_rows, const int32_t* group_start) {
  if (!linear_dims_ok(L)) return MOE_VQ_EINVAL;
  if (n_rows < 0 || n_rows > MAX_ROWS) return MOE_VQ_EINVAL;
  if (!L->w || off16(L->w) || off4(L->bias)) return MOE_VQ_EINVAL;
  if (L->n_groups > 1 && !group_start) return MOE_VQ_EINVAL;
  if (off4(group_start)) return MOE_VQ_EINVAL;
  return MOE_VQ_OK;
}

int check_linear_ws(const LinearPlan& p, const void* ws, size_t ws_bytes) {
  if (!ws || ((uintptr_t)ws & 255)) return MOE_VQ_EINVAL;
  return ws_bytes < p.total ? MOE_VQ_ENOSPACE : MOE_VQ_OK;
}

// What a product reads beside its rows (bias: also the size of dbias).
struct LinearSpans {
  Span w, bias, table;
  LinearSpans(const moe_vq_linear* L, const LinearPlan& p, const int32_t* group_start)
      : w{L->w, (size_t)p.G * p.R * p.K * p.size}, bias{L->bias, (size_t)p.G * p.R * 4}, table{group_start, ((size_t)p.G + 1) * 4} {}
};

// Either gradient call: x and z as they are, or (kept8) in 8 bits.
int backward(const moe_vq_linear* L, const void* x, const moe_vq_rows8* x8, int n_rows, const int32_t* group_start,
             const void* z, const moe_vq_rows8* z8, const void* dy, int dy_dtype, void* dx, void* dw, float* dbias, void* ws,
             size_t ws_bytes, void* stream, bool kept8) {
  int st = check_linear(L, n_rows, group_start);
  if (st) return st;
  if (!dtype_ok(dy_dtype)) return MOE_VQ_EINVAL;
  if (!dx && !dw && !dbias) return MOE_VQ_OK;
  if (off16(x) || off16(z) || off16(dy) || off16(dx) || off16(dw) || off4(dbias)) return MOE_VQ_EINVAL;
  for (const moe_vq_rows8* r : {x8, z8})  // (the buffers of no rows may be null)
    if (r && ((n_rows > 0 && (!r->q || !r->e)) || off16(r->q))) return MOE_VQ_EINVAL;
  if (n_rows > 0 && (!dy || (dw && !x && !x8) || (L->act != MOE_VQ_ACT_NONE && !z && !z8))) return MOE_VQ_EINVAL;
  const LinearPlan p = linear_plan(L, n_rows, true, kept8);
  if ((st = check_linear_ws(p, ws, ws_bytes))) return st;
  const LinearSpans in(L, p, group_start);
  const bool act = L->act != MOE_VQ_ACT_NONE;
  const Span dx_s{dx, (size_t)p.M * p.K * p.size}, dw_s{dw, in.w.n}, db_s{dbias, in.bias.n}, ws_s{ws, p.total};
  const Span dy_s{dy, (size_t)p.M * p.N * size_of(dy_dtype)}, z_s{act ? z : nullptr, (size_t)p.M * p.R * p.size};
  const Span x_s{dw ? x : nullptr, dx_s.n}, w_s{dx ? L->w : nullptr, in.w.n};  // (each read for one product only)
  // In order: dz and its column sums' parts from dy and z; then dx from dz and w, dw from dz and x and the sum of the bias
  // parts, which may run side by side in one launch.  So dx and dw may lie over z, and over dy where dz is another
  // tensor (without an activation both products read dy), but neither over what the other reads or writes.  dw may
  // lie over w all the same: launch_linear_backward then makes dx in a launch of its own before dw.
  if (clash({dx_s, dw_s, db_s, ws_s}, {x_s, in.table}) || clash({db_s, ws_s}, {dy_s, z_s, w_s}) || overlap(dx_s, w_s) ||
      (!act && (overlap(dx_s, dy_s) || overlap(dw_s, dy_s))))
    return MOE_VQ_EINVAL;
  const moe_vq_rows8 *xr = dw ? x8 : nullptr, *zr = act ? z8 : nullptr;
  if (clash({dx_s, dw_s, db_s, ws_s}, {bytes8(xr, p.M, p.K), scales8(xr, p.M, p.K), bytes8(zr, p.M, p.R), scales8(zr, p.M, p.R)}))
    return MOE_VQ_EINVAL;
  LinearCall c{};
  c.L = L;
  c.x = x;
  c.group_start = group_start;
  c.y_dtype = dy_dtype;
  c.z = const_cast<void*>(z);
  if (x8) c.x8 = *x8;
  if (z8) c.z8 = *z8;
  c.dy = dy;
  c.dx = dx;
  c.dw = dw;
  c.dbias = dbias;
  c.ws = ws;
  return hip_status(launch_linear_backward(p, c, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t moe_vq_sort_bytes(int n_tokens, int top_k, int n_experts) {
  if (!rows_dims_ok(n_tokens, top_k, 1) || n_experts < 1 || n_experts > MAX_E) return 0;
  // (the workgroup count falls where the workgroups grow: what the largest smaller call needs)
  const int P = n_tokens * top_k;
  const int nb = P > 131072 && sort_blocks(P) < sort_blocks(131072) ? sort_blocks(131072) : sort_blocks(P);
  return align256((size_t)(nb < 1 ? 1 : nb) * n_experts * sizeof(int32_t));
}

int moe_vq_sort_pairs(const int32_t* topk_ids, int n_tokens, int top_k, int n_experts, int32_t* expert_start,
                      int32_t* pair_row, int32_t* row_pair, void* ws, size_t ws_bytes, void* stream) {
  if (!rows_dims_ok(n_tokens, top_k, 1) || n_experts < 1 || n_experts > MAX_E) return MOE_VQ_EINVAL;
  if (!expert_start || off4(expert_start)) return MOE_VQ_EINVAL;
  if (n_tokens > 0 && (!topk_ids || !pair_row || !row_pair)) return MOE_VQ_EINVAL;
  if (off4(topk_ids) || off4(pair_row) || off4(row_pair)) return MOE_VQ_EINVAL;
  if (!ws || ((uintptr_t)ws & 255)) return MOE_VQ_EINVAL;
  SortArgs a{};
  a.ids = topk_ids;
  a.P = n_tokens * top_k;
  a.E = n_experts;
  a.start = expert_start;
  a.pair_row = pair_row;
  a.row_pair = row_pair;
  a.hist = static_cast<int32_t*>(ws);
  const size_t hist = (size_t)sort_blocks(a.P) * n_experts * sizeof(int32_t), pairs = (size_t)a.P * 4;
  if (ws_bytes < hist) return MOE_VQ_ENOSPACE;
  if (clash({{expert_start, ((size_t)n_experts + 1) * 4}, {pair_row, pairs}, {row_pair, pairs}, {ws, hist}}, {{topk_ids, pairs}}))
    return MOE_VQ_EINVAL;
  return hip_status(launch_sort(a, static_cast<hipStream_t>(stream)));
}

int moe_vq_gather_rows(const void* x, int dtype, int n_tokens, int top_k, int n_cols, const int32_t* pair_row,
                       void* xs, void* stream) {
  if (!rows_dims_ok(n_tokens, top_k, n_cols) || !dtype_ok(dtype)) return MOE_VQ_EINVAL;
  if (n_tokens == 0) return MOE_VQ_OK;
  if (!x || !pair_row || !xs || off16(x) || off16(xs) || off4(pair_row)) return MOE_VQ_EINVAL;
  const size_t bytes = (size_t)n_tokens * n_cols * size_of(dtype);
  if (clash({{xs, bytes * top_k}}, {{x, bytes}, {pair_row, (size_t)n_tokens * top_k * 4}})) return MOE_VQ_EINVAL;
  RowsArgs a{};
  a.pair_row = pair_row;
  a.x = x;
  a.y = xs;
  a.T = n_tokens; a.k = top_k; a.C = n_cols;
  return hip_status(launch_gather(a, dtype, static_cast<hipStream_t>(stream)));
}

int moe_vq_combine_rows(const void* rows, int dtype, int n_tokens, int top_k, int n_cols, const int32_t* pair_row,
                        const float* w, const void* residual, void* y, int y_dtype, void* stream) {
  if (!rows_dims_ok(n_tokens, top_k, n_cols) || !dtype_ok(dtype) || !dtype_ok(y_dtype)) return MOE_VQ_EINVAL;
  if (n_tokens == 0) return MOE_VQ_OK;
  if (!rows || !pair_row || !y || off16(rows) || off16(y) || off16(residual)) return MOE_VQ_EINVAL;
  if (off4(pair_row) || off4(w)) return MOE_VQ_EINVAL;
  const size_t cells = (size_t)n_tokens * n_cols, bytes = cells * size_of(y_dtype), pairs = (size_t)n_tokens * top_k * 4;
  if (clash({{y, bytes}}, {{rows, cells * top_k * size_of(dtype)}, {residual == y ? nullptr : residual, bytes},
                           {pair_row, pairs}, {w, pairs}}))
    return MOE_VQ_EINVAL;
  RowsArgs a{};
  a.pair_row = pair_row;
  a.pair_w = w;
  a.x = rows;
  a.add = residual;
  a.y = y;
  a.T = n_tokens; a.k = top_k; a.C = n_cols;
  return hip_status(launch_combine_rows(a, dtype, y_dtype, static_cast<hipStream_t>(stream)));
}

int moe_vq_combine_rows_backward(const void* dy, int dy_dtype, int n_tokens, int top_k, int n_cols,
                                 const int32_t* pair_row, const float* w, const void* rows, int dtype, void* drows,
                                 float* dw, void* stream) {
  if (!rows_dims_ok(n_tokens, top_k, n_cols) || !dtype_ok(dtype) || !dtype_ok(dy_dtype)) return MOE_VQ_EINVAL;
  if (n_tokens == 0 || (!drows && !dw)) return MOE_VQ_OK;
  if (!dy || !pair_row || (dw && !rows) || off16(dy) || off16(rows) || off16(drows)) return MOE_VQ_EINVAL;
  if (off4(pair_row) || off4(w) || off4(dw)) return MOE_VQ_EINVAL;
  const size_t cells = (size_t)n_tokens * n_cols, bytes = cells * top_k * size_of(dtype), pairs = (size_t)n_tokens * top_k * 4;
  // (a workgroup reads the weights of its own pairs before it writes their gradients: dw may be w itself)
  if (clash({{drows, bytes}, {dw, pairs}}, {{rows, bytes}, {dy, cells * size_of(dy_dtype)}, {pair_row, pairs}}) ||
      overlap({drows, bytes}, {w, pairs}) || (dw != w && overlap({dw, pairs}, {w, pairs})))
    return MOE_VQ_EINVAL;
  RowsArgs a{};
  a.pair_row = pair_row;
  a.pair_w = w;
  a.x = rows;
  a.add = dy;
  a.y = drows;
  a.dw = dw;
  a.T = n_tokens; a.k = top_k; a.C = n_cols;
  return hip_status(launch_combine_rows_backward(a, dtype, dy_dtype, static_cast<hipStream_t>(stream)));
}

size_t moe_vq_linear_bytes(const moe_vq_linear* L, int n_rows, int backward) {
  if (!linear_dims_ok(L) || n_rows < 0 || n_rows > MAX_ROWS || (backward != 0 && backward != 1)) return 0;
  return linear_max_bytes(L, n_rows, backward != 0);
}

int moe_vq_linear_forward(const moe_vq_linear* L, const void* x, int n_rows, const int32_t* group_start,
                          const void* residual, void* y, int y_dtype, void* z, void* ws, size_t ws_bytes,
                          void* stream) {
  int st = check_linear(L, n_rows, group_start);
  if (st) return st;
  if (!dtype_ok(y_dtype)) return MOE_VQ_EINVAL;
  if (n_rows == 0) return MOE_VQ_OK;
  if (!x || !y || off16(x) || off16(y) || off16(residual) || off16(z)) return MOE_VQ_EINVAL;
  const LinearPlan p = linear_plan(L, n_rows, false);
  if ((st = check_linear_ws(p, ws, ws_bytes))) return st;
  const size_t xb = (size_t)p.M * p.K * p.size, zb = (size_t)p.M * p.R * p.size, yb = (size_t)p.M * p.N * size_of(y_dtype);
  const LinearSpans in(L, p, group_start);
  if (clash({{y, yb}, {z, zb}, {ws, p.total}}, {{x, xb}, in.w, in.bias, in.table}) ||
      clash({{z, zb}, {ws, p.total}}, {{residual, yb}}) || (y != residual && overlap({y, yb}, {residual, yb})))
    return MOE_VQ_EINVAL;
  LinearCall c{};
  c.L = L;
  c.x = x;
  c.group_start = group_start;
  c.residual = residual;
  c.y = y;
  c.y_dtype = y_dtype;
  c.z = z;
  c.ws = ws;
  return hip_status(launch_linear_forward(p, c, static_cast<hipStream_t>(stream)));
}

int moe_vq_linear_backward(const moe_vq_linear* L, const void* x, int n_rows, const int32_t* group_start,
                           const void* z, const void* dy, int dy_dtype, void* dx, void* dw, float* dbias, void* ws,
                           size_t ws_bytes, void* stream) {
  return backward(L, x, nullptr, n_rows, group_start, z, nullptr, dy, dy_dtype, dx, dw, dbias, ws, ws_bytes, stream, false);
}

size_t moe_vq_linear_bytes8(const moe_vq_linear* L, int n_rows) {
  if (!linear_dims_ok(L) || n_rows < 0 || n_rows > MAX_ROWS) return 0;
  return linear_max_bytes(L, n_rows, true, true);
}

int moe_vq_linear_backward8(const moe_vq_linear* L, const void* x, const moe_vq_rows8* x8, int n_rows,
                            const int32_t* group_start, const void* z, const moe_vq_rows8* z8, const void* dy,
                            int dy_dtype, void* dx, void* dw, float* dbias, void* ws, size_t ws_bytes, void* stream) {
  if ((x && x8) || (z && z8)) return MOE_VQ_EINVAL;
  return backward(L, x, x8, n_rows, group_start, z, z8, dy, dy_dtype, dx, dw, dbias, ws, ws_bytes, stream, true);
}

}  // extern "C"
