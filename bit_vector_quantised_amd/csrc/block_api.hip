// C ABI of the norm, the choice of experts and rows in 8 bits: argument checks and the launches.  Every check
// runs on the host before any HIP call.
#include "api_checks.h"
#include "dense.h"

using namespace mvq;

namespace {

bool norm_dims_ok(int n_rows, int n_cols, float eps) {
  return n_rows >= 0 && n_rows <= MAX_ROWS && n_cols >= 1 && n_cols <= MAX_DIM && eps > 0.f && eps <= 3.4e38f;
}

// Rows in 8 bits: columns up to those of the widest dense product, and as many rows as 2^34 columns in all.
bool rows8_dims_ok(int n_rows, int n_cols) {
  return n_rows >= 0 && n_rows <= MAX_ROWS && n_cols >= 1 && n_cols <= 2 * MAX_DIM &&
         (size_t)n_rows * rows8_pitch(n_cols) <= (size_t)1 << 34;
}
bool rows8_ok(const moe_vq_rows8* r) { return r && r->q && r->e && !off16(r->q); }

bool choice_ok(const moe_vq_choice* c) {
  if (!c || c->n_experts < 1 || c->n_experts > MAX_E || c->top_k < 1 || c->top_k > MAX_K) return false;
  if (c->score != MOE_VQ_SCORE_SOFTMAX && c->score != MOE_VQ_SCORE_SIGMOID) return false;
  if (c->n_groups < 1 || c->n_groups > 64 || c->n_experts % c->n_groups) return false;
  if (c->top_groups < 1 || c->top_groups > c->n_groups || c->group_best < 1 || c->group_best > 2) return false;
  if (c->top_k > c->top_groups * (c->n_experts / c->n_groups)) return false;
  return (c->renorm == 0 || c->renorm == 1) && c->scale >= -3.4e38f && c->scale <= 3.4e38f && !off4(c->bias);
}

ChooseArgs choose_args(const moe_vq_choice* c, const float* logits, int n_tokens, const int32_t* ids, const float* w) {
  ChooseArgs a{};
  a.logits = logits;
  a.bias = c->bias;
  a.ids = const_cast<int32_t*>(ids);
  a.w = const_cast<float*>(w);
  a.T = n_tokens; a.E = c->n_experts; a.k = c->top_k;
  a.groups = c->n_groups; a.top_groups = c->top_groups; a.best = c->group_best;
  a.sigmoid = c->score == MOE_VQ_SCORE_SIGMOID;
  a.renorm = c->renorm != 0;
  a.scale = c->scale;
  return a;
}

}  // namespace

extern "C" {

int moe_vq_norm_forward(const void* x, int dtype, const void* residual, void* s, int s_dtype, int n_rows, int n_cols,
                        const float* gain, float eps, void* y, int y_dtype, const moe_vq_rows8* y8, void* stream) {
  if (!norm_dims_ok(n_rows, n_cols, eps) || !dtype_ok(dtype) || !dtype_ok(s_dtype) || !dtype_ok(y_dtype)) return MOE_VQ_EINVAL;
  if (n_rows == 0 || (!s && !y && !y8)) return MOE_VQ_OK;
  if (!x || !gain || off16(x) || off16(residual) || off16(s) || off16(y) || off4(gain)) return MOE_VQ_EINVAL;
  if (y8 && (!rows8_ok(y8) || !rows8_dims_ok(n_rows, n_cols))) return MOE_VQ_EINVAL;
  const size_t cells = (size_t)n_rows * n_cols;
  const Span x_s{x, cells * size_of(dtype)}, r_s{residual, cells * size_of(s_dtype)}, s_s{s, r_s.n}, y_s{y, cells * size_of(y_dtype)};
  const Span g_s{gain, (size_t)n_cols * 4}, q_s = bytes8(y8, n_rows, n_cols), e_s = scales8(y8, n_rows, n_cols);
  // (a row is read whole before any of its outputs is written: s may be residual, and s or y be x, of one type)
  const bool s_x = s && s == x && s_dtype == dtype, s_r = s && s == residual, y_x = y && y == x && y_dtype == dtype;
  if (clash({s_s, y_s, q_s, e_s}, {g_s}) || clash({q_s, e_s}, {x_s, r_s}) || (!s_x && overlap(s_s, x_s)) ||
      (!s_r && overlap(s_s, r_s)) || (!y_x && overlap(y_s, x_s)) || overlap(y_s, r_s))
    return MOE_VQ_EINVAL;
  NormArgs a{};
  a.x = x;
  a.res = residual;
  a.s = s;
  a.gain = gain;
  a.y = y;
  if (y8) { a.q = y8->q; a.e = y8->e; }
  a.eps = eps;
  a.M = n_rows; a.C = n_cols;
  return hip_status(launch_norm(a, dtype, s_dtype, y_dtype, static_cast<hipStream_t>(stream)));
}

size_t moe_vq_norm_bytes(int n_rows, int n_cols) {
  if (!norm_dims_ok(n_rows, n_cols, 1.f)) return 0;
  return align256((size_t)(n_rows ? norm_back_blocks(n_rows, n_cols) : 1) * n_cols * sizeof(float));
}

int moe_vq_norm_backward(const void* s, int s_dtype, int n_rows, int n_cols, const float* gain, float eps, const void* dy,
                         const void* dy2, int dy_dtype, const void* ds, void* dx, int dx_dtype, float* dgain, void* ws,
                         size_t ws_bytes, void* stream) {
  if (!norm_dims_ok(n_rows, n_cols, eps) || !dtype_ok(s_dtype) || !dtype_ok(dy_dtype) || !dtype_ok(dx_dtype)) return MOE_VQ_EINVAL;
  if (!dgain && (!dx || n_rows == 0)) return MOE_VQ_OK;
  if (off16(s) || off16(dy) || off16(dy2) || off16(ds) || off16(dx) || off4(gain) || off4(dgain)) return MOE_VQ_EINVAL;
  if (n_rows > 0 && (!s || !gain || !dy)) return MOE_VQ_EINVAL;
  if (dgain && (!ws || ((uintptr_t)ws & 255))) return MOE_VQ_EINVAL;
  const size_t need = (size_t)norm_back_blocks(n_rows, n_cols) * n_cols * sizeof(float);
  if (dgain && ws_bytes < need) return MOE_VQ_ENOSPACE;
  const size_t cells = (size_t)n_rows * n_cols;
  const Span s_s{s, cells * size_of(s_dtype)}, d_s{dy, cells * size_of(dy_dtype)}, d2_s{dy2, d_s.n}, ds_s{ds, cells * size_of(dx_dtype)};
  const Span dx_s{dx, ds_s.n}, g_s{gain, (size_t)n_cols * 4}, dg_s{dgain, g_s.n}, ws_s{dgain ? ws : nullptr, need};
  if (clash({dx_s, dg_s, ws_s}, {s_s, d_s, d2_s, g_s}) || clash({dg_s, ws_s}, {ds_s}) || (dx != ds && overlap(dx_s, ds_s)))
    return MOE_VQ_EINVAL;
  NormBackArgs a{};
  a.s = s;
  a.dy = dy;
  a.dy2 = dy2;
  a.ds = ds;
  a.dx = dx;
  a.gain = gain;
  a.dgain = dgain;
  a.part = static_cast<float*>(ws);
  a.eps = eps;
  a.M = n_rows; a.C = n_cols;
  return hip_status(launch_norm_back(a, dy_dtype, s_dtype, dx_dtype, static_cast<hipStream_t>(stream)));
}

int moe_vq_choose(const moe_vq_choice* c, const float* logits, int n_tokens, int32_t* ids, float* w, void* stream) {
  if (!choice_ok(c) || n_tokens < 0 || n_tokens > MAX_T) return MOE_VQ_EINVAL;
  if (n_tokens == 0) return MOE_VQ_OK;
  if (!logits || !ids || !w || off4(logits) || off4(ids) || off4(w)) return MOE_VQ_EINVAL;
  const size_t pairs = (size_t)n_tokens * c->top_k * 4;
  if (clash({{ids, pairs}, {w, pairs}}, {{logits, (size_t)n_tokens * c->n_experts * 4}, {c->bias, (size_t)c->n_experts * 4}}))
    return MOE_VQ_EINVAL;
  return hip_status(launch_choose(choose_args(c, logits, n_tokens, ids, w), static_cast<hipStream_t>(stream)));
}

int moe_vq_choose_backward(const moe_vq_choice* c, const float* logits, int n_tokens, const int32_t* ids, const float* dw,
                           float* dlogits, void* stream) {
  if (!choice_ok(c) || n_tokens < 0 || n_tokens > MAX_T) return MOE_VQ_EINVAL;
  if (n_tokens == 0) return MOE_VQ_OK;
  if (!logits || !ids || !dw || !dlogits || off4(logits) || off4(ids) || off4(dw) || off4(dlogits)) return MOE_VQ_EINVAL;
  const size_t pairs = (size_t)n_tokens * c->top_k * 4, all = (size_t)n_tokens * c->n_experts * 4;
  // (a token's logits are read before its gradients are written: dlogits may be logits)
  if (clash({{dlogits, all}}, {{ids, pairs}, {dw, pairs}, {c->bias, (size_t)c->n_experts * 4}}) ||
      (dlogits != logits && overlap({dlogits, all}, {logits, all})))
    return MOE_VQ_EINVAL;
  ChooseArgs a = choose_args(c, logits, n_tokens, ids, dw);
  a.dlogits = dlogits;
  return hip_status(launch_choose_back(a, static_cast<hipStream_t>(stream)));
}

size_t moe_vq_rows8_pitch(int n_cols) { return n_cols < 1 || n_cols > 2 * MAX_DIM ? 0 : rows8_pitch(n_cols); }

int moe_vq_rows8_pack(const void* x, int dtype, int n_rows, int n_cols, const int32_t* group_start, int n_groups,
                      const moe_vq_rows8* r, void* stream) {
  if (!rows8_dims_ok(n_rows, n_cols) || !dtype_ok(dtype)) return MOE_VQ_EINVAL;
  if (group_start && (n_groups < 1 || n_groups > MAX_E || off4(group_start))) return MOE_VQ_EINVAL;
  if (n_rows == 0) return MOE_VQ_OK;
  if (!x || off16(x) || !rows8_ok(r)) return MOE_VQ_EINVAL;
  const Span q = bytes8(r, n_rows, n_cols), e = scales8(r, n_rows, n_cols);
  if (clash({q, e}, {{x, (size_t)n_rows * n_cols * size_of(dtype)}, {group_start, ((size_t)n_groups + 1) * 4}})) return MOE_VQ_EINVAL;
  Rows8Args a{};
  a.x = x;
  a.q = r->q;
  a.e = r->e;
  a.start = group_start;
  a.M = n_rows; a.C = n_cols; a.G = n_groups;
  return hip_status(launch_rows8_pack(a, dtype, static_cast<hipStream_t>(stream)));
}

int moe_vq_rows8_unpack(const moe_vq_rows8* r, int n_rows, int n_cols, const int32_t* group_start, int n_groups, void* x,
                        int dtype, void* stream) {
  if (!rows8_dims_ok(n_rows, n_cols) || !dtype_ok(dtype)) return MOE_VQ_EINVAL;
  if (group_start && (n_groups < 1 || n_groups > MAX_E || off4(group_start))) return MOE_VQ_EINVAL;
  if (n_rows == 0) return MOE_VQ_OK;
  if (!x || off16(x) || !rows8_ok(r)) return MOE_VQ_EINVAL;
  if (clash({{x, (size_t)n_rows * n_cols * size_of(dtype)}},
            {bytes8(r, n_rows, n_cols), scales8(r, n_rows, n_cols), {group_start, ((size_t)n_groups + 1) * 4}}))
    return MOE_VQ_EINVAL;
  Rows8Args a{};
  a.q = r->q;
  a.e = r->e;
  a.y = x;
  a.start = group_start;
  a.M = n_rows; a.C = n_cols; a.G = n_groups;
  a.pitch = n_cols;
  return hip_status(launch_rows8_unpack(a, dtype, static_cast<hipStream_t>(stream)));
}

int moe_vq_gather_rows8(const moe_vq_rows8* r, int n_tokens, int top_k, int n_cols, const int32_t* pair_row, void* xs,
                        int dtype, void* stream) {
  if (n_tokens < 0 || n_tokens > MAX_T || top_k < 1 || top_k > MAX_K || !rows8_dims_ok(n_tokens, n_cols) || !dtype_ok(dtype))
    return MOE_VQ_EINVAL;
  if (n_tokens == 0) return MOE_VQ_OK;
  if (!rows8_ok(r) || !pair_row || !xs || off16(xs) || off4(pair_row)) return MOE_VQ_EINVAL;
  if (clash({{xs, (size_t)n_tokens * top_k * n_cols * size_of(dtype)}},
            {bytes8(r, n_tokens, n_cols), scales8(r, n_tokens, n_cols), {pair_row, (size_t)n_tokens * top_k * 4}}))
    return MOE_VQ_EINVAL;
  Rows8Args a{};
  a.q = r->q;
  a.e = r->e;
  a.y = xs;
  a.pair_row = pair_row;
  a.M = n_tokens; a.C = n_cols; a.k = top_k;
  a.pitch = n_cols;
  return hip_status(launch_rows8_unpack(a, dtype, static_cast<hipStream_t>(stream)));
}

int moe_vq_act_backward8(const moe_vq_rows8* z8, int act, float swiglu_limit, int n_tokens, int top_k, int n_out,
                         const int32_t* pair_row, const float* w, const void* dy, int dy_dtype, void* dz, void* y, int dtype,
                         float* dw, void* stream) {
  if (n_tokens < 0 || n_tokens > MAX_T || top_k < 1 || top_k > MAX_K || n_out < 1 || n_out > MAX_DIM) return MOE_VQ_EINVAL;
  if (act < MOE_VQ_ACT_NONE || act > MOE_VQ_ACT_SWIGLU || !dtype_ok(dtype) || !dtype_ok(dy_dtype)) return MOE_VQ_EINVAL;
  if (act == MOE_VQ_ACT_SWIGLU && !(swiglu_limit >= 0.f && swiglu_limit <= 3.4e38f)) return MOE_VQ_EINVAL;
  const int P = n_tokens * top_k, R = act == MOE_VQ_ACT_SWIGLU ? 2 * n_out : n_out;
  if (P == 0 || (!dz && !y && !dw)) return MOE_VQ_OK;
  if (!rows8_ok(z8) || !pair_row || !dy || off16(dy) || off16(dz) || off16(y)) return MOE_VQ_EINVAL;
  if (off4(pair_row) || off4(w) || off4(dw)) return MOE_VQ_EINVAL;
  const size_t pairs = (size_t)P * 4, size = size_of(dtype);
  const Span dy_s{dy, (size_t)P * n_out * size_of(dy_dtype)}, y_s{y, (size_t)P * n_out * size}, dz_s{dz, (size_t)P * R * size};
  const Span dw_s{dw, pairs}, w_s{w, pairs};
  // (a pair's weight is read before its gradient is written: dw may be w)
  if (clash({dz_s, y_s, dw_s}, {dy_s, {pair_row, pairs}, bytes8(z8, P, R), scales8(z8, P, R)}) || clash({dz_s, y_s}, {w_s}) ||
      (dw != w && overlap(dw_s, w_s)))
    return MOE_VQ_EINVAL;
  ActBackArgs a{};
  a.q = z8->q;
  a.e = z8->e;
  a.pair_row = pair_row;
  a.w = w;
  a.dy = dy;
  a.dz = dz;
  a.y = y;
  a.dw = dw;
  a.P = P; a.N = n_out; a.R = R; a.act = act;
  a.lim = swiglu_limit;
  return hip_status(launch_act_back(a, dtype, dy_dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
