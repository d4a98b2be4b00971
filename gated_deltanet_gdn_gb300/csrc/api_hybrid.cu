// C ABI of the operators around the rule in a hybrid stack (include/gdn.h): argument
// validation and dispatch of the paged cache's append and attention and of the block norms.
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/gdn.h"
#include "kernels.h"

namespace gdn {
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int launch_status(cudaError_t e) {
  return e == cudaSuccess ? GDN_OK : e == cudaErrorNotSupported ? GDN_ERR_UNSUPPORTED : GDN_ERR_CUDA;
}
int esize(int dtype) { return dtype == GDN_BF16 ? 2 : 4; }

// A stride the kernels' 16-byte accesses can use.
bool stride_ok(long long s, int es) { return s >= 0 && (s * es) % 16 == 0; }

int check_paged(const gdn_paged_dims* d) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->N < 0 || d->B < 0 || d->Hq < 1 || d->Hk < 1 || d->Hq % d->Hk != 0) return GDN_ERR_INVALID_ARG;
  if (d->page_size < 1 || d->num_pages < 0 || d->max_pages < 0) return GDN_ERR_INVALID_ARG;
  if (d->flags & ~GDN_FLAG_ROPE_PAIRS) return GDN_ERR_INVALID_ARG;
  if (d->dtype != GDN_F32 && d->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (d->D != 64 && d->D != 128) return GDN_ERR_UNSUPPORTED;
  if (d->page_size % 16 != 0) return GDN_ERR_UNSUPPORTED;
  if ((long long)d->N * d->Hq > (1 << 30)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}
bool has_work(const gdn_paged_dims* d) { return d->N > 0 && d->B > 0; }

int check_cache(const gdn_paged_dims* d, const gdn_paged_cache* c) {
  const int es = esize(d->dtype);
  if (!c || !c->k || !c->v || !c->page_table || !c->cu_seqlens || !c->kv_lens) return GDN_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return GDN_ERR_INVALID_ARG;
  if (!aligned(c->page_table, 4) || !aligned(c->cu_seqlens, 4) || !aligned(c->kv_lens, 4)) return GDN_ERR_INVALID_ARG;
  if (d->num_pages < 1 || d->max_pages < 1 || c->page_table_stride < 0) return GDN_ERR_INVALID_ARG;
  const long long s[6] = {c->k_page_stride, c->k_head_stride, c->k_row_stride,
                          c->v_page_stride, c->v_head_stride, c->v_row_stride};
  for (long long x : s)
    if (!stride_ok(x, es)) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}
bool tokens_ok(const gdn_tokens* t, int es) {
  return t && t->p && aligned(t->p, 16) && stride_ok(t->token_stride, es) && stride_ok(t->head_stride, es);
}

PagedArgs paged_args(const gdn_paged_dims* d, const gdn_paged_cache* c) {
  PagedArgs p{};
  p.N = d->N; p.B = d->B; p.Hq = d->Hq; p.Hk = d->Hk; p.D = d->D;
  p.page_size = d->page_size; p.num_pages = d->num_pages; p.max_pages = d->max_pages;
  p.bf16 = d->dtype == GDN_BF16;
  if (c) {
    p.page_table = c->page_table; p.cu = c->cu_seqlens; p.lens = c->kv_lens;
    p.pt_stride = c->page_table_stride;
    p.kc = c->k; p.vc = c->v;
    p.k_ps = c->k_page_stride; p.k_hs = c->k_head_stride; p.k_rs = c->k_row_stride;
    p.v_ps = c->v_page_stride; p.v_hs = c->v_head_stride; p.v_rs = c->v_row_stride;
  }
  return p;
}

int check_norm(const gdn_norm_dims* d) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->R < 0 || d->G < 1 || d->C < 1) return GDN_ERR_INVALID_ARG;
  if (d->flags & ~GDN_FLAG_GATE_SIGMOID) return GDN_ERR_INVALID_ARG;
  if (!std::isfinite(d->eps) || d->eps < 0.f) return GDN_ERR_INVALID_ARG;
  if (d->dtype != GDN_F32 && d->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (d->C > NORM_MAX_WIDTH || (long long)d->R * d->G > INT_MAX) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}
// Element-aligned rows with strides that do not go backwards; NULL rows are absent parts.
bool rows_ok(const gdn_rows& r, int es) {
  return !r.p || (aligned(r.p, es) && r.row_stride >= 0 && r.group_stride >= 0);
}
bool rows_wide(const gdn_rows& r, int es) {
  return !r.p || (aligned(r.p, 16) && (r.row_stride * es) % 16 == 0 && (r.group_stride * es) % 16 == 0);
}

NormArgs norm_args(const gdn_norm_dims* d, const gdn_norm_parts* q) {
  NormArgs a{};
  a.R = d->R; a.G = d->G; a.C = d->C;
  a.bf16 = d->dtype == GDN_BF16;
  a.sigmoid = (d->flags & GDN_FLAG_GATE_SIGMOID) != 0;
  a.eps = d->eps;
  a.x = q->x.p; a.gate = q->gate.p; a.residual = q->residual.p;
  a.w_post = q->w_post; a.res_scale = q->res_scale; a.w_pre = q->w_pre;
  a.x_rs = q->x.row_stride; a.x_gs = q->x.group_stride;
  a.gate_rs = q->gate.row_stride; a.gate_gs = q->gate.group_stride;
  a.res_rs = q->residual.row_stride; a.res_gs = q->residual.group_stride;
  return a;
}
// The checks and the width rule that forward and backward share; *wide: 16-byte accesses.
int check_parts(const gdn_norm_dims* d, const gdn_norm_parts* q, bool* wide) {
  const int es = esize(d->dtype);
  if (!q || !q->x.p) return GDN_ERR_INVALID_ARG;
  if (!rows_ok(q->x, es) || !rows_ok(q->gate, es) || !rows_ok(q->residual, es)) return GDN_ERR_INVALID_ARG;
  const void* w[3] = {q->w_post, q->res_scale, q->w_pre};
  *wide = (d->C * es) % 16 == 0 && rows_wide(q->x, es) && rows_wide(q->gate, es) && rows_wide(q->residual, es);
  for (const void* x : w) {
    if (x && !aligned(x, es)) return GDN_ERR_INVALID_ARG;
    if (x && !aligned(x, 16)) *wide = false;
  }
  return GDN_OK;
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_kv_append(const gdn_paged_dims* d, const gdn_paged_cache* cache, const gdn_tokens* k, const gdn_tokens* v,
                  const gdn_tokens* q, const gdn_tokens* q_out, const float* cos_table, const float* sin_table,
                  int positions, int rot, void* stream) {
  int st = check_paged(d);
  if (st != GDN_OK) return st;
  if (rot < 0 || rot > d->D || rot % 16 != 0) return GDN_ERR_INVALID_ARG;
  if (!has_work(d)) return GDN_OK;
  if ((st = check_cache(d, cache)) != GDN_OK) return st;
  const int es = esize(d->dtype);
  const bool with_q = q && q->p;
  if (!tokens_ok(k, es) || !tokens_ok(v, es)) return GDN_ERR_INVALID_ARG;
  if (with_q && (!tokens_ok(q, es) || !tokens_ok(q_out, es))) return GDN_ERR_INVALID_ARG;
  if (rot > 0 && (!cos_table || !sin_table || !aligned(cos_table, 16) || !aligned(sin_table, 16) || positions < 1))
    return GDN_ERR_INVALID_ARG;
  AppendArgs a{};
  a.p = paged_args(d, cache);
  a.k = k->p; a.kn_ts = k->token_stride; a.kn_hs = k->head_stride;
  a.v = v->p; a.vn_ts = v->token_stride; a.vn_hs = v->head_stride;
  if (with_q) {
    a.q = q->p; a.q_ts = q->token_stride; a.q_hs = q->head_stride;
    a.q_out = q_out->p; a.qo_ts = q_out->token_stride; a.qo_hs = q_out->head_stride;
  }
  a.cos = cos_table; a.sin = sin_table; a.positions = positions; a.rot = rot;
  a.pairs = (d->flags & GDN_FLAG_ROPE_PAIRS) != 0;
  a.p.err = device_error_word();
  if (!a.p.err) return GDN_ERR_CUDA;
  return launch_status(launch_kv_append(a, static_cast<cudaStream_t>(stream)));
}

size_t gdn_paged_attn_workspace_bytes(const gdn_paged_dims* d, int max_q, int max_kv) {
  if (check_paged(d) != GDN_OK || !has_work(d) || max_q < 1 || max_kv < 1) return 0;
  AttnArgs a{};
  a.p = paged_args(d, nullptr);
  a.max_q = max_q; a.max_kv = max_kv;
  return paged_attn_workspace(a);
}

int gdn_paged_attn(const gdn_paged_dims* d, const gdn_paged_cache* cache, const gdn_tokens* q, float scale, int max_q,
                   int max_kv, const gdn_tokens* out, float* lse, void* workspace, void* stream) {
  int st = check_paged(d);
  if (st != GDN_OK) return st;
  if (!std::isfinite(scale) || scale <= 0.f) return GDN_ERR_INVALID_ARG;
  if (!has_work(d)) return GDN_OK;
  if (max_q < 1 || max_kv < 1) return GDN_ERR_INVALID_ARG;
  if ((st = check_cache(d, cache)) != GDN_OK) return st;
  const int es = esize(d->dtype);
  if (!tokens_ok(q, es) || !tokens_ok(out, es) || !aligned(lse, 4)) return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256)) return GDN_ERR_INVALID_ARG;
  AttnArgs a{};
  a.p = paged_args(d, cache);
  a.q = q->p; a.q_ts = q->token_stride; a.q_hs = q->head_stride;
  a.out = out->p; a.o_ts = out->token_stride; a.o_hs = out->head_stride;
  a.lse = lse; a.scale = scale; a.max_q = max_q; a.max_kv = max_kv;
  a.ws = static_cast<float*>(workspace);
  a.p.err = device_error_word();
  if (!a.p.err) return GDN_ERR_CUDA;
  return launch_status(launch_paged_attn(a, static_cast<cudaStream_t>(stream)));
}

int gdn_block_norm_fwd(const gdn_norm_dims* d, const gdn_norm_parts* parts, void* h, void* y, float* stats,
                       void* stream) {
  int st = check_norm(d);
  if (st != GDN_OK) return st;
  if (d->R == 0) return GDN_OK;
  bool wide = false;
  if ((st = check_parts(d, parts, &wide)) != GDN_OK) return st;
  const int es = esize(d->dtype);
  if (!h || !aligned(h, es) || !stats || !aligned(stats, 8)) return GDN_ERR_INVALID_ARG;
  if (parts->w_pre ? (!y || !aligned(y, es)) : y != nullptr) return GDN_ERR_INVALID_ARG;
  if (!aligned(h, 16) || !aligned(y, 16)) wide = false;
  NormArgs a = norm_args(d, parts);
  a.h = h; a.y = y; a.stats = stats;
  a.err = device_error_word();
  if (!a.err) return GDN_ERR_CUDA;
  return launch_status(launch_block_norm(a, wide, false, static_cast<cudaStream_t>(stream)));
}

size_t gdn_block_norm_workspace_bytes(const gdn_norm_dims* d) {
  if (check_norm(d) != GDN_OK || d->R == 0) return 0;
  return (size_t)norm_bwd_parts(d->C) * 3 * d->C * sizeof(float);
}

int gdn_block_norm_bwd(const gdn_norm_dims* d, const gdn_norm_parts* parts, const float* stats, const gdn_rows* dh,
                       const gdn_rows* dy, const gdn_norm_grads* grads, void* workspace, void* stream) {
  int st = check_norm(d);
  if (st != GDN_OK) return st;
  if (!grads) return GDN_ERR_INVALID_ARG;
  if (d->R == 0) return GDN_OK;  // sums over no rows are the caller's zeros
  bool wide = false;
  if ((st = check_parts(d, parts, &wide)) != GDN_OK) return st;
  const int es = esize(d->dtype);
  const gdn_rows none{};
  const gdn_rows rh = dh ? *dh : none, ry = dy ? *dy : none;
  if (!stats || !aligned(stats, 8) || !workspace || !aligned(workspace, 256)) return GDN_ERR_INVALID_ARG;
  if (!rows_ok(rh, es) || !rows_ok(ry, es)) return GDN_ERR_INVALID_ARG;
  if ((parts->w_pre != nullptr) != (ry.p != nullptr)) return GDN_ERR_INVALID_ARG;
  if (!rh.p && !ry.p) return GDN_ERR_INVALID_ARG;
  if (!grads->dx) return GDN_ERR_INVALID_ARG;
  if ((grads->dgate && !parts->gate.p) || (grads->dresidual && !parts->residual.p) ||
      (grads->dw_post && !parts->w_post) || (grads->dres_scale && !parts->res_scale) ||
      (grads->dw_pre && !parts->w_pre))
    return GDN_ERR_INVALID_ARG;
  void* const rows[3] = {grads->dx, grads->dgate, grads->dresidual};
  for (void* p : rows) {
    if (!aligned(p, es)) return GDN_ERR_INVALID_ARG;
    if (!aligned(p, 16)) wide = false;
  }
  if (!aligned(grads->dw_post, es) || !aligned(grads->dres_scale, es) || !aligned(grads->dw_pre, es))
    return GDN_ERR_INVALID_ARG;
  if (!rows_wide(rh, es) || !rows_wide(ry, es)) wide = false;
  NormArgs a = norm_args(d, parts);
  a.stats = const_cast<float*>(stats);
  a.dh = rh.p; a.dh_rs = rh.row_stride; a.dh_gs = rh.group_stride;
  a.dy = ry.p; a.dy_rs = ry.row_stride; a.dy_gs = ry.group_stride;
  a.dx = grads->dx; a.dgate = grads->dgate; a.dresidual = grads->dresidual;
  a.dw_post = grads->dw_post; a.dres_scale = grads->dres_scale; a.dw_pre = grads->dw_pre;
  a.partial = static_cast<float*>(workspace);
  a.err = device_error_word();
  if (!a.err) return GDN_ERR_CUDA;
  return launch_status(launch_block_norm(a, wide, true, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
