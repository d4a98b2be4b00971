// C ABI of the recurrent mixers' other operators and of the serving plan (include/gdn.h): argument
// validation and dispatch of the causal convolution, the selective scan and the page plan.
#include <climits>
#include <cstdint>

#include "../../include/gdn.h"
#include "kernels.h"
#include "packed.cuh"

namespace gdn {
namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int launch_status(cudaError_t e) {
  return e == cudaSuccess ? GDN_OK : e == cudaErrorNotSupported ? GDN_ERR_UNSUPPORTED : GDN_ERR_CUDA;
}
int esize(int dtype) { return dtype == GDN_BF16 ? 2 : 4; }

// Sequences; training: the backward's calls, whose states are rows of the sequences.
int check_packed(const gdn_packed* q, bool training) {
  if (!q || q->N < 0 || q->B < 0 || q->pool < 0) return GDN_ERR_INVALID_ARG;
  if (q->N > (1 << 30) || q->B > (1 << 30)) return GDN_ERR_UNSUPPORTED;
  if (!q->cu_seqlens && (q->B == 0 ? q->N != 0 : q->N % q->B != 0)) return GDN_ERR_INVALID_ARG;
  if (!aligned(q->cu_seqlens, 4) || !aligned(q->kv_lens, 4) || !aligned(q->slots, 4)) return GDN_ERR_INVALID_ARG;
  if (training && (q->kv_lens || q->slots)) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}
bool pool_ok(const gdn_packed* q) { return q->slots || q->pool >= q->B; }
PackedArgs packed_args(const gdn_packed* q, int flags) {
  PackedArgs p{};
  p.N = q->N; p.B = q->B; p.T = q->cu_seqlens || q->B == 0 ? 0 : q->N / q->B;
  p.cu = q->cu_seqlens; p.lens = q->kv_lens; p.slots = q->slots; p.pool = q->pool;
  p.zero_tail = (flags & GDN_FLAG_ZERO_PADDING) != 0;
  return p;
}
// Rows of the given type: a pointer aligned to it, a stride that does not go backwards.
bool rows_ok(const gdn_rows* r, int es) { return r && r->p && aligned(r->p, es) && r->row_stride >= 0 && r->group_stride >= 0; }
bool rows_wide(const gdn_rows& r, int bytes, int es) {
  return aligned(r.p, bytes) && (r.row_stride * es) % bytes == 0 && (r.group_stride * es) % bytes == 0;
}

int check_conv(const gdn_conv_dims* d) {
  if (!d || d->C < 1) return GDN_ERR_INVALID_ARG;
  if (d->flags & ~(GDN_FLAG_CONV_SILU | GDN_FLAG_ZERO_PADDING)) return GDN_ERR_INVALID_ARG;
  if (d->dtype != GDN_F32 && d->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (d->taps < 2 || d->taps > CONV_MAX_TAPS || d->C > (1 << 24)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}
ConvArgs conv_args(const gdn_conv_dims* d, const gdn_packed* q, int max_q) {
  ConvArgs a{};
  a.q = packed_args(q, d->flags);
  a.C = d->C; a.taps = d->taps;
  a.bf16 = d->dtype == GDN_BF16;
  a.silu = (d->flags & GDN_FLAG_CONV_SILU) != 0;
  a.max_q = q->cu_seqlens ? max_q : a.q.T;
  return a;
}

int check_scan(const gdn_scan_dims* d) {
  if (!d || d->D < 1 || d->G < 1 || d->D % d->G != 0) return GDN_ERR_INVALID_ARG;
  if (d->flags & ~(GDN_FLAG_DT_SOFTPLUS | GDN_FLAG_ZERO_PADDING)) return GDN_ERR_INVALID_ARG;
  if (d->dtype != GDN_F32 && d->dtype != GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if ((d->S != 8 && d->S != 16 && d->S != 32 && d->S != 64) || d->D > (1 << 20)) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}
ScanArgs scan_args(const gdn_scan_dims* d, const gdn_packed* q, int max_q) {
  ScanArgs a{};
  a.q = packed_args(q, d->flags);
  a.D = d->D; a.G = d->G; a.NS = d->S;
  a.bf16 = d->dtype == GDN_BF16;
  a.softplus = (d->flags & GDN_FLAG_DT_SOFTPLUS) != 0;
  a.max_q = q->cu_seqlens ? (max_q < q->N ? max_q : q->N) : a.q.T;
  return a;
}
// The checks of the inputs that forward and backward share; *wide: accesses of four elements.
int scan_parts(const gdn_scan_dims* d, const gdn_scan_parts* p, ScanArgs* a, bool* wide) {
  const int es = esize(d->dtype);
  if (!p) return GDN_ERR_INVALID_ARG;
  if (a->q.N > 0) {
    if (!rows_ok(&p->u, es) || !rows_ok(&p->dt, es) || !rows_ok(&p->B, es) || !rows_ok(&p->C, es)) return GDN_ERR_INVALID_ARG;
    if (p->z.p && !rows_ok(&p->z, es)) return GDN_ERR_INVALID_ARG;
  }
  if (!p->A || !aligned(p->A, 16) || !aligned(p->skip, 16) || !aligned(p->dt_bias, 16) || !aligned(p->h0, 16))
    return GDN_ERR_INVALID_ARG;
  a->u = p->u.p; a->u_ts = p->u.row_stride;
  a->dt = p->dt.p; a->dt_ts = p->dt.row_stride;
  a->z = p->z.p; a->z_ts = p->z.row_stride;
  a->B = p->B.p; a->b_ts = p->B.row_stride; a->b_gs = p->B.group_stride;
  a->C = p->C.p; a->c_ts = p->C.row_stride; a->c_gs = p->C.group_stride;
  a->A = p->A; a->skip = p->skip; a->bias = p->dt_bias; a->h0 = p->h0;
  *wide = (d->D / d->G) % 4 == 0 && rows_wide(p->u, 4 * es, es) && rows_wide(p->dt, 4 * es, es) &&
          rows_wide(p->B, 4 * es, es) && rows_wide(p->C, 4 * es, es) && (!p->z.p || rows_wide(p->z, 4 * es, es));
  return GDN_OK;
}
bool nothing(const gdn_packed* q) { return q->N == 0 && q->B == 0; }

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_causal_conv_fwd(const gdn_conv_dims* d, const gdn_packed* q, const gdn_rows* x, const void* weight, const void* bias,
                        const void* state0, int max_q, const gdn_rows* y, void* state_final, void* stream) {
  int st = check_conv(d);
  if (st != GDN_OK || (st = check_packed(q, false)) != GDN_OK) return st;
  if (nothing(q)) return GDN_OK;
  const int es = esize(d->dtype);
  if (max_q < 1 || !weight || !aligned(weight, es) || !aligned(bias, es) || !aligned(state0, es) || !aligned(state_final, es))
    return GDN_ERR_INVALID_ARG;
  if (q->N > 0 && (!rows_ok(x, es) || !rows_ok(y, es))) return GDN_ERR_INVALID_ARG;
  if ((state0 || state_final) && !pool_ok(q)) return GDN_ERR_INVALID_ARG;
  ConvArgs a = conv_args(d, q, max_q);
  bool wide = (d->C * es) % 16 == 0 && aligned(weight, 16) && aligned(bias, 16) && aligned(state0, 16) && aligned(state_final, 16);
  if (q->N > 0) {
    a.x = x->p; a.x_ts = x->row_stride;
    a.y = const_cast<void*>(y->p); a.y_ts = y->row_stride;
    wide = wide && rows_wide(*x, 16, es) && rows_wide(*y, 16, es);
  }
  a.w = weight; a.bias = bias; a.state0 = state0; a.state_final = state_final;
  a.q.err = device_error_word();
  if (!a.q.err) return GDN_ERR_CUDA;
  return launch_status(launch_causal_conv(a, wide, static_cast<cudaStream_t>(stream)));
}

size_t gdn_causal_conv_workspace_bytes(const gdn_conv_dims* d, const gdn_packed* q) {
  if (check_conv(d) != GDN_OK || check_packed(q, true) != GDN_OK || nothing(q)) return 0;
  return causal_conv_workspace(conv_args(d, q, 1));
}

int gdn_causal_conv_bwd(const gdn_conv_dims* d, const gdn_packed* q, const gdn_rows* x, const void* weight, const void* bias,
                        const void* state0, const gdn_rows* dy, const void* dstate, void* dx, void* dweight, void* dbias,
                        void* dstate0, void* workspace, void* stream) {
  int st = check_conv(d);
  if (st != GDN_OK || (st = check_packed(q, true)) != GDN_OK) return st;
  if (nothing(q)) return GDN_OK;  // sums over no rows are the caller's zeros
  const int es = esize(d->dtype);
  const void* const elems[8] = {weight, bias, state0, dstate, dx, dweight, dbias, dstate0};
  for (const void* p : elems)
    if (!aligned(p, es)) return GDN_ERR_INVALID_ARG;
  if (!weight || !dweight || (dbias && !bias) || !workspace || !aligned(workspace, 256)) return GDN_ERR_INVALID_ARG;
  if (q->N > 0 && (!rows_ok(x, es) || !rows_ok(dy, es) || !dx)) return GDN_ERR_INVALID_ARG;
  ConvArgs a = conv_args(d, q, 1);
  const int vec = 4 * es;
  bool wide = d->C % 4 == 0 && aligned(weight, vec) && aligned(bias, vec) && aligned(state0, vec) && aligned(dstate, vec) &&
              aligned(dx, vec) && aligned(dstate0, vec);
  if (q->N > 0) {
    a.x = x->p; a.x_ts = x->row_stride;
    a.dy = dy->p; a.dy_ts = dy->row_stride;
    wide = wide && rows_wide(*x, vec, es) && rows_wide(*dy, vec, es);
  }
  a.w = weight; a.bias = bias; a.state0 = state0; a.dstate = dstate;
  a.dx = dx; a.dw = dweight; a.dbias = dbias; a.dstate0 = dstate0;
  a.partial = static_cast<float*>(workspace);
  a.q.err = device_error_word();
  if (!a.q.err) return GDN_ERR_CUDA;
  return launch_status(launch_causal_conv_bwd(a, wide, static_cast<cudaStream_t>(stream)));
}

size_t gdn_selective_scan_residual_bytes(const gdn_scan_dims* d, const gdn_packed* q) {
  if (check_scan(d) != GDN_OK || check_packed(q, true) != GDN_OK || nothing(q)) return 0;
  const ScanArgs a = scan_args(d, q, 1);
  return (size_t)packed_numbers(a.q, SCAN_KEEP) * scan_quads(d->D, d->G) * 4 * d->S * sizeof(float);
}

size_t gdn_selective_scan_workspace_bytes(const gdn_scan_dims* d, const gdn_packed* q, int max_q) {
  if (check_scan(d) != GDN_OK || check_packed(q, false) != GDN_OK || nothing(q) || max_q < 1) return 0;
  return selective_scan_workspace(scan_args(d, q, max_q));
}

int gdn_selective_scan_fwd(const gdn_scan_dims* d, const gdn_packed* q, const gdn_scan_parts* parts, int max_q,
                           const gdn_rows* y, float* h_final, float* residuals, void* workspace, void* stream) {
  int st = check_scan(d);
  if (st != GDN_OK || (st = check_packed(q, residuals != nullptr)) != GDN_OK) return st;
  if (nothing(q)) return GDN_OK;
  if (max_q < 1) return GDN_ERR_INVALID_ARG;
  const int es = esize(d->dtype);
  ScanArgs a = scan_args(d, q, max_q);
  bool wide = false;
  if ((st = scan_parts(d, parts, &a, &wide)) != GDN_OK) return st;
  const gdn_rows none{};
  const gdn_rows ry = y ? *y : none;
  if ((q->N > 0 && !rows_ok(&ry, es)) || !aligned(h_final, 16) || !aligned(residuals, 16)) return GDN_ERR_INVALID_ARG;
  if ((parts->h0 || h_final) && !pool_ok(q)) return GDN_ERR_INVALID_ARG;
  if (selective_scan_workspace(a) && (!workspace || !aligned(workspace, 256))) return GDN_ERR_INVALID_ARG;
  wide = wide && rows_wide(ry, 4 * es, es);
  a.y = const_cast<void*>(ry.p); a.y_ts = ry.row_stride;
  a.h_final = h_final; a.kept = residuals; a.ws = workspace;
  a.q.err = device_error_word();
  if (!a.q.err) return GDN_ERR_CUDA;
  return launch_status(launch_selective_scan(a, wide, static_cast<cudaStream_t>(stream)));
}

size_t gdn_selective_scan_bwd_workspace_bytes(const gdn_scan_dims* d, const gdn_packed* q, int max_q) {
  if (check_scan(d) != GDN_OK || check_packed(q, true) != GDN_OK || nothing(q) || max_q < 1) return 0;
  return selective_scan_bwd_workspace(scan_args(d, q, max_q));
}

int gdn_selective_scan_bwd(const gdn_scan_dims* d, const gdn_packed* q, const gdn_scan_parts* parts, const float* residuals,
                           int max_q, const gdn_rows* dy, const float* dh_final, const gdn_scan_grads* grads, void* workspace,
                           void* stream) {
  int st = check_scan(d);
  if (st != GDN_OK || (st = check_packed(q, true)) != GDN_OK) return st;
  if (!grads) return GDN_ERR_INVALID_ARG;
  if (nothing(q)) return GDN_OK;  // sums over no rows are the caller's zeros
  if (max_q < 1) return GDN_ERR_INVALID_ARG;
  const int es = esize(d->dtype);
  ScanArgs a = scan_args(d, q, max_q);
  bool wide = false;
  if ((st = scan_parts(d, parts, &a, &wide)) != GDN_OK) return st;
  const gdn_rows none{};
  const gdn_rows ry = dy ? *dy : none;
  if ((q->N > 0 && !rows_ok(&ry, es)) || !residuals || !aligned(residuals, 16) || !aligned(dh_final, 16)) return GDN_ERR_INVALID_ARG;
  const gdn_scan_grads& g = *grads;
  if (!g.dA || (q->N > 0 && (!g.du || !g.ddt || !g.dB || !g.dC))) return GDN_ERR_INVALID_ARG;
  if ((q->N > 0 && (g.dz != nullptr) != (parts->z.p != nullptr)) || (g.dskip && !parts->skip) || (g.ddt_bias && !parts->dt_bias))
    return GDN_ERR_INVALID_ARG;
  const void* const rows[5] = {g.du, g.ddt, g.dz, g.dB, g.dC};
  for (const void* p : rows) {
    if (!aligned(p, es)) return GDN_ERR_INVALID_ARG;
    wide = wide && aligned(p, 4 * es);
  }
  const void* const sums[4] = {g.dA, g.dskip, g.ddt_bias, g.dh0};
  for (const void* p : sums)
    if (!aligned(p, 16)) return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256)) return GDN_ERR_INVALID_ARG;
  wide = wide && rows_wide(ry, 4 * es, es);
  a.dy = ry.p; a.dy_ts = ry.row_stride;
  a.kept = const_cast<float*>(residuals);
  a.dh_final = dh_final;
  a.du = g.du; a.ddt = g.ddt; a.dz = g.dz; a.dB = g.dB; a.dC = g.dC;
  a.dA = g.dA; a.dskip = g.dskip; a.dbias = g.ddt_bias; a.dh0 = g.dh0;
  a.ws = workspace;
  a.q.err = device_error_word();
  if (!a.q.err) return GDN_ERR_CUDA;
  return launch_status(launch_selective_scan_bwd(a, wide, static_cast<cudaStream_t>(stream)));
}

int gdn_page_plan(const gdn_plan_dims* d, int* page_table, long long page_table_stride, const int* kv_lens,
                  const int* new_tokens, int* free_pages, const int* free_count, const gdn_plan_out* out, void* stream) {
  if (!d || d->B < 0 || d->page_size < 1 || d->max_pages < 0 || d->num_free < 0 || d->max_tokens < 0) return GDN_ERR_INVALID_ARG;
  if (d->B > PLAN_MAX_REQUESTS || d->max_tokens > (1 << 30)) return GDN_ERR_UNSUPPORTED;
  if (!out || !out->cu_seqlens || !out->free_count || !free_count) return GDN_ERR_INVALID_ARG;
  if (d->B > 0 && (!kv_lens || !new_tokens || !out->kv_lens)) return GDN_ERR_INVALID_ARG;
  if (d->B > 0 && d->max_pages > 0 && (!page_table || page_table_stride < d->max_pages)) return GDN_ERR_INVALID_ARG;
  if (d->num_free > 0 && !free_pages) return GDN_ERR_INVALID_ARG;
  if (d->max_tokens > 0 && (!out->requests || !out->positions || !out->slots)) return GDN_ERR_INVALID_ARG;
  const void* const ints[10] = {page_table, kv_lens, new_tokens, free_pages, free_count,
                                out->cu_seqlens, out->kv_lens, out->free_count, out->requests, out->positions};
  for (const void* p : ints)
    if (!aligned(p, 4)) return GDN_ERR_INVALID_ARG;
  if (!aligned(out->slots, 8)) return GDN_ERR_INVALID_ARG;
  // every CTA reads the inputs for itself, so none may be written
  const int* const outs[3] = {out->cu_seqlens, out->kv_lens, out->free_count};
  for (const int* p : outs)
    if (p && (p == kv_lens || p == new_tokens || p == free_count)) return GDN_ERR_INVALID_ARG;
  PlanArgs a{};
  a.B = d->B; a.page_size = d->page_size; a.max_pages = d->max_pages; a.num_free = d->num_free; a.max_tokens = d->max_tokens;
  a.page_table = page_table; a.pt_stride = page_table_stride;
  a.kv_lens = kv_lens; a.new_tokens = new_tokens; a.free_pages = free_pages; a.free_count = free_count;
  a.cu = out->cu_seqlens; a.lens_out = out->kv_lens; a.count_out = out->free_count;
  a.requests = out->requests; a.positions = out->positions; a.slots = out->slots;
  a.err = device_error_word();
  if (!a.err) return GDN_ERR_CUDA;
  return launch_status(launch_page_plan(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
