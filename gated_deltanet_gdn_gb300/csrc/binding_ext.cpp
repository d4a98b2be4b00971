// Compiled argument marshalling of the paged cache, block norm, convolution, selective scan and plan calls: takes the tensors
// apart, checks them, allocates what the caller left out and calls the C ABI on the current
// stream. Nothing is computed here.
//
// A decoding step makes these calls once per layer on a few kilobytes; the ctypes
// marshalling of the same arguments took 30 to 40 us a call (Grace, Python 3.12), several
// times the kernels' own time.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/DimVector.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/zeros.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <array>
#include <climits>
#include <initializer_list>
#include <string>

#include "../../include/gdn.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;  // binding.GdnError

// A refusal, as GdnError(name, status, message).
struct Refusal {
  std::string name, msg;
  int status;
};
[[noreturn]] void refuse(const char* name, const std::string& msg, int status = GDN_ERR_INVALID_ARG) {
  throw Refusal{name, msg, status};
}
void check(const char* fn, int status) {
  if (status != GDN_OK) refuse(fn, gdn_status_string(status), status);
}
std::string show(at::IntArrayRef v) {
  std::string s = "[";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + "]";
}

// Other Python threads run while a call allocates and launches, which waits when the launch
// queue or the memory is full.
struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  NoGil() = default;
  NoGil(const NoGil&) = delete;
  ~NoGil() { PyEval_RestoreThread(state); }
};

struct NotTensor {};
const Tensor* optional_tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
    throw NotTensor{};
  }
  return &THPVariable_Unpack(o);
}
const Tensor& tensor(PyObject* o, const char* name) {
  const Tensor* t = optional_tensor(o, name);
  if (!t) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
    throw NotTensor{};
  }
  return *t;
}
long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw NotTensor{};
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw NotTensor{};
  return v;
}
PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }

int dtype_code(const Tensor& t) {
  if (t.scalar_type() == at::kFloat) return GDN_F32;
  if (t.scalar_type() == at::kBFloat16) return GDN_BF16;
  refuse("dtype", std::string("unsupported dtype ") + c10::toString(t.scalar_type()) + " (float32 or bfloat16)",
         GDN_ERR_UNSUPPORTED);
}
int to_int(int64_t v, const char* name) {
  if (v < 0 || v > INT_MAX) refuse(name, std::string(name) + " is out of range", GDN_ERR_UNSUPPORTED);
  return (int)v;
}
void on_device(const Tensor& t, c10::Device dev, const char* name) {
  if (!t.is_cuda() || t.device() != dev) refuse(name, std::string(name) + " must be a CUDA tensor on " + dev.str());
}
// A dimension of one element has no stride of its own.
long long step(const Tensor& t, int64_t d) { return t.size(d) == 1 ? 0 : t.stride(d); }
void unit_channels(const Tensor& t, const char* name) {
  if (t.numel() > 0 && t.size(-1) != 1 && t.stride(-1) != 1)
    refuse(name, std::string(name) + " must have contiguous channels");
}

// A gradient that would be lost without a word is refused: the paged calls have no backward, the mixers' has functions of
// its own.
void no_gradient(const Tensor* t, const char* name) {
  if (t && c10::GradMode::is_enabled() && t->requires_grad())
    refuse(name, std::string(name) + " requires a gradient, and this call has no backward: call it under torch.no_grad() or detach " + name,
           GDN_ERR_UNSUPPORTED);
}

gdn_tokens tokens(const Tensor& t, at::IntArrayRef shape, const Tensor& like, const char* name) {
  if (t.sizes() != shape) refuse(name, std::string(name) + " must be " + show(shape) + ", got " + show(t.sizes()));
  on_device(t, like.device(), name);
  if (t.scalar_type() != like.scalar_type()) refuse(name, std::string(name) + " must have the cache's type");
  unit_channels(t, name);
  return gdn_tokens{t.data_ptr(), step(t, 0), step(t, 1)};
}
void int_array(const Tensor& t, at::IntArrayRef shape, c10::Device dev, const char* name) {
  if (t.scalar_type() != at::kInt || t.sizes() != shape)
    refuse(name, std::string(name) + " must be int32 " + show(shape) + ", got " + c10::toString(t.scalar_type()) + " " +
                     show(t.sizes()));
  on_device(t, dev, name);
  unit_channels(t, name);
}

// dims and cache of a paged call; the first token tensor gives N.
void paged(const Tensor& tok, int64_t Hq, const Tensor& kc, const Tensor& vc, const Tensor& table, const Tensor& cu,
           const Tensor& lens, long long flags, gdn_paged_dims* d, gdn_paged_cache* c) {
  const c10::Device dev = kc.device();
  if (tok.dim() != 3) refuse("tokens", "token tensors must be [N, heads, D]");
  if (kc.dim() != 4) refuse("k_cache", "k_cache must be [pages, heads, page size, D]");
  if (vc.sizes() != kc.sizes() || vc.scalar_type() != kc.scalar_type())
    refuse("v_cache", "v_cache must be like k_cache");
  on_device(kc, dev, "k_cache");
  on_device(vc, dev, "v_cache");
  unit_channels(kc, "k_cache");
  unit_channels(vc, "v_cache");
  if (lens.dim() != 1) refuse("kv_lens", "kv_lens must be [sequences]");
  if (table.dim() != 2) refuse("page_table", "page_table must be [sequences, pages per sequence]");
  const int64_t B = lens.size(0);
  int_array(lens, {B}, dev, "kv_lens");
  int_array(cu, {B + 1}, dev, "cu_seqlens");
  int_array(table, {B, table.size(1)}, dev, "page_table");
  d->N = to_int(tok.size(0), "N"); d->B = to_int(B, "B");
  d->Hq = to_int(Hq, "Hq"); d->Hk = to_int(kc.size(1), "Hk"); d->D = to_int(kc.size(3), "D");
  d->page_size = to_int(kc.size(2), "page_size"); d->num_pages = to_int(kc.size(0), "num_pages");
  d->max_pages = to_int(table.size(1), "max_pages");
  d->dtype = dtype_code(kc); d->flags = (int)flags;
  c->k = kc.data_ptr(); c->v = vc.data_ptr();
  c->k_page_stride = step(kc, 0); c->k_head_stride = step(kc, 1); c->k_row_stride = step(kc, 2);
  c->v_page_stride = step(vc, 0); c->v_head_stride = step(vc, 1); c->v_row_stride = step(vc, 2);
  c->page_table = table.data_ptr<int>(); c->page_table_stride = table.stride(0);
  c->cu_seqlens = cu.data_ptr<int>(); c->kv_lens = lens.data_ptr<int>();
}

const float* rope_table(const Tensor& t, const Tensor& like, c10::Device dev, const char* name) {
  if (t.dim() != 2 || t.sizes() != like.sizes() || t.scalar_type() != at::kFloat || !t.is_contiguous())
    refuse(name, std::string(name) + " must be a contiguous float32 [positions, rot / 2] table");
  on_device(t, dev, name);
  return t.data_ptr<float>();
}

// New memory of the current device, which the callers have set to `dev`. It comes from PyTorch's allocator without its
// dispatcher, which took a third of a short call's host time (one token of attention: 6.5 us, through the dispatcher
// 9.8), and without the checks of its empty() (0.4 us).
Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, c10::Device) {
  int64_t n = 1;
  for (int64_t v : sizes) n *= v;
  c10::Allocator* const allocator = c10::cuda::CUDACachingAllocator::get();
  const size_t bytes = (size_t)n * c10::elementSize(type);
  c10::Storage storage(c10::Storage::use_byte_size_t(), bytes, allocator->allocate(bytes), allocator, true);
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(std::move(storage), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                      c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
  return t;
}

// A contiguous vector of n elements, `at` bytes into memory that it shares (at a multiple of their size).
Tensor part_of(const Tensor& all, int64_t at, int64_t n, at::ScalarType type) {
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                      c10::scalarTypeToTypeMeta(type));
  c10::TensorImpl* const impl = t.unsafeGetTensorImpl();
  impl->set_storage_offset(at / (int64_t)c10::elementSize(type));
  impl->set_sizes_contiguous({n});
  return t;
}

// Scratch of at least `need` bytes on the current device: the caller's, or new.
void* scratch(const Tensor* w, size_t need, const Tensor& like, c10::DataPtr* own) {
  if (w) {
    on_device(*w, like.device(), "workspace");
    if (!w->is_contiguous() || w->nbytes() < need)
      refuse("workspace", "workspace must be contiguous and hold " + std::to_string(need) + " bytes");
    return w->data_ptr();
  }
  *own = c10::cuda::CUDACachingAllocator::get()->allocate(need ? need : 1);
  return own->get();
}

template <class F>
PyObject* guarded(const char* fn, PyObject* const* args, Py_ssize_t n, Py_ssize_t want, F body) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", fn, want);
    return nullptr;
  }
  try {
    return body();
  } catch (const Refusal& r) {
    PyObject* e = g_error ? PyObject_CallFunction(g_error, "sis", r.name.c_str(), r.status, r.msg.c_str()) : nullptr;
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
      PyErr_SetString(PyExc_RuntimeError, r.msg.c_str());
    }
  } catch (const NotTensor&) {
  } catch (...) {  // PyTorch's own, as its calls raise them (out of memory among them)
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// (k, v, k_cache, v_cache, page_table, cu_seqlens, kv_lens, q, q_out, cos, sin, flags)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("kv_append", a, n, 12, [&]() -> PyObject* {
    const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &kc = tensor(a[2], "k_cache"),
                 &vc = tensor(a[3], "v_cache");
    const Tensor &table = tensor(a[4], "page_table"), &cu = tensor(a[5], "cu_seqlens"), &lens = tensor(a[6], "kv_lens");
    const Tensor *q = optional_tensor(a[7], "q"), *qo = optional_tensor(a[8], "q_out"),
                 *cos = optional_tensor(a[9], "cos"), *sin = optional_tensor(a[10], "sin");
    no_gradient(&k, "k"); no_gradient(&v, "v"); no_gradient(&kc, "k_cache"); no_gradient(&vc, "v_cache");
    no_gradient(q, "q"); no_gradient(qo, "q_out"); no_gradient(cos, "cos"); no_gradient(sin, "sin");
    if (q && q->dim() != 3) refuse("q", "q must be [N, heads, D]");
    gdn_paged_dims d;
    gdn_paged_cache c;
    paged(k, q ? q->size(1) : (kc.dim() == 4 ? kc.size(1) : 1), kc, vc, table, cu, lens, integer(a[11]), &d, &c);
    const gdn_tokens kt = tokens(k, {d.N, d.Hk, d.D}, kc, "k"), vt = tokens(v, {d.N, d.Hk, d.D}, kc, "v");
    gdn_tokens qt{}, qot{};
    Tensor own;
    if (q) {
      qt = tokens(*q, {d.N, d.Hq, d.D}, kc, "q");
      if (qo) qot = tokens(*qo, q->sizes(), kc, "q_out");
    }
    if (!cos != !sin) refuse("cos", "cos and sin go together");
    const float *cp = nullptr, *sp = nullptr;
    int positions = 0, rot = 0;
    if (cos) {
      cp = rope_table(*cos, *cos, kc.device(), "cos");
      sp = rope_table(*sin, *cos, kc.device(), "sin");
      positions = to_int(cos->size(0), "positions");
      rot = to_int(2 * cos->size(1), "rot");
    }
    {
      const NoGil nogil;
      const c10::cuda::OptionalCUDAGuard guard(kc.device());
      if (q && !qo) {
        own = fresh(q->sizes(), kc.scalar_type(), kc.device());
        qot = tokens(own, q->sizes(), kc, "q_out");
      }
      check("gdn_kv_append", gdn_kv_append(&d, &c, &kt, &vt, q ? &qt : nullptr, q ? &qot : nullptr, cp, sp, positions, rot,
                                           c10::cuda::getCurrentCUDAStream(kc.device().index()).stream()));
    }
    if (!q) Py_RETURN_NONE;
    if (own.defined()) return wrap(own);
    Py_INCREF(a[8]);
    return a[8];
  });
}

// (q, k_cache, v_cache, page_table, cu_seqlens, kv_lens, scale, max_q, max_kv, out, lse, workspace)
PyObject* paged_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("paged_attn", a, n, 12, [&]() -> PyObject* {
    const Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache");
    const Tensor &table = tensor(a[3], "page_table"), &cu = tensor(a[4], "cu_seqlens"), &lens = tensor(a[5], "kv_lens");
    const Tensor *out = optional_tensor(a[9], "out"), *lse = optional_tensor(a[10], "lse");
    no_gradient(&q, "q"); no_gradient(&kc, "k_cache"); no_gradient(&vc, "v_cache"); no_gradient(out, "out");
    no_gradient(lse, "lse");
    if (q.dim() != 3) refuse("q", "q must be [N, heads, D]");
    gdn_paged_dims d;
    gdn_paged_cache c;
    paged(q, q.size(1), kc, vc, table, cu, lens, 0, &d, &c);
    const gdn_tokens qt = tokens(q, {d.N, d.Hq, d.D}, kc, "q");
    double scale = 1.0 / std::sqrt((double)(d.D > 0 ? d.D : 1));
    if (a[6] != Py_None) scale = number(a[6]);
    const long long cap = (long long)d.max_pages * d.page_size;
    const int max_q = a[7] == Py_None ? (d.N > 0 ? d.N : 1) : to_int(integer(a[7]), "max_q");
    const int max_kv = a[8] == Py_None ? (int)(cap < 1 ? 1 : cap > INT_MAX ? INT_MAX : cap) : to_int(integer(a[8]), "max_kv");
    const Tensor* given = optional_tensor(a[11], "workspace");
    Tensor own;
    gdn_tokens ot{};
    if (out) ot = tokens(*out, q.sizes(), kc, "out");
    if (lse) {
      if (lse->scalar_type() != at::kFloat || lse->sizes() != at::IntArrayRef({d.N, d.Hq}) || !lse->is_contiguous())
        refuse("lse", "lse must be a contiguous float32 [N, Hq]");
      on_device(*lse, kc.device(), "lse");
    }
    {
      const NoGil nogil;
      const c10::cuda::OptionalCUDAGuard guard(kc.device());
      c10::DataPtr ws;
      if (!out) {
        own = fresh(q.sizes(), kc.scalar_type(), kc.device());
        ot = tokens(own, q.sizes(), kc, "out");
      }
      void* w = scratch(given, gdn_paged_attn_workspace_bytes(&d, max_q, max_kv), kc, &ws);
      check("gdn_paged_attn", gdn_paged_attn(&d, &c, &qt, (float)scale, max_q, max_kv, &ot, lse ? lse->data_ptr<float>() : nullptr,
                                             w, c10::cuda::getCurrentCUDAStream(kc.device().index()).stream()));
    }
    if (own.defined()) return wrap(own);
    Py_INCREF(a[9]);
    return a[9];
  });
}

// A tensor of x's shape as rows [R, G, C] with contiguous channels (a 2-D tensor has G = 1).
gdn_rows rows(const Tensor* t, const Tensor& x, const char* name) {
  if (!t) return gdn_rows{};
  if (t->sizes() != x.sizes() || t->scalar_type() != x.scalar_type())
    refuse(name, std::string(name) + " must have x's type and be " + show(x.sizes()) + ", got " + show(t->sizes()));
  on_device(*t, x.device(), name);
  if (t->numel() == 0) return gdn_rows{t->data_ptr(), 0, 0};
  unit_channels(*t, name);
  const int64_t nd = t->dim();
  if (nd == 2) return gdn_rows{t->data_ptr(), step(*t, 0), 0};
  // the leading dimensions fold into one when each stride is the next one's times its size
  int64_t last = -1, size = 1;
  for (int64_t i = nd - 3; i >= 0; --i) {
    if (t->size(i) == 1) continue;
    if (last >= 0 && t->stride(i) != t->stride(last) * size)
      refuse(name, std::string("the leading dimensions of ") + name + " must fold into one");
    if (last < 0) last = i;
    size *= t->size(i);
  }
  return gdn_rows{t->data_ptr(), last < 0 ? 0 : t->stride(last), step(*t, nd - 2)};
}
const void* weight(const Tensor* w, const Tensor& x, const char* name) {
  if (!w) return nullptr;
  if (w->dim() != 1 || w->size(0) != x.size(-1) || w->scalar_type() != x.scalar_type() || !w->is_contiguous())
    refuse(name, std::string(name) + " must be contiguous, of x's type and [" + std::to_string(x.size(-1)) + "]");
  on_device(*w, x.device(), name);
  return w->data_ptr();
}

struct Norm {
  const Tensor* part[6];  // x, gate, residual, w_post, res_scale, w_pre
  gdn_norm_dims d;
  gdn_norm_parts p;
  Norm(PyObject* x_, PyObject* const* a, double eps, long long flags) {
    static const char* const names[6] = {"x", "gate", "residual", "w_post", "res_scale", "w_pre"};
    const Tensor& x = tensor(x_, "x");
    part[0] = &x;
    for (int i = 1; i < 6; ++i) part[i] = optional_tensor(a[i - 1], names[i]);
    if (x.dim() < 2) refuse("x", "x must be [rows, C] or [rows..., groups, C]");
    on_device(x, x.device(), "x");
    const int64_t C = x.size(-1), G = x.dim() == 2 ? 1 : x.size(-2);
    d.C = to_int(C, "C");
    d.G = to_int(G > 0 ? G : 1, "G");
    d.R = to_int(x.numel() ? x.numel() / (C * G) : 0, "R");
    d.dtype = dtype_code(x);
    d.flags = (int)flags;
    d.eps = (float)eps;
    p.x = rows(part[0], x, names[0]);
    p.gate = rows(part[1], x, names[1]);
    p.residual = rows(part[2], x, names[2]);
    p.w_post = weight(part[3], x, names[3]);
    p.res_scale = weight(part[4], x, names[4]);
    p.w_pre = weight(part[5], x, names[5]);
  }
};

// (x, gate, residual, w_post, res_scale, w_pre, eps, flags) -> (h, y, stats)
PyObject* block_norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("block_norm_fwd", a, n, 8, [&]() -> PyObject* {
    const Norm q(a[0], a + 1, number(a[6]), integer(a[7]));
    const Tensor& x = *q.part[0];
    Tensor h, y, stats;
    {
      const NoGil nogil;
      const c10::cuda::OptionalCUDAGuard guard(x.device());
      h = fresh(x.sizes(), x.scalar_type(), x.device());
      if (q.p.w_pre) y = fresh(x.sizes(), x.scalar_type(), x.device());
      stats = fresh({q.d.R, q.d.G, 2}, at::kFloat, x.device());
      check("gdn_block_norm_fwd", gdn_block_norm_fwd(&q.d, &q.p, h.data_ptr(), y.defined() ? y.data_ptr() : nullptr,
                                                     stats.data_ptr<float>(),
                                                     c10::cuda::getCurrentCUDAStream(x.device().index()).stream()));
    }
    PyObject* yo = y.defined() ? wrap(y) : Py_NewRef(Py_None);
    return Py_BuildValue("(NNN)", wrap(h), yo, wrap(stats));
  });
}

// (x, stats, dh, dy, gate, residual, w_post, res_scale, w_pre, eps, flags, workspace)
// -> (dx, dgate, dresidual, dw_post, dres_scale, dw_pre)
PyObject* block_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("block_norm_bwd", a, n, 12, [&]() -> PyObject* {
    const Norm q(a[0], a + 4, number(a[9]), integer(a[10]));
    const Tensor &x = *q.part[0], &stats = tensor(a[1], "stats");
    const Tensor *dh = optional_tensor(a[2], "dh"), *dy = optional_tensor(a[3], "dy");
    if (stats.scalar_type() != at::kFloat || stats.sizes() != at::IntArrayRef({q.d.R, q.d.G, 2}) || !stats.is_contiguous())
      refuse("stats", "stats must be the forward's");
    on_device(stats, x.device(), "stats");
    const gdn_rows rh = rows(dh, x, "dh"), ry = rows(dy, x, "dy");
    const Tensor* given = optional_tensor(a[11], "workspace");
    Tensor g[6];
    {
      const NoGil nogil;
      const c10::cuda::OptionalCUDAGuard guard(x.device());
      c10::DataPtr ws;
      void* p[6];
      for (int i = 0; i < 6; ++i) {
        // without rows nothing is launched, and the weights' sums are zero
        if (q.part[i])
          g[i] = q.d.R == 0 ? at::zeros(q.part[i]->sizes(), x.options())
                            : fresh(q.part[i]->sizes(), x.scalar_type(), x.device());
        p[i] = g[i].defined() ? g[i].data_ptr() : nullptr;
      }
      const gdn_norm_grads grads{p[0], p[1], p[2], p[3], p[4], p[5]};
      void* w = scratch(given, gdn_block_norm_workspace_bytes(&q.d), x, &ws);
      check("gdn_block_norm_bwd", gdn_block_norm_bwd(&q.d, &q.p, stats.data_ptr<float>(), dh ? &rh : nullptr, dy ? &ry : nullptr,
                                                     &grads, w, c10::cuda::getCurrentCUDAStream(x.device().index()).stream()));
    }
    PyObject* out = PyTuple_New(6);
    for (int i = 0; out && i < 6; ++i) PyTuple_SET_ITEM(out, i, g[i].defined() ? wrap(g[i]) : Py_NewRef(Py_None));
    return out;
  });
}

// Bytes that a call reads or writes: rows of `width`, `step` apart.
struct Span {
  const char* name;
  uintptr_t at;
  int64_t rows, step, width;
};
Span span(const Tensor* t, const char* name) {  // contiguous
  if (!t) return Span{name, 0, 0, 0, 0};
  return Span{name, reinterpret_cast<uintptr_t>(t->data_ptr()), t->numel() > 0, 0, (int64_t)t->nbytes()};
}
Span span(const gdn_rows& r, int64_t n, int64_t groups, int64_t width, int64_t es, const char* name) {
  return Span{name, reinterpret_cast<uintptr_t>(r.p), r.p && width > 0 ? n : 0, r.row_stride * es,
              ((groups - 1) * r.group_stride + width) * es};
}
// Whether two share a byte. Rows as far apart as the other's may lie between those (columns of one buffer); of other rows,
// ranges that meet count as shared.
bool meet(const Span& a, const Span& b) {
  if (a.rows == 0 || b.rows == 0) return false;
  const int64_t along_a = (a.rows - 1) * a.step, along_b = (b.rows - 1) * b.step;
  if (a.at + along_a + a.width <= b.at || b.at + along_b + b.width <= a.at) return false;
  if (along_a && along_b && a.step != b.step) return true;
  const int64_t step = along_a ? a.step : b.step;
  if (!along_a && !along_b) return true;
  int64_t d = (int64_t)(a.at - b.at) % step;
  if (d < 0) d += step;
  return d < b.width || d + a.width > step;
}
// Refuses an output on the memory of what the call reads; `same`: spans that it may be.
void apart(const Span& out, std::initializer_list<Span> reads, std::initializer_list<Span> same = {}) {
  for (const Span& r : reads)
    if (meet(out, r)) refuse(out.name, std::string(out.name) + " shares memory with " + r.name);
  for (const Span& r : same)
    if ((out.at != r.at || out.step != r.step) && meet(out, r))
      refuse(out.name, std::string(out.name) + " shares memory with " + r.name + " and is not the same");
}

// The sequences of a convolution or scan call: [B, T, ...] tensors, or [N, ...] with cu_seqlens.
struct Seqs {
  gdn_packed q{};
  at::DimVector lead;  // [B, T] or [N]
  int max_q = 1;
  c10::Device dev;
  at::ScalarType type;
  Seqs(const Tensor& x, const char* name, const Tensor* slots, const Tensor* cu, const Tensor* lens, PyObject* max_q_)
      : dev(x.device()), type(x.scalar_type()) {
    on_device(x, dev, name);
    dtype_code(x);
    if (cu) {
      if (x.dim() != 2) refuse(name, std::string(name) + " must be [tokens, channels] with cu_seqlens");
      if (cu->dim() != 1 || cu->size(0) < 1) refuse("cu_seqlens", "cu_seqlens must be [sequences + 1]");
      q.B = to_int(cu->size(0) - 1, "B");
      int_array(*cu, {(int64_t)q.B + 1}, dev, "cu_seqlens");
      q.cu_seqlens = cu->data_ptr<int>();
      max_q = (int)std::max<int64_t>(x.size(0), 1);
      if (max_q_ != Py_None) max_q = to_int(integer(max_q_), "max_q");
    } else {
      if (x.dim() != 3) refuse(name, std::string(name) + " must be [sequences, tokens, channels], or [tokens, channels] with cu_seqlens");
      q.B = to_int(x.size(0), "B");
      max_q = to_int(std::max<int64_t>(x.size(1), 1), "tokens");
    }
    for (int64_t i = 0; i + 1 < x.dim(); ++i) lead.push_back(x.size(i));
    q.N = to_int(x.dim() == 2 ? x.size(0) : x.size(0) * x.size(1), "N");
    q.pool = q.B;
    if (lens) {
      int_array(*lens, {q.B}, dev, "kv_lens");
      q.kv_lens = lens->data_ptr<int>();
    }
    if (slots) {
      int_array(*slots, {q.B}, dev, "slots");
      q.slots = slots->data_ptr<int>();
      with_slots = true;
    }
  }
  // [lead..., tail...] with contiguous channels; the leading dimensions fold into one.
  gdn_rows rows(const Tensor* t, at::IntArrayRef tail, const char* name) const {
    if (!t) return gdn_rows{};
    at::DimVector want(lead);
    want.append(tail.begin(), tail.end());
    if (t->sizes() != at::IntArrayRef(want) || t->scalar_type() != type)
      refuse(name, std::string(name) + " must be " + c10::toString(type) + " " + show(want) + ", got " +
                       c10::toString(t->scalar_type()) + " " + show(t->sizes()));
    on_device(*t, dev, name);
    if (t->numel() == 0) return gdn_rows{t->data_ptr(), 0, 0};
    unit_channels(*t, name);
    const int64_t nl = (int64_t)lead.size();
    long long rs = step(*t, nl - 1);
    if (nl == 2 && t->size(0) > 1) {
      if (t->size(1) == 1) rs = t->stride(0);
      else if (t->stride(0) != t->size(1) * t->stride(1))
        refuse(name, std::string("the leading dimensions of ") + name + " must fold into one");
    }
    return gdn_rows{t->data_ptr(), rs, tail.size() == 2 ? step(*t, nl) : 0};
  }
  // Rows to be written: no two of them on the same memory.
  gdn_rows out_rows(const Tensor& t, int64_t width, const char* name) const {
    const gdn_rows r = rows(&t, {width}, name);
    if (q.N > 1 && width > 0 && r.row_stride < width) refuse(name, std::string(name) + " must have rows of its own");
    return r;
  }
  // A contiguous tensor [rows of the pool or sequences, tail...].
  void* state(const Tensor* t, at::IntArrayRef tail, at::ScalarType want, bool pooled, const char* name) {
    if (!t) return nullptr;
    if (t->dim() != 1 + (int64_t)tail.size() || t->sizes().slice(1) != tail || t->scalar_type() != want || !t->is_contiguous())
      refuse(name, std::string(name) + " must be contiguous " + c10::toString(want) + " [" + (pooled ? "rows" : "sequences") +
                       ", ...] with rows " + show(tail) + ", got " + c10::toString(t->scalar_type()) + " " + show(t->sizes()));
    on_device(*t, dev, name);
    if (with_slots && pooled) {
      if (pool_known && t->size(0) != q.pool) refuse(name, "the state pools must have the same number of rows");
      q.pool = to_int(t->size(0), "pool");
      pool_known = true;
    } else if (t->size(0) != q.B) {
      refuse(name, std::string(name) + " must have a row for each of the " + std::to_string(q.B) + " sequences");
    }
    return t->data_ptr();
  }
  bool with_slots = false, pool_known = false;
};
const void* exactly(const Tensor* t, at::IntArrayRef sizes, at::ScalarType type, c10::Device dev, const char* name) {
  if (!t) return nullptr;
  if (t->sizes() != sizes || t->scalar_type() != type || !t->is_contiguous())
    refuse(name, std::string(name) + " must be contiguous " + c10::toString(type) + " " + show(sizes) + ", got " +
                     c10::toString(t->scalar_type()) + " " + show(t->sizes()));
  on_device(*t, dev, name);
  return t->data_ptr();
}
void* stream_of(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

struct Conv {
  gdn_conv_dims d;
  const void *w, *bias;
  Conv(const Seqs& s, const Tensor& x, const Tensor& weight, const Tensor* b, long long flags) {
    const int64_t C = x.size(-1);
    if (weight.dim() != 2) refuse("weight", "weight must be [channels, taps]");
    d.C = to_int(C, "C");
    d.taps = to_int(weight.size(1), "taps");
    d.dtype = dtype_code(x);
    d.flags = (int)flags;
    w = exactly(&weight, {C, weight.size(1)}, s.type, s.dev, "weight");
    bias = exactly(b, {C}, s.type, s.dev, "bias");
  }
};

// (x, weight, bias, state0, state_final, slots, cu_seqlens, kv_lens, max_q, flags, out) -> (y, state_final)
PyObject* causal_conv_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("causal_conv_fwd", a, n, 11, [&]() -> PyObject* {
    const Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight");
    const Tensor *bias = optional_tensor(a[2], "bias"), *state0 = optional_tensor(a[3], "state0"),
                 *state_final = optional_tensor(a[4], "state_final"), *slots = optional_tensor(a[5], "slots"),
                 *out = optional_tensor(a[10], "out");
    no_gradient(&x, "x"); no_gradient(&weight, "weight"); no_gradient(bias, "bias"); no_gradient(state0, "state0");
    no_gradient(state_final, "state_final"); no_gradient(out, "out");
    Seqs s(x, "x", slots, optional_tensor(a[6], "cu_seqlens"), optional_tensor(a[7], "kv_lens"), a[8]);
    Conv c(s, x, weight, bias, integer(a[9]));
    const gdn_rows xr = s.rows(&x, {c.d.C}, "x");
    const std::array<int64_t, 2> row{c.d.taps - 1, c.d.C};
    const void* s0 = s.state(state0, row, s.type, true, "state0");
    void* sf = s.state(state_final, row, s.type, true, "state_final");
    if (slots && !state_final) refuse("state_final", "with slots give state_final (it may be state0)");
    gdn_rows yr{};
    if (out) yr = s.out_rows(*out, c.d.C, "out");
    const Span xs = span(xr, s.q.N, 1, c.d.C, x.element_size(), "x"), ws = span(&weight, "weight"), bs = span(bias, "bias"),
               fs = span(state_final, "state_final"), is = span(state0, "state0");
    if (out) apart(span(yr, s.q.N, 1, c.d.C, x.element_size(), "out"), {xs, ws, bs, is, fs});
    if (state_final) apart(fs, {xs, ws, bs}, {is});
    Tensor y, sfo;
    {
      const NoGil nogil;
      const c10::cuda::OptionalCUDAGuard guard(s.dev);
      if (!out) {
        y = fresh(x.sizes(), s.type, s.dev);
        yr = s.rows(&y, {c.d.C}, "out");
        c.d.flags |= GDN_FLAG_ZERO_PADDING;
      }
      if (!state_final) {
        sfo = fresh({s.q.B, row[0], row[1]}, s.type, s.dev);
        sf = sfo.data_ptr();
      }
      check("gdn_causal_conv_fwd", gdn_causal_conv_fwd(&c.d, &s.q, &xr, c.w, c.bias, s0, s.max_q, &yr, sf, stream_of(s.dev)));
    }
    return Py_BuildValue("(NN)", out ? Py_NewRef(a[10]) : wrap(y), state_final ? Py_NewRef(a[4]) : wrap(sfo));
  });
}

// (x, weight, bias, dy, state0, dstate, cu_seqlens, flags, workspace) -> (dx, dweight, dbias, dstate0)
PyObject* causal_conv_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("causal_conv_bwd", a, n, 9, [&]() -> PyObject* {
    const Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight"), &dy = tensor(a[3], "dy");
    const Tensor *bias = optional_tensor(a[2], "bias"), *state0 = optional_tensor(a[4], "state0"),
                 *dstate = optional_tensor(a[5], "dstate"), *given = optional_tensor(a[8], "workspace");
    Seqs s(x, "x", nullptr, optional_tensor(a[6], "cu_seqlens"), nullptr, Py_None);
    Conv c(s, x, weight, bias, integer(a[7]));
    const gdn_rows xr = s.rows(&x, {c.d.C}, "x"), dyr = s.rows(&dy, {c.d.C}, "dy");
    const std::array<int64_t, 2> row{c.d.taps - 1, c.d.C};
    const void *s0 = s.state(state0, row, s.type, false, "state0"), *ds = s.state(dstate, row, s.type, false, "dstate");
    Tensor g[4];
    {
      const NoGil nogil;
      const c10::cuda::OptionalCUDAGuard guard(s.dev);
      const bool none = s.q.N == 0 && s.q.B == 0;  // nothing is launched, and the weights' sums are zero
      g[0] = fresh(x.sizes(), s.type, s.dev);
      g[1] = none ? at::zeros(weight.sizes(), weight.options()) : fresh(weight.sizes(), s.type, s.dev);
      if (bias) g[2] = none ? at::zeros(bias->sizes(), bias->options()) : fresh(bias->sizes(), s.type, s.dev);
      if (state0) g[3] = fresh(state0->sizes(), s.type, s.dev);
      c10::DataPtr ws;
      void* w = scratch(given, gdn_causal_conv_workspace_bytes(&c.d, &s.q), x, &ws);
      check("gdn_causal_conv_bwd",
            gdn_causal_conv_bwd(&c.d, &s.q, &xr, c.w, c.bias, s0, &dyr, ds, g[0].data_ptr(), g[1].data_ptr(),
                                bias ? g[2].data_ptr() : nullptr, state0 ? g[3].data_ptr() : nullptr, w, stream_of(s.dev)));
    }
    PyObject* r = PyTuple_New(4);
    for (int i = 0; r && i < 4; ++i) PyTuple_SET_ITEM(r, i, g[i].defined() ? wrap(g[i]) : Py_NewRef(Py_None));
    return r;
  });
}

// The inputs that the scan's forward and backward share: (u, dt, A, B, C, D, z, dt_bias)
struct Scan {
  gdn_scan_dims d;
  gdn_scan_parts p{};
  const Tensor* part[8];
  Scan(const Seqs& s, PyObject* const* a, long long flags) {
    static const char* const names[8] = {"u", "dt", "A", "B", "C", "D", "z", "dt_bias"};
    for (int i = 0; i < 8; ++i) part[i] = i < 5 ? &tensor(a[i], names[i]) : optional_tensor(a[i], names[i]);
    const Tensor &A = *part[2], &B = *part[3];
    const int64_t D = part[0]->size(-1);
    if (A.dim() != 2) refuse("A", "A must be [channels, states]");
    if (B.dim() != part[0]->dim() + 1) refuse("B", "B and C must be [..., groups, states]");
    d.D = to_int(D, "D");
    d.G = to_int(B.size(-2), "G");
    d.S = to_int(A.size(1), "S");
    d.dtype = dtype_code(*part[0]);
    d.flags = (int)flags;
    p.u = s.rows(part[0], {D}, names[0]);
    p.dt = s.rows(part[1], {D}, names[1]);
    p.A = static_cast<const float*>(exactly(&A, {D, d.S}, at::kFloat, s.dev, names[2]));
    p.B = s.rows(&B, {d.G, d.S}, names[3]);
    p.C = s.rows(part[4], {d.G, d.S}, names[4]);
    p.skip = static_cast<const float*>(exactly(part[5], {D}, at::kFloat, s.dev, names[5]));
    p.z = s.rows(part[6], {D}, names[6]);
    p.dt_bias = static_cast<const float*>(exactly(part[7], {D}, at::kFloat, s.dev, names[7]));
  }
};

// (u, dt, A, B, C, D, z, dt_bias, h0, h_final, slots, cu_seqlens, kv_lens, max_q, flags, save, out, workspace)
// -> (y, h_final, residuals or None)
PyObject* selective_scan_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("selective_scan_fwd", a, n, 18, [&]() -> PyObject* {
    const Tensor& u = tensor(a[0], "u");
    const Tensor *h0 = optional_tensor(a[8], "h0"), *h_final = optional_tensor(a[9], "h_final"),
                 *slots = optional_tensor(a[10], "slots"), *out = optional_tensor(a[16], "out"),
                 *given = optional_tensor(a[17], "workspace");
    Seqs s(u, "u", slots, optional_tensor(a[11], "cu_seqlens"), optional_tensor(a[12], "kv_lens"), a[13]);
    Scan c(s, a, integer(a[14]));
    static const char* const names[8] = {"u", "dt", "A", "B", "C", "D", "z", "dt_bias"};
    for (int i = 0; i < 8; ++i) no_gradient(c.part[i], names[i]);
    no_gradient(h0, "h0"); no_gradient(h_final, "h_final"); no_gradient(out, "out");
    const int save = PyObject_IsTrue(a[15]);
    if (save < 0) return nullptr;
    const std::array<int64_t, 2> row{c.d.D, c.d.S};
    c.p.h0 = static_cast<const float*>(s.state(h0, row, at::kFloat, true, "h0"));
    float* hf = static_cast<float*>(s.state(h_final, row, at::kFloat, true, "h_final"));
    if (slots && !h_final) refuse("h_final", "with slots give h_final (it may be h0)");
    gdn_rows yr{};
    if (out) yr = s.out_rows(*out, c.d.D, "out");
    if (out || h_final) {
      const int64_t es = u.element_size();
      const Span us = span(c.p.u, s.q.N, 1, c.d.D, es, "u"), ds = span(c.p.dt, s.q.N, 1, c.d.D, es, "dt"),
                 zs = span(c.p.z, s.q.N, 1, c.d.D, es, "z"), bs = span(c.p.B, s.q.N, c.d.G, c.d.S, es, "B"),
                 cs = span(c.p.C, s.q.N, c.d.G, c.d.S, es, "C"), as = span(c.part[2], "A"), ss = span(c.part[5], "D"),
                 ts = span(c.part[7], "dt_bias"), fs = span(h_final, "h_final"), is = span(h0, "h0");
      if (out) apart(span(yr, s.q.N, 1, c.d.D, es, "out"), {bs, cs, as, ss, ts, is, fs}, {us, ds, zs});
      if (h_final) apart(fs, {us, ds, zs, bs, cs, as, ss, ts}, {is});
    }
    Tensor y, hfo, kept;
    {
      const NoGil nogil;
      const c10::cuda::OptionalCUDAGuard guard(s.dev);
      if (!out) {
        y = fresh(u.sizes(), s.type, s.dev);
        yr = s.rows(&y, {c.d.D}, "out");
        c.d.flags |= GDN_FLAG_ZERO_PADDING;
      }
      if (!h_final) {
        hfo = fresh({s.q.B, row[0], row[1]}, at::kFloat, s.dev);
        hf = hfo.data_ptr<float>();
      }
      float* rp = nullptr;
      if (save) {
        // an element at least, so that a call without tokens has residuals too
        kept = fresh({(int64_t)std::max<size_t>(gdn_selective_scan_residual_bytes(&c.d, &s.q) / sizeof(float), 4)}, at::kFloat, s.dev);
        rp = kept.data_ptr<float>();
      }
      c10::DataPtr ws;
      const size_t need = gdn_selective_scan_workspace_bytes(&c.d, &s.q, s.max_q);
      void* w = need || given ? scratch(given, need, u, &ws) : nullptr;
      check("gdn_selective_scan_fwd", gdn_selective_scan_fwd(&c.d, &s.q, &c.p, s.max_q, &yr, hf, rp, w, stream_of(s.dev)));
    }
    return Py_BuildValue("(NNN)", out ? Py_NewRef(a[16]) : wrap(y), h_final ? Py_NewRef(a[9]) : wrap(hfo),
                         save ? wrap(kept) : Py_NewRef(Py_None));
  });
}

// (u, dt, A, B, C, D, z, dt_bias, dy, residuals, dh_final, need_dh0, cu_seqlens, max_q, flags, workspace)
// -> (du, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0)
PyObject* selective_scan_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("selective_scan_bwd", a, n, 16, [&]() -> PyObject* {
    const Tensor &u = tensor(a[0], "u"), &dy = tensor(a[8], "dy"), &kept = tensor(a[9], "residuals");
    const Tensor *dh = optional_tensor(a[10], "dh_final"), *given = optional_tensor(a[15], "workspace");
    const int need_dh0 = PyObject_IsTrue(a[11]);
    if (need_dh0 < 0) return nullptr;
    Seqs s(u, "u", nullptr, optional_tensor(a[12], "cu_seqlens"), nullptr, a[13]);
    const Scan c(s, a, integer(a[14]));
    const gdn_rows dyr = s.rows(&dy, {c.d.D}, "dy");
    const std::array<int64_t, 2> row{c.d.D, c.d.S};
    const float* dhp = static_cast<const float*>(s.state(dh, row, at::kFloat, false, "dh_final"));
    const int64_t size = (int64_t)std::max<size_t>(gdn_selective_scan_residual_bytes(&c.d, &s.q) / sizeof(float), 4);
    if (kept.scalar_type() != at::kFloat || kept.sizes() != at::IntArrayRef({size}) || !kept.is_contiguous())
      refuse("residuals", "residuals must be the forward's");
    on_device(kept, s.dev, "residuals");
    Tensor g[9];
    {
      const NoGil nogil;
      const c10::cuda::OptionalCUDAGuard guard(s.dev);
      const bool none = s.q.N == 0 && s.q.B == 0;  // nothing is launched, and the parameters' sums are zero
      for (int i = 0; i < 8; ++i)
        if (c.part[i])
          g[i] = none ? at::zeros(c.part[i]->sizes(), c.part[i]->options())
                      : fresh(c.part[i]->sizes(), c.part[i]->scalar_type(), s.dev);
      if (need_dh0) g[8] = fresh({s.q.B, row[0], row[1]}, at::kFloat, s.dev);
      auto fp = [&](int i) { return g[i].defined() ? g[i].data_ptr<float>() : nullptr; };
      const gdn_scan_grads grads{g[0].data_ptr(), g[1].data_ptr(), g[6].defined() ? g[6].data_ptr() : nullptr, g[3].data_ptr(),
                                 g[4].data_ptr(), fp(2), fp(5), fp(7), fp(8)};
      c10::DataPtr ws;
      void* w = scratch(given, gdn_selective_scan_bwd_workspace_bytes(&c.d, &s.q, s.max_q), u, &ws);
      check("gdn_selective_scan_bwd", gdn_selective_scan_bwd(&c.d, &s.q, &c.p, kept.data_ptr<float>(), s.max_q, &dyr, dhp, &grads,
                                                             w, stream_of(s.dev)));
    }
    PyObject* r = PyTuple_New(9);
    for (int i = 0; r && i < 9; ++i) PyTuple_SET_ITEM(r, i, g[i].defined() ? wrap(g[i]) : Py_NewRef(Py_None));
    return r;
  });
}

// (page_table, kv_lens, new_tokens, free_pages, free_count, page_size, max_tokens)
// -> (cu_seqlens, kv_lens, free_count, requests, positions, slots)
PyObject* page_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("page_plan", a, n, 7, [&]() -> PyObject* {
    const Tensor &table = tensor(a[0], "page_table"), &lens = tensor(a[1], "kv_lens"), &fresh_tokens = tensor(a[2], "new_tokens"),
                 &pages = tensor(a[3], "free_pages"), &count = tensor(a[4], "free_count");
    const c10::Device dev = table.device();
    if (table.dim() != 2) refuse("page_table", "page_table must be [requests, pages per request]");
    if (pages.dim() != 1) refuse("free_pages", "free_pages must be [pages]");
    const int64_t B = table.size(0);
    int_array(table, {B, table.size(1)}, dev, "page_table");
    int_array(lens, {B}, dev, "kv_lens");
    int_array(fresh_tokens, {B}, dev, "new_tokens");
    int_array(pages, {pages.size(0)}, dev, "free_pages");
    int_array(count, {1}, dev, "free_count");
    gdn_plan_dims d;
    d.B = to_int(B, "B");
    d.page_size = to_int(integer(a[5]), "page_size");
    d.max_pages = to_int(table.size(1), "max_pages");
    d.num_free = to_int(pages.size(0), "num_free");
    d.max_tokens = to_int(integer(a[6]), "max_tokens");
    Tensor o[6];
    {
      const NoGil nogil;
      const c10::cuda::OptionalCUDAGuard guard(dev);
      // one allocation for all six, on 16-byte boundaries (six took half of the call's time)
      const int64_t sizes[6] = {d.max_tokens, d.max_tokens, d.max_tokens, B + 1, B, 1};
      int64_t at[7] = {0};
      for (int i = 0; i < 6; ++i) at[i + 1] = at[i] + (sizes[i] * (i ? 4 : 8) + 15) / 16 * 16;
      const Tensor all = fresh({at[6]}, at::kByte, dev);
      for (int i = 0; i < 6; ++i) o[i] = part_of(all, at[i], sizes[i], i ? at::kInt : at::kLong);
      const gdn_plan_out out{o[3].data_ptr<int>(), o[4].data_ptr<int>(), o[5].data_ptr<int>(), o[1].data_ptr<int>(),
                             o[2].data_ptr<int>(), reinterpret_cast<long long*>(o[0].data_ptr<int64_t>())};
      check("gdn_page_plan", gdn_page_plan(&d, table.data_ptr<int>(), B > 1 ? table.stride(0) : table.size(1), lens.data_ptr<int>(),
                                           fresh_tokens.data_ptr<int>(), pages.data_ptr<int>(), count.data_ptr<int>(), &out,
                                           stream_of(dev)));
    }
    std::rotate(o, o + 3, o + 6);  // cu_seqlens, kv_lens, free_count, slots, requests, positions
    std::rotate(o + 3, o + 4, o + 6);
    PyObject* r = PyTuple_New(6);
    for (int i = 0; r && i < 6; ++i) PyTuple_SET_ITEM(r, i, wrap(o[i]));
    return r;
  });
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XSETREF(g_error, Py_NewRef(cls));
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"kv_append", FAST(kv_append), nullptr},
                         {"paged_attn", FAST(paged_attn), nullptr},
                         {"block_norm_fwd", FAST(block_norm_fwd), nullptr},
                         {"block_norm_bwd", FAST(block_norm_bwd), nullptr},
                         {"causal_conv_fwd", FAST(causal_conv_fwd), nullptr},
                         {"causal_conv_bwd", FAST(causal_conv_bwd), nullptr},
                         {"selective_scan_fwd", FAST(selective_scan_fwd), nullptr},
                         {"selective_scan_bwd", FAST(selective_scan_bwd), nullptr},
                         {"page_plan", FAST(page_plan), nullptr},
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdn_ext", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gdn_ext(void) { return PyModule_Create(&module); }
