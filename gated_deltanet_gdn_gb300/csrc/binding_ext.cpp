// Compiled argument marshalling of the paged cache and block norm calls: takes the tensors
// apart, checks them, allocates what the caller left out and calls the C ABI on the current
// stream. Nothing is computed here.
//
// A decoding step makes these calls once per layer on a few kilobytes; the ctypes
// marshalling of the same arguments took 30 to 40 us a call (Grace, Python 3.12), several
// times the kernels' own time.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/zeros.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

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

// The paged calls have no backward: a gradient that would be lost without a word is refused.
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

// New memory comes from PyTorch's allocator without its dispatcher, which took a third of a
// short call's host time (one token of attention: 6.5 us, through the dispatcher 9.8).
Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, c10::Device dev) {
  return Tensor(at::detail::empty_cuda(sizes, type, dev, std::nullopt));
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

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XSETREF(g_error, Py_NewRef(cls));
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"kv_append", FAST(kv_append), nullptr},
                         {"paged_attn", FAST(paged_attn), nullptr},
                         {"block_norm_fwd", FAST(block_norm_fwd), nullptr},
                         {"block_norm_bwd", FAST(block_norm_bwd), nullptr},
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdn_ext", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gdn_ext(void) { return PyModule_Create(&module); }
