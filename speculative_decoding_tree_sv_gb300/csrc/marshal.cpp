// Argument marshalling of the cache operators' Python calls: checks the tensors
// and hands their addresses to the C entry points of include/sv.h.
//
// An append of one token is about 5 us of GPU time; checked and marshalled in
// Python its call took 10.7 us of host time (a page release 6.3), so these six
// calls do it here.  The module sees tensors through torch's own Python object
// and computes nothing.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "../../include/sv.h"

namespace {

using at::Tensor;

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

[[noreturn]] void refuse(const std::string& why) { throw Refused(why); }

std::string shape_of(const Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

// The arguments of one call, in order.
struct Args {
  PyObject* const* at;
  Py_ssize_t n;
  long device;  // the current one; below 0: CUDA is not initialised

  const Tensor* tensor(int i, const char* name, bool optional = false) const {
    if (optional && at[i] == Py_None) return nullptr;
    if (!THPVariable_Check(at[i])) refuse(std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(at[i]);
  }
  long number(int i) const {
    const long v = PyLong_AsLong(at[i]);
    if (v == -1 && PyErr_Occurred()) throw std::exception();
    return v;
  }
  void* pointer(int i) const {
    void* v = PyLong_AsVoidPtr(at[i]);
    if (v == nullptr && PyErr_Occurred()) throw std::exception();
    return v;
  }
  // int32, contiguous, of `count` elements (any if below 0).
  const Tensor* ints(int i, const char* name, int64_t count = -1) const {
    const Tensor* t = tensor(i, name);
    if (t->scalar_type() != at::kInt || !t->is_contiguous())
      refuse(std::string(name) + " must be a contiguous int32 tensor");
    if (count >= 0 && t->numel() != count)
      refuse(std::string(name) + " must have " + std::to_string(count) + " elements, got " +
             std::to_string(t->numel()));
    return t;
  }
  void on_device(std::initializer_list<const Tensor*> tensors) const {
    for (const Tensor* t : tensors) {
      if (t == nullptr) continue;
      if (!t->is_cuda()) refuse("the library takes device memory; got a tensor on " + t->device().str());
      if (t->get_device() != device)
        refuse("got a tensor on " + t->device().str() + ", the current device is cuda:" + std::to_string(device));
    }
  }
};

int* data(const Tensor* t) { return t ? static_cast<int*>(t->data_ptr()) : nullptr; }
void* bytes(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
size_t size(const Tensor* t) { return t ? t->nbytes() : 0; }

int small(int64_t v, const char* name) {
  if (v < 0 || v > 0x7fffffff) refuse(std::string(name) + " does not fit 32 bits");
  return static_cast<int>(v);
}

struct Pool {
  int layers, pages, heads, page, dim;
  int64_t stride;  // elements from a layer to the next
};

// A cache [layers, pages, Hkv, page, D], or one layer of it without the first.
Pool pool(const Tensor& k, const Tensor* v) {
  const int64_t d = k.dim();
  if ((d != 4 && d != 5) || k.element_size() != 2)
    refuse("a cache is [layers, pages, Hkv, page_size, D] or [pages, Hkv, page_size, D] of 16-bit elements");
  if (!k.is_contiguous() && !(d == 5 && k.size(0) > 0 && k.select(0, 0).is_contiguous()))
    refuse("a layer of the cache must be contiguous");
  if (v != nullptr && (v->sizes() != k.sizes() || v->scalar_type() != k.scalar_type() || v->strides() != k.strides()))
    refuse("k_cache and v_cache must have the same shape, type and strides");
  if (d == 5 && k.size(0) > 1 && k.stride(0) < k.select(0, 0).numel()) refuse("the layers of the cache overlap");
  const int64_t o = d - 4;
  return {d == 5 ? small(k.size(0), "layers") : 1, small(k.size(o), "pages"), small(k.size(o + 1), "heads"),
          small(k.size(o + 2), "page size"), small(k.size(o + 3), "head dim"),
          d == 5 && k.size(0) > 1 ? k.stride(0) : 0};
}

struct State {
  const Tensor *table, *held, *refs;
  int rows, width, pages;
};

State state(const Args& a, int table, int held, int refs) {
  State s;
  s.table = a.ints(table, "block_table");
  if (s.table->dim() != 2) refuse("block_table must be [rows, max_pages]");
  s.held = a.ints(held, "held_pages", s.table->size(0));
  s.refs = a.ints(refs, "page_refs");
  s.rows = small(s.table->size(0), "rows");
  s.width = small(s.table->size(1), "max_pages");
  s.pages = small(s.refs->numel(), "pages");
  return s;
}

struct Pairs {
  const Tensor *src, *dst, *count;
  int most;
};

Pairs pairs(const Args& a, int src, int dst, int count, int64_t room) {
  Pairs p{a.ints(src, "copy_src"), a.ints(dst, "copy_dst"), a.ints(count, "copy_count", 1), 0};
  p.most = small(std::min(p.src->numel(), p.dst->numel()), "copies");
  if (p.most < room) refuse("copy_src and copy_dst need room for " + std::to_string(room) + " entries");
  return p;
}

sv_stream_t stream(const Args& a, int i) { return static_cast<sv_stream_t>(a.pointer(i)); }

// Every function takes its tensors, then (page_size,) workspace, device, stream.

sv_status kv_append(const Args& a) {
  const Tensor &k = *a.tensor(0, "k"), &v = *a.tensor(1, "v"), &kc = *a.tensor(2, "k_cache"), &vc = *a.tensor(3, "v_cache");
  const Pool p = pool(kc, &vc);
  if (k.dim() != kc.dim() - 1 || v.sizes() != k.sizes() || v.strides() != k.strides())
    refuse("k and v must have the cache's layers and the same shape and strides");
  if (k.scalar_type() != kc.scalar_type() || v.scalar_type() != kc.scalar_type())
    refuse(std::string("k and v must have the cache's type ") + c10::toString(kc.scalar_type()));
  const int64_t T = k.size(-3);
  if (k.size(-2) != p.heads || k.size(-1) != p.dim || (k.dim() == 4 && k.size(0) != p.layers))
    refuse("k must be [" + std::to_string(p.layers) + " layers, tokens, " + std::to_string(p.heads) + ", " +
           std::to_string(p.dim) + "], got " + shape_of(k));
  if ((p.dim > 1 && k.stride(-1) != 1) || (p.heads > 1 && k.stride(-2) != p.dim))
    refuse("the heads of k and v must be contiguous");
  const Tensor* table = a.ints(4, "block_table");
  if (table->dim() != 2) refuse("block_table must be [batch, max_pages]");
  const int64_t B = table->size(0);
  const Tensor *ctx = a.ints(5, "ctx_lens", B), *cu = a.ints(6, "cu_tokens", B + 1);
  const Tensor* after = a.at[7] == Py_None ? nullptr : a.ints(7, "new_ctx_lens", B);
  const Tensor* ws = a.tensor(8, "workspace", true);
  a.on_device({&k, &v, &kc, &vc, table, ctx, cu, after, ws});
  return sv_kv_append(k.data_ptr(), v.data_ptr(), T > 1 ? k.stride(-3) : static_cast<int64_t>(p.heads) * p.dim,
                      p.layers > 1 ? k.stride(0) : 0, kc.data_ptr(), vc.data_ptr(), p.stride, p.layers, p.pages,
                      data(table), small(table->size(1), "max_pages"), data(ctx), data(cu), small(B, "batch"),
                      small(T, "tokens"), p.heads, p.dim, p.page, data(after), bytes(ws), size(ws), stream(a, 10));
}

sv_status pages_release(const Args& a) {
  const State s = state(a, 1, 2, 3);
  const Tensor *keep = a.ints(0, "keep_lens", s.rows), *ws = a.tensor(5, "workspace", true);
  a.on_device({keep, s.table, s.held, s.refs, ws});
  return sv_pages_release(data(keep), s.rows, data(s.table), s.width, data(s.held), data(s.refs), s.pages,
                          small(a.number(4), "page_size"), bytes(ws), size(ws), stream(a, 7));
}

sv_status pages_fork(const Args& a) {
  const State s = state(a, 2, 4, 5);
  const Tensor* parents = a.ints(0, "parents");
  const Tensor *children = a.ints(1, "children", parents->numel()), *ctx = a.ints(3, "ctx_lens", s.rows);
  const Tensor* ws = a.tensor(7, "workspace", true);
  a.on_device({parents, children, s.table, ctx, s.held, s.refs, ws});
  if (parents->numel() == 0) return SV_OK;
  return sv_pages_fork(data(parents), data(children), small(parents->numel(), "pairs"), data(s.table), s.rows, s.width,
                       data(ctx), data(s.held), data(s.refs), s.pages, small(a.number(6), "page_size"), bytes(ws),
                       size(ws), stream(a, 9));
}

sv_status pages_reserve(const Args& a) {
  const State s = state(a, 2, 3, 4);
  const Tensor *ctx = a.ints(0, "ctx_lens", s.rows), *after = a.ints(1, "new_lens", s.rows);
  const Pairs c = pairs(a, 5, 6, 7, s.rows);
  const Tensor* ws = a.tensor(9, "workspace", true);
  a.on_device({ctx, after, s.table, s.held, s.refs, c.src, c.dst, c.count, ws});
  return sv_pages_reserve(data(ctx), data(after), s.rows, data(s.table), s.width, data(s.held), data(s.refs), s.pages,
                          small(a.number(8), "page_size"), data(c.src), data(c.dst), data(c.count), bytes(ws),
                          size(ws), stream(a, 11));
}

sv_status pages_compact(const Args& a) {
  const State s = state(a, 0, 1, 2);
  const Tensor* table = a.ints(3, "block_table_out", s.table->numel());
  const Tensor* refs = a.ints(4, "page_refs_out", s.pages);
  const Pairs c = pairs(a, 5, 6, 7, std::max(s.pages / 2, 1));
  const Tensor *live = a.ints(8, "num_live", 1), *ws = a.tensor(9, "workspace", true);
  a.on_device({s.table, s.held, s.refs, table, refs, c.src, c.dst, c.count, live, ws});
  return sv_pages_compact(data(s.table), data(s.held), s.rows, s.width, data(s.refs), s.pages, data(table), data(refs),
                          data(c.src), data(c.dst), data(c.count), data(live), bytes(ws), size(ws), stream(a, 11));
}

sv_status pages_copy(const Args& a) {
  const Tensor &kc = *a.tensor(0, "k_cache"), *vc = a.tensor(1, "v_cache", true);
  const Pool p = pool(kc, vc);
  const Pairs c = pairs(a, 2, 3, 4, 0);
  const Tensor* ws = a.tensor(5, "workspace", true);
  a.on_device({&kc, vc, c.src, c.dst, c.count, ws});
  return sv_pages_copy(kc.data_ptr(), bytes(vc), p.stride, p.layers, p.pages,
                       small(static_cast<int64_t>(p.heads) * p.page * p.dim, "page"), data(c.src), data(c.dst),
                       data(c.count), c.most, bytes(ws), size(ws), stream(a, 7));
}

// The Python side of one function of N arguments, `device` the one before the last.
template <sv_status (*F)(const Args&), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    if (n != N) refuse("expected " + std::to_string(N) + " arguments, got " + std::to_string(n));
    Args a{args, n, 0};
    a.device = a.number(N - 2);
    return PyLong_FromLong(F(a));
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <sv_status (*F)(const Args&), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&call<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<kv_append, 11>("kv_append"),
                         method<pages_release, 8>("pages_release"),
                         method<pages_fork, 10>("pages_fork"),
                         method<pages_reserve, 12>("pages_reserve"),
                         method<pages_compact, 12>("pages_compact"),
                         method<pages_copy, 8>("pages_copy"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
