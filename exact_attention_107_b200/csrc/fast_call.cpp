// fast_call.cpp -- the rotary, paged-cache and score-modified calls without the interpreter.
//
// A call of a small size is bound by the host: the Python marshalling of its tensors (checks,
// allocations, twenty-odd ctypes arguments) takes 17 to 21 us next to 4 to 10 us on the GPU.  These
// functions do the ordinary call in C++: plain tensors of the right types, shapes and layout on the
// current device, launched on its current stream.  Whatever else they are given they hand back
// (NotImplemented), and the Python path, which states the checks and their messages, takes it.
// The C ABI's entry points come as addresses (bind), so that every library in use is reached alike.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fa.h"

namespace {

using at::Tensor;

// The declarations give the types, so that a changed signature does not compile here.
decltype(&fa_rotary) g_rotary;
decltype(&fa_paged_append) g_append;
decltype(&fa_paged_attention) g_decode;
decltype(&fa_paged_workspace_size) g_decode_ws;
decltype(&fa_fwd_mod) g_fwd;
decltype(&fa_bwd_mod) g_bwd;
decltype(&fa_bwd_workspace_size) g_bwd_ws;
decltype(&fa_mask_plan) g_plan;
decltype(&fa_mask_plan_size) g_plan_size;

// A call's tensors, checked as they are taken: `ok` turns false at the first that is not ordinary.
struct Call {
  bool ok = true;
  int device = -1;
  at::ScalarType type = at::kFloat;

  // A plain CUDA tensor, or null for None where that is allowed.
  const Tensor* tensor(PyObject* o, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    if (!THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided) ok = false;
    else if (device < 0) device = t.get_device();
    else if (t.get_device() != device) ok = false;
    return ok ? &t : nullptr;
  }
  // The first 16-bit tensor of four axes sets the element type.
  const Tensor* first(PyObject* o) {
    const Tensor* t = tensor(o);
    if (!t) return nullptr;
    type = t->scalar_type();
    if ((type != at::kBFloat16 && type != at::kHalf) || t->dim() != 4) ok = false;
    return ok ? t : nullptr;
  }
  const Tensor* typed(PyObject* o, at::ScalarType want, int dim, bool optional = false) {
    const Tensor* t = tensor(o, optional);
    if (t && (t->scalar_type() != want || t->dim() != dim || !t->is_contiguous())) ok = false;
    return ok ? t : nullptr;
  }
  bool shape(const Tensor* t, std::initializer_list<int64_t> s) {
    if (!t) return ok;
    int i = 0;
    for (const int64_t n : s)
      if (t->size(i++) != n) ok = false;
    return ok;
  }
  bool flag(PyObject* o) {
    if (o == Py_True) return true;
    if (o != Py_False) ok = false;
    return false;
  }
  double number(PyObject* o) {
    if (PyFloat_CheckExact(o)) return PyFloat_AS_DOUBLE(o);
    if (PyLong_CheckExact(o)) {
      const double v = PyLong_AsDouble(o);
      if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        ok = false;
      }
      return v;
    }
    ok = false;
    return 0.0;
  }
  // A cap: 0, or a number that is none as a float either.
  float cap(PyObject* o) {
    const double v = number(o);
    if (v != 0.0 && static_cast<float>(v) == 0.f) ok = false;
    return static_cast<float>(v);
  }
  int whole(PyObject* o) {
    int over = 0;
    const long v = PyLong_CheckExact(o) ? PyLong_AsLongAndOverflow(o, &over) : -1;
    if (v < 0 || v > INT_MAX || over) ok = false;
    return ok ? static_cast<int>(v) : 0;
  }
  bool here() {
    if (ok && c10::cuda::current_device() != device) ok = false;
    return ok;
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }
  Tensor empty(at::IntArrayRef size, at::ScalarType t) const {
    return at::detail::empty_cuda(size, t, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(device)), std::nullopt);
  }
  int code() const { return type == at::kHalf ? 1 : 0; }
};

const void* ptr(const Tensor* t) { return t ? t->const_data_ptr() : nullptr; }
const int* ints(const Tensor* t) { return static_cast<const int*>(ptr(t)); }
const float* floats(const Tensor* t) { return static_cast<const float*>(ptr(t)); }

// Element strides of batch, head and token; false where the kernel would not read them.
bool strides(const Tensor& t, long long (&s)[3]) {
  for (int i = 0; i < 3; ++i) {
    s[i] = t.size(i) > 1 ? t.stride(i) : 0;
    if (s[i] % 8 != 0 || s[i] < 0) return false;
  }
  return (t.stride(3) == 1 || t.size(3) <= 1) && reinterpret_cast<uintptr_t>(t.const_data_ptr()) % 16 == 0;
}

PyObject* back() { Py_RETURN_NOTIMPLEMENTED; }
PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* tuple(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o = nullptr;
    if (t.defined()) {
      o = wrap(t);
    } else {
      Py_INCREF(Py_None);
      o = Py_None;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// Allocation and launch run without the interpreter's lock, as torch's own calls do: either may wait
// for something that another Python thread has to do.
struct NoLock {
  PyThreadState* state = PyEval_SaveThread();
  ~NoLock() { PyEval_RestoreThread(state); }
};

// Every function: C++ exceptions become Python's, of the types that torch's own calls raise
// (torch.OutOfMemoryError for an allocation that fails).
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guard(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(a, n);
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

// (q | None, k | None, table, positions | None, interleaved, inverse) -> (q, k)
PyObject* rotary(PyObject* const* a, Py_ssize_t n) {
  if (n != 6 || !g_rotary || (a[0] == Py_None && a[1] == Py_None)) return back();
  Call c;
  const Tensor* some = c.first(a[0] != Py_None ? a[0] : a[1]);
  const Tensor *q = a[0] != Py_None ? some : nullptr, *k = a[1] == Py_None ? nullptr : a[0] == Py_None ? some : c.tensor(a[1]);
  const Tensor* table = c.typed(a[2], at::kFloat, 2);
  const Tensor* pos = c.tensor(a[3], true);
  const bool interleaved = c.flag(a[4]), inverse = c.flag(a[5]);
  if (!c.here()) return back();
  const int64_t B = some->size(0), N = some->size(2), D = some->size(3), R = table->size(1);
  long long qs[3] = {}, ks[3] = {};
  if (q && !strides(*q, qs)) return back();
  if (k && (k->scalar_type() != c.type || k->dim() != 4 || !c.shape(k, {B, k->size(1), N, D}) || !strides(*k, ks))) return back();
  if (R < 2 || R > D || R % 2 != 0 || table->size(0) < 1 || table->size(0) > INT_MAX) return back();
  long long stride = 0;
  if (pos) {
    if (pos->scalar_type() != at::kInt || !pos->is_contiguous() || pos->dim() < 1 || pos->dim() > 2 ||
        pos->size(pos->dim() - 1) != N)
      return back();
    if (pos->dim() == 2) {
      if (pos->size(0) != 1 && pos->size(0) != B) return back();
      stride = pos->size(0) > 1 ? N : 0;
    }
  }
  const int64_t H = q ? q->size(1) : 0, Hkv = k ? k->size(1) : 0;
  if (B * N > INT_MAX || H + Hkv > 65535 || B * N * D == 0 || (q && H == 0) || (k && Hkv == 0)) return back();
  Tensor qo, ko;
  const int st = [&] {
    NoLock lock;
    if (q) qo = c.empty({B, H, N, D}, c.type);
    if (k) ko = c.empty({B, Hkv, N, D}, c.type);
    return g_rotary(ptr(q), ptr(k), q ? qo.data_ptr() : nullptr, k ? ko.data_ptr() : nullptr, floats(table),
                          ints(pos), qs, ks, stride, static_cast<int>(table->size(0)), static_cast<int>(B),
                          static_cast<int>(H), static_cast<int>(Hkv), static_cast<int>(N), static_cast<int>(D),
                          static_cast<int>(R), interleaved, inverse, c.code(), c.stream());
  }();
  return st != 0 ? PyLong_FromLong(st) : tuple({qo, ko});
}

// Pools (num_pages, Hkv, page, D), block table (B, width) and lengths (B) of a cache.
struct Cache {
  const Tensor *k, *v, *table, *lens;
  bool take(Call& c, PyObject* const* a) {
    k = c.typed(a[0], c.type, 4);
    v = c.typed(a[1], c.type, 4);
    table = c.typed(a[2], at::kInt, 2);
    lens = c.typed(a[3], at::kInt, 1);
    return c.ok && c.shape(v, {k->size(0), k->size(1), k->size(2), k->size(3)}) && k->size(0) <= INT_MAX &&
           k->size(2) <= INT_MAX && table->size(1) <= INT_MAX;
  }
};

// (k, v, k_pages, v_pages, block_table, seq_lens, new_lens | None, q | None, table | None, interleaved) -> (q | None,)
PyObject* append(PyObject* const* a, Py_ssize_t n) {
  if (n != 10 || !g_append) return back();
  Call c;
  const Tensor *k = c.first(a[0]), *v = c.tensor(a[1]);
  Cache cache;
  if (!c.ok || !cache.take(c, a + 2)) return back();
  const Tensor* fresh = c.typed(a[6], at::kInt, 1, true);
  const Tensor* q = c.tensor(a[7], true);
  const Tensor* table = c.typed(a[8], at::kFloat, 2, true);
  const bool interleaved = c.flag(a[9]);
  if (!c.here()) return back();
  const int64_t B = k->size(0), Hkv = k->size(1), T = k->size(2), D = k->size(3);
  long long ks[3], vs[3], qs[3] = {};
  if (v->scalar_type() != c.type || v->dim() != 4 || !c.shape(v, {B, Hkv, T, D}) || !strides(*k, ks) || !strides(*v, vs)) return back();
  if (cache.k->size(1) != Hkv || cache.k->size(3) != D || !c.shape(cache.lens, {B}) || cache.table->size(0) != B || !c.shape(fresh, {B})) return back();
  int64_t H = 0;
  if (q) {
    H = q->dim() == 4 ? q->size(1) : 0;
    if (H == 0 || q->scalar_type() != c.type || !c.shape(q, {B, H, T, D}) || !strides(*q, qs)) return back();
  }
  const int64_t R = table ? table->size(1) : 0, rows = table ? table->size(0) : 0;
  if (table && (R < 2 || R > D || R % 2 != 0 || rows < 1 || rows > INT_MAX)) return back();
  if (B * T > INT_MAX || H + 2 * Hkv > 65535 || B * T * D * Hkv == 0) return back();
  Tensor qo;
  const int st = [&] {
    NoLock lock;
    if (q) qo = c.empty({B, H, T, D}, c.type);
    return g_append(
      ptr(k), ptr(v), const_cast<void*>(ptr(cache.k)), const_cast<void*>(ptr(cache.v)), ptr(q), q ? qo.data_ptr() : nullptr,
      ints(cache.table), ints(cache.lens), ints(fresh), floats(table), ks, vs, qs, static_cast<int>(rows),
      static_cast<int>(cache.table->size(1)), static_cast<int>(cache.k->size(0)), static_cast<int>(cache.k->size(2)),
      static_cast<int>(B), static_cast<int>(H), static_cast<int>(Hkv), static_cast<int>(T), static_cast<int>(D),
      static_cast<int>(R), interleaved, c.code(), c.stream());
  }();
  return st != 0 ? PyLong_FromLong(st) : tuple({qo});
}

// (q, k_pages, v_pages, block_table, seq_lens, scale, softcap, slopes | None, window) -> (o, lse)
PyObject* decode(PyObject* const* a, Py_ssize_t n) {
  if (n != 9 || !g_decode) return back();
  Call c;
  const Tensor* q = c.first(a[0]);
  Cache cache;
  if (!q || !q->is_contiguous() || !cache.take(c, a + 1)) return back();
  const double scale = c.number(a[5]);
  const float cap = c.cap(a[6]);
  const Tensor* slopes = c.typed(a[7], at::kFloat, 1, true);
  const int window = c.whole(a[8]);
  if (!c.here()) return back();
  const int64_t B = q->size(0), H = q->size(1), T = q->size(2), D = q->size(3), Hkv = cache.k->size(1);
  if (cache.k->size(3) != D || !c.shape(cache.lens, {B}) || cache.table->size(0) != B || !c.shape(slopes, {H})) return back();
  if (B > INT_MAX || H > INT_MAX || T > INT_MAX || Hkv > INT_MAX) return back();
  const int b = static_cast<int>(B), h = static_cast<int>(H), hk = static_cast<int>(Hkv), t = static_cast<int>(T), d = static_cast<int>(D);
  const size_t bytes = g_decode_ws(b, h, hk, t, d);
  if (bytes == 0) return back();
  Tensor o, lse, ws;
  const int st = [&] {
    NoLock lock;
    o = c.empty({B, H, T, D}, c.type), lse = c.empty({B, H, T}, at::kFloat);
    ws = c.empty({static_cast<int64_t>(bytes)}, at::kByte);
    return g_decode(ptr(q), ptr(cache.k), ptr(cache.v), ints(cache.table), ints(cache.lens), o.data_ptr(),
                          static_cast<float*>(lse.data_ptr()), ws.data_ptr(), bytes, floats(slopes),
                          cap, window, static_cast<int>(cache.table->size(1)),
                          static_cast<int>(cache.k->size(0)), static_cast<int>(cache.k->size(2)), b, h, hk, t, d,
                          static_cast<float>(scale), c.code(), c.stream());
  }();
  return st != 0 ? PyLong_FromLong(st) : tuple({o, lse});
}

// q, k, v, plan and slopes of a score-modified call.
struct Mods {
  const Tensor *q, *k, *v, *plan, *slopes;
  int64_t B, H, Hkv, N, D;
  bool take(Call& c, PyObject* const* qkv, PyObject* plan_o, PyObject* slopes_o) {
    q = c.first(qkv[0]);
    k = c.typed(qkv[1], c.type, 4);
    v = c.typed(qkv[2], c.type, 4);
    plan = c.tensor(plan_o, true);
    slopes = c.typed(slopes_o, at::kFloat, 1, true);
    if (!c.ok || !q->is_contiguous()) return false;
    B = q->size(0), H = q->size(1), N = q->size(2), D = q->size(3), Hkv = k->size(1);
    return c.shape(k, {B, Hkv, N, D}) && c.shape(v, {B, Hkv, N, D}) && c.shape(slopes, {H}) && B > 0 && H > 0 && N > 0 &&
           Hkv > 0 && B * H <= INT_MAX && N <= INT_MAX;
  }
};

// (q, k, v, plan | None, slopes | None, softcap, scale, causal) -> (o, lse); the plan is the mask's, of q's B and N
PyObject* forward(PyObject* const* a, Py_ssize_t n) {
  if (n != 8 || !g_fwd) return back();
  Call c;
  Mods m;
  if (!m.take(c, a, a[3], a[4])) return back();
  const float cap = c.cap(a[5]);
  const double scale = c.number(a[6]);
  const bool causal = c.flag(a[7]);
  if (!c.here() || (causal && m.plan)) return back();
  Tensor o, lse;
  const int st = [&] {
    NoLock lock;
    o = c.empty({m.B, m.H, m.N, m.D}, c.type), lse = c.empty({m.B, m.H, m.N}, at::kFloat);
    return g_fwd(ptr(m.q), ptr(m.k), ptr(m.v), o.data_ptr(), static_cast<float*>(lse.data_ptr()), ptr(m.plan),
                       floats(m.slopes), cap, static_cast<int>(m.B), static_cast<int>(m.H),
                       static_cast<int>(m.Hkv), static_cast<int>(m.N), static_cast<int>(m.D),
                       static_cast<float>(scale), causal, c.code(), c.stream());
  }();
  return st != 0 ? PyLong_FromLong(st) : tuple({o, lse});
}

// (q, k, v, plan | None, slopes | None, softcap, scale, causal, o, lse, do) -> (dq, dk, dv)
PyObject* backward(PyObject* const* a, Py_ssize_t n) {
  if (n != 11 || !g_bwd) return back();
  Call c;
  Mods m;
  if (!m.take(c, a, a[3], a[4])) return back();
  const float cap = c.cap(a[5]);
  const double scale = c.number(a[6]);
  const bool causal = c.flag(a[7]);
  const Tensor *o = c.typed(a[8], c.type, 4), *lse = c.typed(a[9], at::kFloat, 3), *dO = c.typed(a[10], c.type, 4);
  if (!c.here() || (causal && m.plan)) return back();
  if (!c.shape(o, {m.B, m.H, m.N, m.D}) || !c.shape(dO, {m.B, m.H, m.N, m.D}) || !c.shape(lse, {m.B, m.H, m.N})) return back();
  const int B = static_cast<int>(m.B), H = static_cast<int>(m.H), N = static_cast<int>(m.N), D = static_cast<int>(m.D);
  const size_t bytes = g_bwd_ws(B, H, N, D);
  if (bytes == 0) return back();
  Tensor dq, dk, dv, ws;
  const int st = [&] {
    NoLock lock;
    dq = c.empty({m.B, m.H, m.N, m.D}, c.type), dk = c.empty({m.B, m.Hkv, m.N, m.D}, c.type);
    dv = c.empty({m.B, m.Hkv, m.N, m.D}, c.type), ws = c.empty({static_cast<int64_t>(bytes)}, at::kByte);
    return g_bwd(ptr(m.q), ptr(m.k), ptr(m.v), ptr(o), ptr(dO), floats(lse), dq.data_ptr(), dk.data_ptr(),
                       dv.data_ptr(), ws.data_ptr(), bytes, ptr(m.plan), floats(m.slopes), cap, B, H,
                       static_cast<int>(m.Hkv), N, D, static_cast<float>(scale), causal, c.code(), c.stream());
  }();
  return st != 0 ? PyLong_FromLong(st) : tuple({dq, dk, dv});
}

// (documents | None, prefix | None, B, N, causal, window, device index) -> (plan,)
PyObject* mask_plan(PyObject* const* a, Py_ssize_t n) {
  if (n != 7 || !g_plan) return back();
  Call c;
  const int B = c.whole(a[2]), N = c.whole(a[3]), window = c.whole(a[5]), device = c.whole(a[6]);
  const bool causal = c.flag(a[4]);
  c.device = device;
  const Tensor* documents = c.typed(a[0], at::kInt, 2, true);
  const Tensor* prefix = c.typed(a[1], at::kInt, 1, true);
  if (!c.here() || !c.shape(documents, {B, N}) || !c.shape(prefix, {B})) return back();
  const size_t bytes = g_plan_size(B, N);
  if (bytes == 0) return back();
  Tensor plan;
  const int st = [&] {
    NoLock lock;
    plan = c.empty({static_cast<int64_t>(bytes)}, at::kByte);
    return g_plan(plan.data_ptr(), bytes, ints(documents), ints(prefix), B, N, causal, window, c.stream());
  }();
  return st != 0 ? PyLong_FromLong(st) : tuple({plan});
}

// bind(addresses of fa_rotary, fa_paged_append, fa_paged_attention, fa_paged_workspace_size, fa_fwd_mod, fa_bwd_mod,
// fa_bwd_workspace_size, fa_mask_plan, fa_mask_plan_size)
PyObject* bind(PyObject* const* a, Py_ssize_t n) {
  void* at[9];
  if (n != 9) {
    PyErr_SetString(PyExc_TypeError, "bind takes nine addresses");
    return nullptr;
  }
  for (int i = 0; i < 9; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i]);
    if (!at[i]) return PyErr_Occurred() ? nullptr : (PyErr_SetString(PyExc_ValueError, "null address"), nullptr);
  }
  g_rotary = reinterpret_cast<decltype(g_rotary)>(at[0]);
  g_append = reinterpret_cast<decltype(g_append)>(at[1]);
  g_decode = reinterpret_cast<decltype(g_decode)>(at[2]);
  g_decode_ws = reinterpret_cast<decltype(g_decode_ws)>(at[3]);
  g_fwd = reinterpret_cast<decltype(g_fwd)>(at[4]);
  g_bwd = reinterpret_cast<decltype(g_bwd)>(at[5]);
  g_bwd_ws = reinterpret_cast<decltype(g_bwd_ws)>(at[6]);
  g_plan = reinterpret_cast<decltype(g_plan)>(at[7]);
  g_plan_size = reinterpret_cast<decltype(g_plan_size)>(at[8]);
  Py_RETURN_NONE;
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guard<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(rotary), ENTRY(append), ENTRY(decode), ENTRY(forward), ENTRY(backward),
                         ENTRY(mask_plan), ENTRY(bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast() { return PyModule_Create(&module); }
