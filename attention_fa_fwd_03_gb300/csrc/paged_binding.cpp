// Python binding of the paged-cache calls (fa_kv_append, fa_paged_fwd,
// fa_page_select, fa_page_assign) and of differentiable attention: checks the tensors, makes the
// device current and calls the C ABI on the stream. It holds no arithmetic. The other calls go
// through ctypes; these are made once per layer and token, where a kernel takes a few
// microseconds, and ctypes with checks in Python took 8 to 10 of them per call.
#include <climits>
#include <cstdint>
#include <exception>
#include <new>

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fa.h"

#include "autograd_binding.h"

namespace {

const char kCapsule[] = "attention_fa_fwd_03_gb300.PagedKV";

// What a PagedKV object has checked once.
struct Handle {
  fa_paged_kv kv;  // with scales: k_bounds and dt are not used
  float *k_scales, *v_scales;
  int device;
  bool e4m3() const { return k_scales != nullptr; }
  fa_paged_kv8 kv8() const {
    return {kv.k, kv.v, k_scales, v_scales, kv.page_table, kv.kv_lens, kv.B, kv.Hkv, kv.D, kv.num_pages,
            kv.page_size, kv.max_pages};
  }
};

// A Python error is set; carried to the function's end as an exception.
struct Failed {};

[[noreturn]] void fail(PyObject* type, const char* text, const char* name) {
  PyErr_Format(type, text, name);
  throw Failed{};
}

// Type of a call's keys, values, queries and outputs: the cache's, or, where it is held in
// 8 bits, that of `t`.
at::ScalarType call_type(const Handle& h, const at::Tensor& t, const char* name) {
  if (!h.e4m3()) return h.kv.dt == FA_BF16 ? at::kBFloat16 : at::kHalf;
  if (t.scalar_type() != at::kHalf && t.scalar_type() != at::kBFloat16) fail(PyExc_ValueError, "%s: fp16 or bf16", name);
  return t.scalar_type();
}
fa_dtype code_of(at::ScalarType t) { return t == at::kBFloat16 ? FA_BF16 : FA_FP16; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s: expected a tensor", name);
  return THPVariable_Unpack(o);
}

// A tensor of this type and shape on the cache's device.
const at::Tensor& checked(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int device) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type || t.sizes() != shape) fail(PyExc_ValueError, "%s: wrong dtype or shape", name);
  if (!t.is_cuda() || t.get_device() != device) fail(PyExc_ValueError, "%s: not on the cache's device", name);
  return t;
}
void* address(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int device) {
  const at::Tensor& t = checked(o, name, type, shape, device);
  if (!t.is_contiguous()) fail(PyExc_ValueError, "%s: must be contiguous", name);
  return t.data_ptr();
}
int* ints(PyObject* o, const char* name, at::IntArrayRef shape, int device) {
  return o == Py_None ? nullptr : static_cast<int*>(address(o, name, at::kInt, shape, device));
}

// A [B, H, T, D] view whose innermost index is contiguous.
void* view(PyObject* o, const char* name, const Handle& h, at::ScalarType type, at::IntArrayRef shape, int64_t* strides) {
  const at::Tensor& t = checked(o, name, type, shape, h.device);
  if (t.stride(3) != 1) fail(PyExc_ValueError, "%s: the innermost index must be contiguous", name);
  // the stride of an index of size 1 is never used and can be anything
  for (int i = 0; i < 3; ++i) strides[i] = shape[i] > 1 ? t.stride(i) : 0;
  return t.data_ptr();
}

void* workspace(PyObject* o, const char* what, int device, size_t* bytes) {
  if (o == Py_None) fail(PyExc_ValueError, "%s needs a workspace tensor (the library never allocates)", what);
  const at::Tensor& t = tensor(o, "workspace");
  if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous())
    fail(PyExc_ValueError, "%s: not contiguous on the cache's device", "workspace");
  *bytes = t.nbytes();
  return t.data_ptr();
}

int integer(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Failed{};
  if (v < INT_MIN || v > INT_MAX) fail(PyExc_ValueError, "%s: out of range", name);
  return static_cast<int>(v);
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Failed{};
  return v != 0;
}
int dim(int64_t n, const char* name) {
  if (n > INT_MAX) fail(PyExc_ValueError, "%s: too large", name);
  return static_cast<int>(n);
}

cudaStream_t stream_of(PyObject* o, int device) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  PyObject* raw = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
  if (!raw) throw Failed{};
  void* p = PyLong_AsVoidPtr(raw);
  Py_DECREF(raw);
  if (!p && PyErr_Occurred()) throw Failed{};
  return static_cast<cudaStream_t>(p);
}

// Other Python threads run while this lives (nothing of Python is touched then): a
// launch waits where the queue of launches is full, for as long as the GPU takes.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// The cache's device is current while this lives.
struct OnDevice {
  c10::DeviceIndex was;
  bool moved;
  explicit OnDevice(int device) : was(c10::cuda::current_device()), moved(was != device) {
    if (moved) c10::cuda::set_device(static_cast<c10::DeviceIndex>(device));
  }
  ~OnDevice() {
    if (!moved) return;
    try {
      c10::cuda::set_device(was);
    } catch (...) {  // it was current a moment ago; a destructor may not throw
    }
  }
};

const Handle& handle_of(PyObject* o) {
  void* p = PyCapsule_GetPointer(o, kCapsule);
  if (!p) throw Failed{};
  return *static_cast<const Handle*>(p);
}

// Runs `body` (a status) with C++ exceptions turned into Python's.
template <class Body>
PyObject* guarded(Py_ssize_t nargs, Py_ssize_t want, const Body& body) {
  if (nargs != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return PyLong_FromLong(static_cast<long>(body()));
  } catch (const Failed&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// handle(k, v, k_bounds, page_table, kv_lens, B, Hkv, D, num_pages, page_size, max_pages, dt, device[, k_scales,
// v_scales]): addresses (k_bounds 0 for none) and sizes, as the PagedKV class has checked them
PyObject* make_handle(PyObject*, PyObject* args) {
  unsigned long long k, v, kb, table, lens, ks = 0, vs = 0;
  int B, Hkv, D, num_pages, page_size, max_pages, dt, device;
  if (!PyArg_ParseTuple(args, "KKKKKiiiiiiii|KK", &k, &v, &kb, &table, &lens, &B, &Hkv, &D, &num_pages, &page_size,
                        &max_pages, &dt, &device, &ks, &vs))
    return nullptr;
  Handle* h = new (std::nothrow) Handle;
  if (!h) return PyErr_NoMemory();
  h->kv.k = reinterpret_cast<void*>(k);
  h->kv.v = reinterpret_cast<void*>(v);
  h->kv.k_bounds = reinterpret_cast<void*>(kb);
  h->k_scales = reinterpret_cast<float*>(ks);
  h->v_scales = reinterpret_cast<float*>(vs);
  h->kv.page_table = reinterpret_cast<const int*>(table);
  h->kv.kv_lens = reinterpret_cast<const int*>(lens);
  h->kv.B = B;
  h->kv.Hkv = Hkv;
  h->kv.D = D;
  h->kv.num_pages = num_pages;
  h->kv.page_size = page_size;
  h->kv.max_pages = max_pages;
  h->kv.dt = static_cast<fa_dtype>(dt);
  h->device = device;
  PyObject* c = PyCapsule_New(h, kCapsule, [](PyObject* o) {
    delete static_cast<Handle*>(PyCapsule_GetPointer(o, kCapsule));
  });
  if (!c) delete h;
  return c;
}

// kv_append(handle, k, v, cos, sin, interleaved, q, q_out, new_lens, stream)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 10, [&] {
    const Handle& h = handle_of(a[0]);
    const fa_paged_kv& c = h.kv;
    int64_t ks[3], vs[3], qs[3] = {0, 0, 0};
    const at::Tensor& k0 = tensor(a[1], "k");
    const int64_t T = k0.dim() == 4 ? k0.size(2) : 0;
    const at::ScalarType type = call_type(h, k0, "k");
    const void* k = view(a[1], "k", h, type, {c.B, c.Hkv, T, c.D}, ks);
    const void* v = view(a[2], "v", h, type, {c.B, c.Hkv, T, c.D}, vs);
    if ((a[6] == Py_None) != (a[7] == Py_None)) fail(PyExc_ValueError, "%s go together", "q and q_out");
    const void* q = nullptr;
    void* q_out = nullptr;
    int64_t Hq = 0;
    if (a[6] != Py_None) {
      const at::Tensor& q0 = tensor(a[6], "q");
      Hq = q0.dim() == 4 ? q0.size(1) : 0;
      q = view(a[6], "q", h, type, {c.B, Hq, T, c.D}, qs);
      q_out = address(a[7], "q_out", type, {c.B, Hq, T, c.D}, h.device);
    }
    if ((a[3] == Py_None) != (a[4] == Py_None)) fail(PyExc_ValueError, "%s go together", "cos and sin");
    const float *cs = nullptr, *sn = nullptr;
    int64_t positions = 0, half = 0;
    if (a[3] != Py_None) {
      const at::Tensor& c0 = tensor(a[3], "cos");
      if (c0.dim() != 2) fail(PyExc_ValueError, "%s and sin are [positions, rot_dim / 2]", "cos");
      positions = c0.size(0);
      half = c0.size(1);
      cs = static_cast<const float*>(address(a[3], "cos", at::kFloat, {positions, half}, h.device));
      sn = static_cast<const float*>(address(a[4], "sin", at::kFloat, {positions, half}, h.device));
    }
    const bool interleaved = truth(a[5]);
    const int* new_lens = ints(a[8], "new_lens", {c.B}, h.device);
    const cudaStream_t stream = stream_of(a[9], h.device);
    const int n_heads = dim(Hq, "q"), n_tokens = dim(T, "k"), n_pos = dim(positions, "cos"), rot = dim(2 * half, "cos");
    const OnDevice on(h.device);
    const Unlocked unlocked;
    if (h.e4m3()) {
      const fa_paged_kv8 c8 = h.kv8();
      return fa_kv_append8(&c8, k, ks, v, vs, q, qs, q_out, n_heads, n_tokens, new_lens, cs, sn, n_pos, rot, interleaved,
                           code_of(type), stream);
    }
    return fa_kv_append(&c, k, ks, v, vs, q, qs, q_out, n_heads, n_tokens, new_lens, cs, sn, n_pos, rot, interleaved, stream);
  });
}

// paged_fwd(handle, q, o, lse, scale, causal, window, new_lens, sel, sel_lens, workspace, stream[, sinks])
PyObject* paged_fwd(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, nargs == 13 ? 13 : 12, [&] {
    const Handle& h = handle_of(a[0]);
    const fa_paged_kv& c = h.kv;
    size_t ws_bytes = 0;
    void* ws = workspace(a[10], "fa_paged_fwd", h.device, &ws_bytes);
    const at::Tensor& q0 = tensor(a[1], "q");
    const int64_t Hq = q0.dim() == 4 ? q0.size(1) : 0, Tq = q0.dim() == 4 ? q0.size(2) : 0;
    const at::ScalarType type = call_type(h, q0, "q");
    const void* q = address(a[1], "q", type, {c.B, Hq, Tq, c.D}, h.device);
    void* o = address(a[2], "o", type, {c.B, Hq, Tq, c.D}, h.device);
    void* lse = address(a[3], "lse", at::kFloat, {c.B, Hq, Tq}, h.device);
    const double scale = PyFloat_AsDouble(a[4]);
    if (scale == -1.0 && PyErr_Occurred()) throw Failed{};
    const bool causal = truth(a[5]);
    const int window = integer(a[6], "window"), sinks = nargs > 12 ? integer(a[12], "sinks") : 0;
    const int* new_lens = ints(a[7], "new_lens", {c.B}, h.device);
    if ((a[8] == Py_None) != (a[9] == Py_None)) fail(PyExc_ValueError, "%s go together", "sel and sel_lens");
    int64_t n_sel = 0;
    if (a[8] != Py_None) {
      const at::Tensor& s0 = tensor(a[8], "sel");
      n_sel = s0.dim() == 3 ? s0.size(2) : 0;
    }
    const int* sel = ints(a[8], "sel", {c.B, c.Hkv, n_sel}, h.device);
    const int* sel_lens = ints(a[9], "sel_lens", {c.B, c.Hkv}, h.device);
    const cudaStream_t stream = stream_of(a[11], h.device);
    const int n_heads = dim(Hq, "q"), n_tokens = dim(Tq, "q"), n_pages = dim(n_sel, "sel");
    const OnDevice on(h.device);
    const Unlocked unlocked;
    if (h.e4m3()) {
      const fa_paged_kv8 c8 = h.kv8();
      return fa_paged_fwd8(&c8, q, o, static_cast<float*>(lse), n_heads, n_tokens, static_cast<float>(scale), causal, window,
                           sinks, new_lens, sel, sel_lens, n_pages, code_of(type), ws, ws_bytes, stream);
    }
    return fa_paged_fwd_sinks(&c, q, o, static_cast<float*>(lse), n_heads, n_tokens, static_cast<float>(scale), causal, window,
                              sinks, new_lens, sel, sel_lens, n_pages, ws, ws_bytes, stream);
  });
}

// page_select(handle, q, sel, sel_lens, keep_first, keep_last, workspace, stream)
PyObject* page_select(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 8, [&] {
    const Handle& h = handle_of(a[0]);
    const fa_paged_kv& c = h.kv;
    size_t ws_bytes = 0;
    void* ws = workspace(a[6], "fa_page_select", h.device, &ws_bytes);
    const at::Tensor &q0 = tensor(a[1], "q"), &s0 = tensor(a[2], "sel");
    const int64_t Hq = q0.dim() == 4 ? q0.size(1) : 0, n_sel = s0.dim() == 3 ? s0.size(2) : 0;
    if (h.e4m3()) return FA_ERR_INVALID_ARG;  // it keeps no bounds
    const void* q = address(a[1], "q", call_type(h, q0, "q"), {c.B, Hq, 1, c.D}, h.device);
    int* sel = static_cast<int*>(address(a[2], "sel", at::kInt, {c.B, c.Hkv, n_sel}, h.device));
    int* sel_lens = static_cast<int*>(address(a[3], "sel_lens", at::kInt, {c.B, c.Hkv}, h.device));
    const int first = integer(a[4], "keep_first"), last = integer(a[5], "keep_last");
    const cudaStream_t stream = stream_of(a[7], h.device);
    const int n_heads = dim(Hq, "q"), n_pages = dim(n_sel, "sel");
    const OnDevice on(h.device);
    const Unlocked unlocked;
    return fa_page_select(&c, q, n_heads, n_pages, first, last, sel, sel_lens, ws, ws_bytes, stream);
  });
}

// page_assign(page_table, kv_lens, held, free_pages, free_count, page_size, T, new_lens, window, sinks, slots, stream)
PyObject* page_assign(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 12, [&] {
    const at::Tensor &table = tensor(a[0], "page_table"), &pages = tensor(a[3], "free_pages");
    if (table.dim() != 2 || pages.dim() != 1) fail(PyExc_ValueError, "%s [B, max_pages], free_pages [num_pages]", "page_table");
    if (!table.is_cuda()) fail(PyExc_ValueError, "%s: not on a CUDA device", "page_table");
    const int device = table.get_device();
    const int64_t B = table.size(0), max_pages = table.size(1), num_pages = pages.size(0);
    int* t = static_cast<int*>(address(a[0], "page_table", at::kInt, {B, max_pages}, device));
    const int* lens = static_cast<int*>(address(a[1], "kv_lens", at::kInt, {B}, device));
    int* held = static_cast<int*>(address(a[2], "held", at::kInt, {B, 3}, device));
    int* stack = static_cast<int*>(address(a[3], "free_pages", at::kInt, {num_pages}, device));
    int* count = static_cast<int*>(address(a[4], "free_count", at::kInt, {2}, device));
    const int page_size = integer(a[5], "page_size"), T = integer(a[6], "T");
    const int* new_lens = ints(a[7], "new_lens", {B}, device);
    const int window = integer(a[8], "window"), sinks = integer(a[9], "sinks");
    int64_t* slots = a[10] == Py_None ? nullptr : static_cast<int64_t*>(address(a[10], "slots", at::kLong, {B, T}, device));
    const cudaStream_t stream = stream_of(a[11], device);
    const int nb = dim(B, "page_table"), np = dim(num_pages, "free_pages"), mp = dim(max_pages, "page_table");
    const OnDevice on(device);
    const Unlocked unlocked;
    return fa_page_assign(t, lens, held, stack, count, nb, np, page_size, mp, T, new_lens, window, sinks, slots, stream);
  });
}

// attention(q, k, v, scale, causal, window, sinks) -> (o, lse), differentiable
PyObject* dense_attention(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  if (nargs != 7) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
    for (const at::Tensor* t : {&q, &k, &v}) {
      if (!t->is_cuda()) fail(PyExc_ValueError, "%s must live on a CUDA device", "tensors");
      if (!t->is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous (row-major [B, H, T, D])", "tensors");
      if (t->dim() != 4) fail(PyExc_ValueError, "%s are [B, H, T, D]", "q, k and v");
    }
    if (q.scalar_type() != at::kHalf && q.scalar_type() != at::kBFloat16) {
      attention::set_status_error(FA_ERR_UNSUPPORTED_DTYPE, "fa_fwd");
      return nullptr;
    }
    if (k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type() || k.get_device() != q.get_device() ||
        v.get_device() != q.get_device() || k.size(0) != q.size(0) || k.size(3) != q.size(3) || v.sizes() != k.sizes())
      fail(PyExc_ValueError, "%s [B, Hkv, Tkv, D] of one shape, of q's type, device, B and D", "k and v are");
    const double scale = PyFloat_AsDouble(a[3]);
    if (scale == -1.0 && PyErr_Occurred()) throw Failed{};
    const bool causal = truth(a[4]);
    const int window = integer(a[5], "window"), sinks = integer(a[6], "sinks");
    attention::Node::List out;
    {
      const Unlocked unlocked;
      out = attention::Node::apply(q, k, v, scale, causal, static_cast<int64_t>(window), static_cast<int64_t>(sinks));
    }
    PyObject* o = THPVariable_Wrap(out[0]);
    PyObject* lse = o ? THPVariable_Wrap(out[1]) : nullptr;
    PyObject* both = lse ? PyTuple_Pack(2, o, lse) : nullptr;
    Py_XDECREF(o);
    Py_XDECREF(lse);
    return both;
  } catch (const Failed&) {
  } catch (const std::exception&) {  // PyTorch's own and FaError
    torch::translate_exception_to_python(std::current_exception());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyMethodDef kMethods[] = {
    {"handle", make_handle, METH_VARARGS, nullptr},
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_append)), METH_FASTCALL, nullptr},
    {"paged_fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(paged_fwd)), METH_FASTCALL, nullptr},
    {"page_select", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(page_select)), METH_FASTCALL, nullptr},
    {"page_assign", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(page_assign)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(dense_attention)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_paged", "Binding of the paged-cache calls and of differentiable attention.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&kModule); }
