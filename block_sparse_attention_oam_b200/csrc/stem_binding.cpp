// Python entries of the operators that run once per layer and token (stem_decode, stem_evict).
//
// A call of one short sequence takes the GPU a few microseconds; the same checks of a dozen
// tensors in Python, and ctypes, take 8 to 12.  Here they take under one.  Each function gets
// the address of libstem's entry point, the problem as a buffer (stem_decode_t, stem_evict_t)
// and the tensors; it returns the entry point's status, or -1 where a tensor has another type,
// shape, device or layout than it must (the caller says which).
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <exception>
#include <initializer_list>

#include "stem.h"

namespace {

constexpr long kMisfit = -1;

struct Misfit {};

// Takes the arguments one by one; `next` members throw Misfit.
struct Args {
  PyObject* const* v;
  int device = -1;

  const at::Tensor& raw() {
    PyObject* o = *v++;
    if (!THPVariable_Check(o)) throw Misfit{};
    return THPVariable_Unpack(o);
  }
  static bool has(const at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape) {
    return t.scalar_type() == type && t.is_contiguous() && t.sizes() == at::IntArrayRef(shape);
  }
  void* fit(const at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape) {
    if (!t.is_cuda() || t.get_device() != device || !has(t, type, shape)) throw Misfit{};
    return t.data_ptr();
  }
  template <typename T>
  T* dense(at::ScalarType type, std::initializer_list<int64_t> shape) {
    return static_cast<T*>(fit(raw(), type, shape));
  }
  template <typename T>
  T* dense_or_null(at::ScalarType type, std::initializer_list<int64_t> shape) {
    if (*v == Py_None) {
      ++v;
      return nullptr;
    }
    return dense<T>(type, shape);
  }
  // [seqs, heads, any stride]
  float* weights(int64_t seqs, int64_t heads, int64_t* stride) {
    if (*v == Py_None) {
      ++v;
      return nullptr;
    }
    const at::Tensor& t = raw();
    if (t.dim() != 3) throw Misfit{};
    if (*stride < 0) *stride = t.size(2);
    return static_cast<float*>(fit(t, at::kFloat, {seqs, heads, *stride}));
  }
  stem_paged_kv_t pages(at::ScalarType type, int64_t seqs, int64_t heads, int64_t d) {
    const at::Tensor &k = raw(), &w = raw(), &table = raw();
    if (k.dim() != 4 || table.dim() != 2 || k.size(0) > INT32_MAX || table.size(1) > INT32_MAX) throw Misfit{};
    stem_paged_kv_t c{};
    c.k_cache = fit(k, type, {k.size(0), STEM_PAGE_SIZE, heads, d});
    c.v_cache = fit(w, type, {k.size(0), STEM_PAGE_SIZE, heads, d});
    c.block_table = static_cast<const int32_t*>(fit(table, at::kInt, {seqs, table.size(1)}));
    c.page_size = STEM_PAGE_SIZE;
    c.max_pages_per_seq = static_cast<int>(table.size(1));
    c.num_slots = static_cast<int>(k.size(0));
    return c;
  }
  void* workspace(size_t* bytes) {
    const at::Tensor& t = raw();
    *bytes = static_cast<size_t>(t.numel());
    return fit(t, at::kByte, {t.numel()});
  }
  // None: the device's current stream; else its handle.
  void* stream() {
    PyObject* o = *v++;
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
    void* handle = PyLong_AsVoidPtr(o);
    if (handle == nullptr && PyErr_Occurred()) throw Misfit{};
    return handle;
  }
};

at::ScalarType cache_type(stem_dtype_t t) { return t == STEM_DT_FP8_E4M3 ? at::kFloat8_e4m3fn : at::kBFloat16; }

// f(entry, problem, args) with the problem's bytes held, exceptions turned into Python's.
template <typename Problem, typename F>
PyObject* call(PyObject* const* argv, Py_ssize_t argc, Py_ssize_t want, F f) {
  if (argc != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, argc);
    return nullptr;
  }
  void* entry = PyLong_AsVoidPtr(argv[0]);
  if (entry == nullptr) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "entry point is NULL");
    return nullptr;
  }
  Py_buffer view;
  if (PyObject_GetBuffer(argv[1], &view, PyBUF_SIMPLE) != 0) return nullptr;
  long status = kMisfit;
  bool failed = false;
  if (view.len != static_cast<Py_ssize_t>(sizeof(Problem))) {
    PyErr_SetString(PyExc_ValueError, "the problem has another size");
    failed = true;
  } else {
    try {
      Args a{argv + 2};
      status = f(entry, static_cast<const Problem*>(view.buf), a);
    } catch (const Misfit&) {
    } catch (const std::exception& e) {
      PyErr_SetString(PyExc_RuntimeError, e.what());
      failed = true;
    }
  }
  PyBuffer_Release(&view);
  return failed || PyErr_Occurred() ? nullptr : PyLong_FromLong(status);
}

// (entry, problem, q, k_cache, v_cache, block_table, kv_lens, prefix_table, weights_in,
//  weights_out, out, lse, ws, stream)
PyObject* decode(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return call<stem_decode_t>(argv, argc, 14, [](void* entry, const stem_decode_t* p, Args& a) -> long {
    const at::ScalarType type = cache_type(p->dtype);
    const int64_t B = p->num_seqs, T = B * p->q_len, Hq = p->num_q_heads, Hkv = p->num_kv_heads, d = p->head_dim;
    const at::Tensor& q = a.raw();
    a.device = q.is_cuda() ? q.get_device() : -1;
    const void* qp = a.fit(q, type, {T, Hq, d});
    const stem_paged_kv_t cache = a.pages(type, B, Hkv, d);
    const int32_t* lens = a.dense<int32_t>(at::kInt, {B});
    const int32_t* prefix = a.dense_or_null<int32_t>(at::kInt, {(p->prefix_len + STEM_PAGE_SIZE - 1) / STEM_PAGE_SIZE});
    int64_t stride = -1;
    const float* w_in = a.weights(B, Hkv, &stride);
    float* w_out = a.weights(B, Hkv, &stride);
    void* out = a.dense<void>(at::kBFloat16, {T, Hq, d});
    float* lse = a.dense_or_null<float>(at::kFloat, {Hq, T});
    size_t bytes = 0;
    void* ws = a.workspace(&bytes);
    void* stream = a.stream();
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(a.device));
    long status;
    Py_BEGIN_ALLOW_THREADS;
    status = reinterpret_cast<decltype(&stem_decode)>(entry)(p, qp, &cache, lens, prefix, w_in, w_out,
                                                             stride < 0 ? 0 : stride, out, lse, ws, bytes, stream);
    Py_END_ALLOW_THREADS;
    return status;
  });
}

// (entry, problem, weights, k_cache, v_cache, block_table of src, the same of dst, kv_lens,
//  kv_lens_out, weights_out, keep, ws, stream)
PyObject* evict(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  return call<stem_evict_t>(argv, argc, 15, [](void* entry, const stem_evict_t* p, Args& a) -> long {
    const at::ScalarType type = cache_type(p->dtype);
    const int64_t B = p->num_seqs, Hkv = p->num_kv_heads, d = p->head_dim;
    const at::Tensor& w = a.raw();
    a.device = w.is_cuda() ? w.get_device() : -1;
    if (w.dim() != 3) throw Misfit{};
    const int64_t stride = w.size(2);
    const float* weights = static_cast<const float*>(a.fit(w, at::kFloat, {B, Hkv, stride}));
    const stem_paged_kv_t src = a.pages(type, B, Hkv, d), dst = a.pages(type, B, Hkv, d);
    const int32_t* lens = a.dense<int32_t>(at::kInt, {B});
    int32_t* lens_out = a.dense<int32_t>(at::kInt, {B});
    int64_t out_stride = -1;
    float* w_out = a.weights(B, Hkv, &out_stride);
    int32_t* keep = a.dense<int32_t>(at::kInt, {B, Hkv, p->budget});
    size_t bytes = 0;
    void* ws = a.workspace(&bytes);
    void* stream = a.stream();
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(a.device));
    long status;
    Py_BEGIN_ALLOW_THREADS;
    status = reinterpret_cast<decltype(&stem_evict)>(entry)(p, &src, lens, weights, stride, &dst, lens_out, w_out,
                                                            out_stride < 0 ? 0 : out_stride, keep, ws, bytes, stream);
    Py_END_ALLOW_THREADS;
    return status;
  });
}

PyMethodDef kMethods[] = {
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(decode)), METH_FASTCALL,
     "stem_decode on checked tensors: its status, or -1."},
    {"evict", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(evict)), METH_FASTCALL,
     "stem_evict on checked tensors: its status, or -1."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "stem_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// What this was built against, looked for in the file before it is loaded.
extern "C" __attribute__((used, visibility("default"))) const char stem_binding_tag[] = STEM_BINDING_TAG;

PyMODINIT_FUNC PyInit_stem_binding() { return PyModule_Create(&kModule); }
