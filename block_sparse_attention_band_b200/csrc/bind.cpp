// Marshalling of the paged cache's three calls from PyTorch tensors to the C
// ABI.  A decode step is these calls in a row, each a few microseconds of GPU
// work: checking ten tensors from Python took 3 to 7 microseconds a call, more
// than the launch itself; here it takes a fraction of one.
//
// Each call gets the config's address, its tensors (or raw integer addresses,
// or None for NULL) and the stream (an integer, or None for the current one of
// the tensors' device).  All tensors have to be on one device, the current one:
// the library launches there.
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <stdexcept>
#include <string>

#include "../../include/prism.h"

namespace {

decltype(&prism_cache_plan) g_plan;
decltype(&prism_cache_store) g_store;
decltype(&prism_cache_attn) g_attn;

// A refused argument: becomes Python's ValueError.
struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

struct Call {
  const char* where;
  int dev = -1;

  [[noreturn]] void refuse(const std::string& what) const { throw Refused(std::string(where) + ": " + what); }

  void on(const at::Tensor& t) {
    if (!t.is_cuda()) throw Refused("tensor arguments must be CUDA tensors (the library takes device pointers)");
    const int d = t.get_device();
    if (d == dev) return;
    if (dev >= 0) refuse("tensors on cuda:" + std::to_string(dev) + " and cuda:" + std::to_string(d));
    const int now = c10::cuda::current_device();
    if (d != now) refuse("tensors on cuda:" + std::to_string(d) + ", the current device is cuda:" + std::to_string(now));
    dev = d;
  }
  static std::string told(const at::Tensor& t) {
    std::ostringstream s;
    s << ", got " << t.scalar_type() << " " << t.sizes() << " strides " << t.strides();
    return s.str();
  }
  // The tensor of an argument, or null for an address or None, put into *addr.
  const at::Tensor* tensor(const char* name, PyObject* x, void** addr) const {
    *addr = nullptr;
    if (x == Py_None) return nullptr;
    if (PyLong_Check(x)) {
      *addr = PyLong_AsVoidPtr(x);
      if (PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(name) + " is no address");
      }
      return nullptr;
    }
    if (!THPVariable_Check(x)) refuse(std::string(name) + " has to be a tensor, an address or None");
    return &THPVariable_Unpack(x);
  }
  // Address of a contiguous tensor of at least (or exactly) numel entries, whose
  // last dims, where it has more than one, are `inner`'s last.
  template <class T>
  T* flat(const char* name, PyObject* x, at::ScalarType type, int64_t numel, bool exact = false,
          std::initializer_list<int64_t> inner = {}) {
    void* addr;
    if (const at::Tensor* t = tensor(name, x, &addr)) {
      if (t->scalar_type() != type || (exact ? t->numel() != numel : t->numel() < numel)) {
        std::ostringstream s;
        s << name << " has to be " << type << " of " << numel << " entries" << told(*t);
        refuse(s.str());
      }
      for (int64_t i = 1, n = (int64_t)inner.size(); i <= n && i < t->dim(); ++i)
        if (t->size(-i) != inner.begin()[n - i]) {
          std::ostringstream s;
          s << name << " has to have rows of " << at::IntArrayRef(inner.begin(), inner.size()) << told(*t);
          refuse(s.str());
        }
      on(*t);
      if (!t->is_contiguous()) throw Refused("tensor arguments must be contiguous");
      addr = t->data_ptr();
    }
    return static_cast<T*>(addr);
  }
  // A bf16 [tokens, heads, 128] view whose last dim is contiguous.  To the library
  // two strides of 0 mean packed rows, so a view of one row for all tokens and
  // heads is refused, and a dim of one entry gets the packed stride.
  void* rows(const char* name, PyObject* x, int64_t tokens, int64_t heads, long long* tok, long long* head) {
    void* addr;
    *tok = *head = 0;
    if (const at::Tensor* t = tensor(name, x, &addr)) {
      on(*t);
      if (t->scalar_type() != at::kBFloat16 || t->dim() != 3 || t->size(0) != tokens || t->size(1) != heads ||
          t->size(2) != 128 || t->stride(2) != 1) {
        std::ostringstream s;
        s << name << " has to be bfloat16 [" << tokens << ", " << heads << ", 128] with a contiguous last dim" << told(*t);
        refuse(s.str());
      }
      *tok = tokens > 1 ? t->stride(0) : heads * 128;
      *head = heads > 1 ? t->stride(1) : 128;
      if (*tok == 0 && *head == 0) refuse(std::string(name) + " is one row for all tokens and heads" + told(*t));
      addr = t->data_ptr();
    }
    return addr;
  }
  // One-byte codes [num_pages, hkv, page, 128] whose pages lie page_stride apart.
  void* pages(const char* name, PyObject* x, const prism_cache_config& c) {
    void* addr;
    if (const at::Tensor* t = tensor(name, x, &addr)) {
      on(*t);
      const int64_t shape[4] = {c.num_pages, c.hkv, c.page, 128}, dense = (int64_t)c.hkv * c.page * 128;
      const int64_t strides[4] = {c.page_stride ? (int64_t)c.page_stride : dense, (int64_t)c.page * 128, 128, 1};
      bool good = t->element_size() == 1 && t->dim() == 4;
      for (int i = 0; good && i < 4; ++i)
        good = t->size(i) == shape[i] && (shape[i] <= 1 || t->stride(i) == strides[i]);
      if (!good) {
        std::ostringstream s;
        s << name << " has to hold one-byte codes " << at::IntArrayRef(shape, 4) << " with strides "
          << at::IntArrayRef(strides, 4) << told(*t);
        refuse(s.str());
      }
      addr = t->data_ptr();
    }
    return addr;
  }
  prism_stream_t stream(PyObject* x) const {
    if (x == Py_None)
      return reinterpret_cast<prism_stream_t>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
    return reinterpret_cast<prism_stream_t>(PyLong_AsVoidPtr(x));
  }
};

const prism_cache_config& config(PyObject* x) { return *static_cast<const prism_cache_config*>(PyLong_AsVoidPtr(x)); }

// Runs f with the number of arguments checked; C++ exceptions become Python's.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  try {
    if (n != want || !g_plan) throw std::runtime_error("wrong number of arguments, or entries() was not called");
    return PyLong_FromLong(f());
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* entries(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 3) return PyErr_Format(PyExc_TypeError, "three addresses");
  g_plan = reinterpret_cast<decltype(g_plan)>(PyLong_AsVoidPtr(a[0]));
  g_store = reinterpret_cast<decltype(g_store)>(PyLong_AsVoidPtr(a[1]));
  g_attn = reinterpret_cast<decltype(g_attn)>(PyLong_AsVoidPtr(a[2]));
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const prism_cache_config& c = config(a[0]);
    Call k{"prism_cache_plan"};
    auto ints = [&](const char* name, PyObject* x, int64_t numel) { return k.flat<int32_t>(name, x, at::kInt, numel); };
    int32_t *held = ints("held", a[1], c.requests), *add = ints("add", a[2], c.requests),
            *ring = ints("ring", a[3], c.num_pages), *state = ints("state", a[4], 4),
            *table = k.flat<int32_t>("table", a[5], at::kInt, (int64_t)c.requests * c.max_pages, false, {c.max_pages}), *lens = ints("lens", a[6], c.requests),
            *starts = ints("starts", a[7], (int64_t)c.requests + 1), *slots = ints("slots", a[8], c.tokens),
            *state_out = ints("state_out", a[9], 4);
    return g_plan(&c, held, add, ring, state, table, lens, starts, slots, state_out, k.stream(a[10]));
  });
}

PyObject* store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&] {
    const prism_cache_config& c = config(a[0]);
    Call k{"prism_cache_store"};
    long long k_tok, k_head, v_tok, v_head;
    const int64_t scales = (int64_t)c.num_pages * c.hkv;
    void *key = k.rows("k", a[1], c.tokens, c.hkv, &k_tok, &k_head), *val = k.rows("v", a[2], c.tokens, c.hkv, &v_tok, &v_head);
    int32_t* slots = k.flat<int32_t>("slots", a[3], at::kInt, c.tokens);
    void *kc = k.pages("k_cache", a[4], c), *vc = k.pages("v_cache", a[5], c);
    float *ks = k.flat<float>("k_scale", a[6], at::kFloat, scales, true, {c.hkv}),
          *vs = k.flat<float>("v_scale", a[7], at::kFloat, scales, true, {c.hkv});
    return g_store(&c, key, k_tok, k_head, val, v_tok, v_head, slots, kc, vc, ks, vs, k.stream(a[8]));
  });
}

PyObject* attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const prism_cache_config& c = config(a[0]);
    Call k{"prism_cache_attn"};
    long long q_tok, q_head, o_tok, o_head;
    const int64_t scales = (int64_t)c.num_pages * c.hkv;
    void* q = k.rows("q", a[1], c.tokens, c.hq, &q_tok, &q_head);
    void *kc = k.pages("k_cache", a[2], c), *vc = k.pages("v_cache", a[3], c);
    float *ks = k.flat<float>("k_scale", a[4], at::kFloat, scales, true, {c.hkv}),
          *vs = k.flat<float>("v_scale", a[5], at::kFloat, scales, true, {c.hkv});
    int32_t *table = k.flat<int32_t>("table", a[6], at::kInt, (int64_t)c.requests * c.max_pages, false, {c.max_pages}),
            *lens = k.flat<int32_t>("lens", a[7], at::kInt, c.requests),
            *starts = k.flat<int32_t>("starts", a[8], at::kInt, (int64_t)c.requests + 1);
    void* o = k.rows("o", a[9], c.tokens, c.hq, &o_tok, &o_head);
    if ((o_tok || o_head) && (o_tok != (long long)c.hq * 128 || o_head != 128))  // (a tensor)
      throw Refused("tensor arguments must be contiguous");
    void* ws;
    size_t bytes = 0;
    if (const at::Tensor* t = k.tensor("workspace", a[10], &ws)) {
      k.on(*t);
      if (!t->is_contiguous()) throw Refused("tensor arguments must be contiguous");
      ws = t->data_ptr();
      bytes = t->nbytes();
    } else if (ws) {
      k.refuse("workspace has to be a tensor: its size is checked");
    }
    const int64_t words = (((int64_t)c.max_pages * c.page + 127) / 128 + 31) / 32;
    uint32_t* mask = k.flat<uint32_t>("mask", a[11], at::kInt, (int64_t)c.requests * c.hq * words, false, {c.hq, words});
    return g_attn(&c, q, q_tok, q_head, kc, vc, ks, vs, table, lens, starts, mask, o, ws, bytes, k.stream(a[12]));
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__prism_bind() {
  static PyMethodDef methods[] = {method<entries>("entries"), method<plan>("plan"), method<store>("store"),
                                  method<attn>("attn"), {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_prism_bind", nullptr, -1, methods,
                               nullptr, nullptr, nullptr, nullptr};
  return PyModule_Create(&module);
}
