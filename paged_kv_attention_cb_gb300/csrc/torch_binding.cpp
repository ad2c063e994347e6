// Checked calls from Python for the entry points of the 8-bit cache and of shared prefixes: a
// CPython module that reads the tensors' types, shapes and addresses itself.
//
// A small decode step takes ~9 us on the GPU; the same checks as Python statements took 10 us and
// the ctypes call with its 34 arguments another 2. Here both are under one. The module only checks
// and passes on: it holds no state but the addresses of libcb's functions and the error class that
// the package hands it (bind), and does not link to libcb.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/TensorBase.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <string>

#include "cb.h"

namespace {

struct Bound {
  decltype(&cb_write_kv_q8) write_kv_q8;
  decltype(&cb_read_kv_q8) read_kv_q8;
  decltype(&cb_paged_attention_q8) paged_attention_q8;
  decltype(&cb_paged_attention_shared) paged_attention_shared;
  decltype(&cb_last_error_message) last_error_message;
} g_lib = {};
PyObject* g_error = nullptr;     // CbError(status, message)
PyObject* g_host_i32 = nullptr;  // anything -> contiguous int32 numpy array

// Thrown once the Python error is set.
struct Raised {};

[[noreturn]] void raise_status(int status, const std::string& message) {
  PyObject* e = PyObject_CallFunction(g_error, "is", status, message.c_str());
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

[[noreturn]] void bad(const std::string& message) { raise_status(CB_ERR_INVALID_ARG, message); }

std::string text(c10::IntArrayRef s) {
  std::string out = "(";
  for (size_t i = 0; i < s.size(); ++i) out += (i ? ", " : "") + std::to_string(s[i]);
  return out + ")";
}

const at::TensorBase& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// A contiguous tensor of this shape and one of these types on `device` (the first tensor's).
void* need(PyObject* o, const char* name, c10::IntArrayRef shape,
           std::initializer_list<c10::ScalarType> types, c10::Device device) {
  const at::TensorBase& t = tensor(o, name);
  bool type_ok = false;
  for (c10::ScalarType s : types) type_ok |= t.scalar_type() == s;
  if (!type_ok) bad(std::string(name) + ": dtype " + c10::toString(t.scalar_type()) + ", not " + c10::toString(*types.begin()));
  if (t.sizes() != shape) bad(std::string(name) + ": shape " + text(t.sizes()) + ", not " + text(shape));
  if (!t.is_contiguous()) bad(std::string(name) + " must be contiguous");
  if (!t.is_cuda() || t.device() != device) bad(std::string(name) + " must be on the CUDA device of the first tensor");
  return const_cast<void*>(t.const_data_ptr());
}

c10::IntArrayRef dims(const at::TensorBase& t, int64_t n, const char* name) {
  if (t.dim() != n) bad(std::string(name) + ": " + std::to_string(t.dim()) + " dimensions, not " + std::to_string(n));
  return t.sizes();
}

int32_t i32(int64_t v, const char* name) {
  if (v < 0 || v > INT32_MAX) bad(std::string(name) + " is too large");
  return (int32_t)v;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) bad(std::string(name) + " is out of range");
  return (int32_t)v;
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return (float)v;
}

int32_t float_code(const at::TensorBase& t, const char* name) {
  if (t.scalar_type() == c10::kBFloat16) return CB_BF16;
  if (t.scalar_type() == c10::kFloat) return CB_F32;
  bad(std::string(name) + ": dtype " + c10::toString(t.scalar_type()) + ", not Float or BFloat16");
}

// A host mirror of n int32 entries (n < 0: any number), held for the length of the call.
class Mirror {
 public:
  Mirror(PyObject* o, int64_t n, const char* name) {
    if (!get(o)) {
      PyErr_Clear();
      converted_ = PyObject_CallFunctionObjArgs(g_host_i32, o, nullptr);
      if (converted_ == nullptr) throw Raised{};
      if (!get(converted_)) {
        Py_CLEAR(converted_);
        PyErr_Clear();
        raise_status(CB_ERR_METADATA, std::string(name) + " must be one-dimensional int32");
      }
    }
    if (n >= 0 && size() != n) {
      const std::string m = std::string(name) + ": " + std::to_string(size()) + " entries, not " + std::to_string(n);
      release();
      raise_status(CB_ERR_METADATA, m);
    }
  }
  ~Mirror() { release(); }
  Mirror(const Mirror&) = delete;
  const int32_t* data() const { return static_cast<const int32_t*>(view_.buf); }
  int64_t size() const { return view_.shape[0]; }

 private:
  bool get(PyObject* o) {
    if (PyObject_GetBuffer(o, &view_, PyBUF_ND | PyBUF_FORMAT) != 0) return false;
    held_ = true;
    const char* f = view_.format ? view_.format : "B";
    if (*f == '@' || *f == '=' || *f == '<') ++f;
    if (view_.ndim == 1 && view_.itemsize == 4 && (f[0] == 'i' || f[0] == 'l') && f[1] == 0) return true;
    PyBuffer_Release(&view_);
    held_ = false;
    return false;
  }
  void release() {
    if (held_) PyBuffer_Release(&view_);
    held_ = false;
    Py_CLEAR(converted_);
  }
  Py_buffer view_ = {};
  bool held_ = false;
  PyObject* converted_ = nullptr;
};

// The device's current stream, or the one given (a torch stream or a raw handle).
void* stream_of(PyObject* o, c10::Device device) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device.index()).stream();
  if (PyLong_Check(o)) {
    void* p = PyLong_AsVoidPtr(o);
    if (p == nullptr && PyErr_Occurred()) throw Raised{};
    return p;
  }
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (h == nullptr) throw Raised{};
  void* p = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (p == nullptr && PyErr_Occurred()) throw Raised{};
  return p;
}

// libcb launches on the current device: the tensors' for the length of the call.
template <typename F>
void call(c10::Device device, F&& f) {
  c10::cuda::OptionalCUDAGuard guard;
  if (c10::cuda::current_device() != device.index()) guard.set_device(device);
  const cb_status status = f();
  if (status != CB_OK) raise_status(status, g_lib.last_error_message());
}

const std::initializer_list<c10::ScalarType> kE4m3 = {c10::kFloat8_e4m3fn, c10::kByte};
const std::initializer_list<c10::ScalarType> kE8m0 = {c10::kFloat8_e8m0fnu, c10::kByte};

struct CacheQ8 {
  void *k, *v, *k_scale, *v_scale;
};

CacheQ8 cache_q8(PyObject* const* a, int64_t NB, int64_t BS, int64_t Hkv, int64_t D, c10::Device dev) {
  const int64_t shape[4] = {NB, BS, Hkv, D};
  const c10::IntArrayRef rows(shape, 4), scales(shape, 3);
  return CacheQ8{need(a[0], "k_cache", rows, kE4m3, dev), need(a[1], "v_cache", rows, kE4m3, dev),
                 need(a[2], "k_scale", scales, kE8m0, dev), need(a[3], "v_scale", scales, kE8m0, dev)};
}

// (k_rows, v_rows, k_cache, v_cache, k_scale, v_scale, slot_mapping, error_word, stream)
void rows_q8(PyObject* const* a, bool write) {
  const char* const kn = write ? "k_new" : "k_out";
  const char* const vn = write ? "v_new" : "v_out";
  const at::TensorBase& k = tensor(a[0], kn);
  const int32_t code = float_code(k, kn);
  const auto ks = dims(k, 3, kn);
  const auto cs = dims(tensor(a[2], "k_cache"), 4, "k_cache");
  const c10::Device dev = k.device();
  void* kp = need(a[0], kn, ks, {k.scalar_type()}, dev);
  void* vp = need(a[1], vn, ks, {k.scalar_type()}, dev);
  const CacheQ8 c = cache_q8(a + 2, cs[0], cs[1], ks[1], ks[2], dev);
  const auto* slots = static_cast<const int64_t*>(need(a[6], "slot_mapping", {ks[0]}, {c10::kLong}, dev));
  int32_t* word = nullptr;
  if (a[7] != Py_None)
    word = static_cast<int32_t*>(need(a[7], "error_word", tensor(a[7], "error_word").sizes(), {c10::kInt}, dev));
  const int32_t T = i32(ks[0], kn), NB = i32(cs[0], "k_cache"), BS = i32(cs[1], "k_cache"), H = i32(ks[1], kn),
                D = i32(ks[2], kn);
  void* s = stream_of(a[8], dev);
  call(dev, [&] {
    return write ? g_lib.write_kv_q8(kp, vp, c.k, c.v, c.k_scale, c.v_scale, slots, T, NB, BS, H, D, code, word, s)
                 : g_lib.read_kv_q8(c.k, c.v, c.k_scale, c.v_scale, slots, kp, vp, T, NB, BS, H, D, code, word, s);
  });
}

// What every step takes.
struct Step {
  c10::Device dev = c10::Device(c10::kCUDA, 0);
  int32_t T, Hq, D, R, stride, NB, BS, Hkv, code;
  c10::ScalarType type;
  void *out, *ws;
  const void *q, *k_new = nullptr, *v_new = nullptr;
  const int32_t *qsl, *seq, *bt;
  const int64_t* slots = nullptr;
  size_t ws_bytes;
};

Step step_of(PyObject* out, PyObject* q, PyObject* k_cache, PyObject* qsl, PyObject* seq, PyObject* bt,
             PyObject* workspace, PyObject* k_new, PyObject* v_new, PyObject* slot_mapping) {
  Step p;
  const at::TensorBase& tq = tensor(q, "q");
  p.type = tq.scalar_type();
  p.code = float_code(tq, "q");
  const auto qs = dims(tq, 3, "q");
  const auto cs = dims(tensor(k_cache, "k_cache"), 4, "k_cache");
  const int64_t R = dims(tensor(seq, "seq_lens"), 1, "seq_lens")[0];
  const int64_t stride = dims(tensor(bt, "block_table"), 2, "block_table")[1];
  p.dev = tq.device();
  p.T = i32(qs[0], "q");
  p.Hq = i32(qs[1], "q");
  p.D = i32(qs[2], "q");
  p.R = i32(R, "seq_lens");
  p.stride = i32(stride, "block_table");
  p.NB = i32(cs[0], "k_cache");
  p.BS = i32(cs[1], "k_cache");
  p.Hkv = i32(cs[2], "k_cache");
  p.q = need(q, "q", qs, {p.type}, p.dev);
  p.out = need(out, "out", qs, {p.type}, p.dev);
  p.qsl = static_cast<const int32_t*>(need(qsl, "query_start_loc", {R + 1}, {c10::kInt}, p.dev));
  p.seq = static_cast<const int32_t*>(need(seq, "seq_lens", {R}, {c10::kInt}, p.dev));
  p.bt = static_cast<const int32_t*>(need(bt, "block_table", {R, stride}, {c10::kInt}, p.dev));
  const at::TensorBase& ws = tensor(workspace, "workspace");
  p.ws = need(workspace, "workspace", ws.sizes(), {ws.scalar_type()}, p.dev);
  p.ws_bytes = (size_t)ws.numel() * ws.element_size();
  if (k_new != Py_None) {
    if (v_new == Py_None || slot_mapping == Py_None) bad("k_new given without v_new or slot_mapping");
    const int64_t rows[3] = {qs[0], cs[2], qs[2]};
    p.k_new = need(k_new, "k_new", rows, {p.type}, p.dev);
    p.v_new = need(v_new, "v_new", rows, {p.type}, p.dev);
    p.slots = static_cast<const int64_t*>(need(slot_mapping, "slot_mapping", {qs[0]}, {c10::kLong}, p.dev));
  }
  return p;
}

// (out, q, k_cache, v_cache, k_scale, v_scale, query_start_loc, seq_lens, block_table,
//  h_query_start_loc, h_seq_lens, workspace, scale, sliding_window, k_new, v_new, slot_mapping,
//  flags, stream)
void attention_q8(PyObject* const* a) {
  const Step p = step_of(a[0], a[1], a[2], a[6], a[7], a[8], a[11], a[14], a[15], a[16]);
  const CacheQ8 c = cache_q8(a + 2, p.NB, p.BS, p.Hkv, p.D, p.dev);
  const Mirror hq(a[9], (int64_t)p.R + 1, "h_query_start_loc"), hs(a[10], p.R, "h_seq_lens");
  const float scale = number(a[12]);
  const int32_t window = integer32(a[13], "sliding_window");
  const uint32_t flags = (uint32_t)integer(a[17]);
  void* s = stream_of(a[18], p.dev);
  call(p.dev, [&] {
    return g_lib.paged_attention_q8(p.out, p.q, c.k, c.v, c.k_scale, c.v_scale, p.k_new, p.v_new, p.slots, p.qsl,
                                    p.seq, p.bt, p.stride, hq.data(), hs.data(), p.R, p.T, p.NB, p.BS, p.Hq, p.Hkv,
                                    p.D, scale, window, p.code, flags, p.ws, p.ws_bytes, s);
  });
}

// (out, q, k_cache, v_cache, query_start_loc, seq_lens, block_table, prefix_lens,
//  h_query_start_loc, h_seq_lens, h_prefix_lens, h_group_start, workspace, scale, sliding_window,
//  k_new, v_new, slot_mapping, flags, stream)
void attention_shared(PyObject* const* a) {
  const Step p = step_of(a[0], a[1], a[2], a[4], a[5], a[6], a[12], a[15], a[16], a[17]);
  const int64_t shape[4] = {p.NB, p.BS, p.Hkv, p.D};
  void* k = need(a[2], "k_cache", shape, {p.type}, p.dev);
  void* v = need(a[3], "v_cache", shape, {p.type}, p.dev);
  const auto* pre = static_cast<const int32_t*>(need(a[7], "prefix_lens", {(int64_t)p.R}, {c10::kInt}, p.dev));
  const Mirror hq(a[8], (int64_t)p.R + 1, "h_query_start_loc"), hs(a[9], p.R, "h_seq_lens"),
      hp(a[10], p.R, "h_prefix_lens"), hg(a[11], -1, "h_group_start");
  if (hg.size() < 1) raise_status(CB_ERR_METADATA, "h_group_start must have n_groups + 1 entries");
  const float scale = number(a[13]);
  const int32_t window = integer32(a[14], "sliding_window");
  const uint32_t flags = (uint32_t)integer(a[18]);
  void* s = stream_of(a[19], p.dev);
  call(p.dev, [&] {
    return g_lib.paged_attention_shared(p.out, p.q, k, v, p.k_new, p.v_new, p.slots, p.qsl, p.seq, p.bt, p.stride,
                                        pre, hq.data(), hs.data(), hp.data(), hg.data(), i32(hg.size() - 1, "h_group_start"),
                                        p.R, p.T, p.NB, p.BS, p.Hq, p.Hkv, p.D, scale, window, p.code, flags, p.ws,
                                        p.ws_bytes, s);
  });
}

// Runs f(args) for exactly n arguments; Python's errors and C++'s come back as Python's.
template <typename F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t n, F&& f) {
  if (have != n) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", have, n);
    return nullptr;
  }
  if (g_error == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, "the binding has not been given libcb (bind)");
    return nullptr;
  }
  try {
    f();
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  Py_RETURN_NONE;
}

PyObject* py_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&] { rows_q8(a, true); });
}
PyObject* py_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&] { rows_q8(a, false); });
}
PyObject* py_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 19, [&] { attention_q8(a); });
}
PyObject* py_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 20, [&] { attention_shared(a); });
}

// bind(addresses of write_kv_q8, read_kv_q8, paged_attention_q8, paged_attention_shared and
// last_error_message, the error class, the converter of host mirrors)
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind takes 7 arguments");
    return nullptr;
  }
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null function address");
      return nullptr;
    }
  }
  g_lib.write_kv_q8 = reinterpret_cast<decltype(g_lib.write_kv_q8)>(p[0]);
  g_lib.read_kv_q8 = reinterpret_cast<decltype(g_lib.read_kv_q8)>(p[1]);
  g_lib.paged_attention_q8 = reinterpret_cast<decltype(g_lib.paged_attention_q8)>(p[2]);
  g_lib.paged_attention_shared = reinterpret_cast<decltype(g_lib.paged_attention_shared)>(p[3]);
  g_lib.last_error_message = reinterpret_cast<decltype(g_lib.last_error_message)>(p[4]);
  Py_INCREF(a[5]);
  Py_INCREF(a[6]);
  Py_XDECREF(g_error);
  Py_XDECREF(g_host_i32);
  g_error = a[5];
  g_host_i32 = a[6];
  Py_RETURN_NONE;
}

#define CB_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef g_methods[] = {{"bind", CB_FAST(py_bind), "Hand over libcb's functions."},
                           {"write_kv_q8", CB_FAST(py_write), "Checked cb_write_kv_q8."},
                           {"read_kv_q8", CB_FAST(py_read), "Checked cb_read_kv_q8."},
                           {"paged_attention_q8", CB_FAST(py_attention), "Checked cb_paged_attention_q8."},
                           {"paged_attention_shared", CB_FAST(py_shared), "Checked cb_paged_attention_shared."},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_cb_torch", "Checked calls of libcb for torch tensors.", -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__cb_torch(void) { return PyModule_Create(&g_module); }
