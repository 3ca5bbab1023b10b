// Python calls of the paged entry points (include/rtp.h): checks of the tensors and marshalling
// only. A decode step makes two such calls per layer and a kernel of a few microseconds each, and
// the same checks in Python with ctypes took 4 us a call more than the launch itself.
// The library's functions come by address (bind), so the build that Python has loaded is called.
#include <Python.h>

#include <ATen/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/rtp.h"

namespace {

decltype(&rtp_paged_reserve_step) f_reserve;
decltype(&rtp_paged_append_kv) f_append;
decltype(&rtp_paged_decode_step) f_decode;
decltype(&rtp_paged_decode_step_append) f_decode_append;

struct Refused {};

[[noreturn]] void refuse(const std::string& why) {
  PyErr_SetString(PyExc_ValueError, why.c_str());
  throw Refused{};
}

// The data of a contiguous tensor of n elements of a type on a device; null for None if that may be
void* data(PyObject* o, const char* what, at::ScalarType type, int64_t n, int64_t dev,
           bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  if (THPVariable_Check(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() == type && t.numel() == n && t.get_device() == dev && t.is_contiguous())
      return t.data_ptr();
    refuse(std::string(what) + ": a contiguous " + c10::toString(type) + " tensor of " +
           std::to_string(n) + " elements on cuda:" + std::to_string(dev) + " is wanted, got " +
           c10::toString(t.scalar_type()) + " of " + std::to_string(t.numel()) + " on " +
           t.device().str() + (t.is_contiguous() ? "" : ", not contiguous"));
  }
  refuse(std::string(what) + ": a tensor is wanted");
}

struct Space { void* p; size_t bytes; };
Space workspace(PyObject* o, int64_t dev) {
  if (o == Py_None) return {nullptr, 0};
  if (!THPVariable_Check(o)) refuse("workspace: a tensor is wanted");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.get_device() != dev || !t.is_contiguous())
    refuse("workspace: a contiguous tensor on cuda:" + std::to_string(dev) + " is wanted");
  return {t.data_ptr(), (size_t)t.numel() * t.element_size()};
}

int64_t number(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
template <class T>
T* address(PyObject* o) { return reinterpret_cast<T*>(number(o)); }

// A stream by its address, or the device's current one for None
rtp_stream_t stream_of(PyObject* o, int64_t dev) {
  if (dev < 0 || c10::cuda::current_device() != dev)
    refuse("tensors are on cuda:" + std::to_string(dev) + ", which is not the current device");
  if (o == Py_None) return reinterpret_cast<rtp_stream_t>(c10::cuda::getCurrentCUDAStream((int)dev).stream());
  return reinterpret_cast<rtp_stream_t>(number(o));
}

template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments are wanted, got %zd", want, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <class F>
int unlocked(F&& f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return rc;
}

using at::kBFloat16;
using at::kFloat;
using at::kInt;
using at::kLong;

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&] {
    f_reserve = reinterpret_cast<decltype(f_reserve)>(number(a[0]));
    f_append = reinterpret_cast<decltype(f_append)>(number(a[1]));
    f_decode = reinterpret_cast<decltype(f_decode)>(number(a[2]));
    f_decode_append = reinterpret_cast<decltype(f_decode_append)>(number(a[3]));
    return 0;
  });
}

// (pool, B, device, lens, new_lens, counters, lens_out, counters_out, slot_map, n_new, step_lens, ws,
// stream); step_lens may be None
PyObject* reserve(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const auto* pool = address<const rtp_page_pool>(a[0]);
    const int64_t B = number(a[1]), dev = number(a[2]), n_new = number(a[9]);
    const auto* lens = static_cast<const int32_t*>(data(a[3], "lens", kInt, B, dev));
    const auto* wish = static_cast<const int32_t*>(data(a[4], "new_lens", kInt, B, dev));
    const auto* ctr = static_cast<const int64_t*>(data(a[5], "counters", kLong, 2, dev));
    auto* lens_out = static_cast<int32_t*>(data(a[6], "lens_out", kInt, B, dev));
    auto* ctr_out = static_cast<int64_t*>(data(a[7], "counters_out", kLong, 2, dev));
    auto* slots = static_cast<int32_t*>(data(a[8], "slot_map", kInt, B * n_new, dev, n_new == 0));
    auto* step = static_cast<int32_t*>(data(a[10], "step_lens", kInt, B, dev, true));
    const Space ws = workspace(a[11], dev);
    const rtp_stream_t st = stream_of(a[12], dev);
    if (n_new != (int32_t)n_new) refuse("n_new is out of range");
    return unlocked([&] {
      return f_reserve(pool, lens, wish, ctr, lens_out, ctr_out, slots, (int32_t)n_new, step, ws.p, ws.bytes,
                       st);
    });
  });
}

// (desc, cache, B, Hkv, device, k_pre, v, start_pos, slot_map, n_new, ws, stream)
PyObject* append_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const auto* desc = address<const rtp_layer_desc>(a[0]);
    const auto* cache = address<const rtp_paged_cache>(a[1]);
    const int64_t B = number(a[2]), Hkv = number(a[3]), dev = number(a[4]), n_new = number(a[9]);
    const int64_t rows = B * n_new * Hkv * 128;
    const auto* k = static_cast<const uint16_t*>(data(a[5], "k_pre", kBFloat16, rows, dev));
    const auto* v = static_cast<const uint16_t*>(data(a[6], "v", kBFloat16, rows, dev));
    const auto* start = static_cast<const int32_t*>(data(a[7], "start_pos", kInt, B, dev));
    const auto* slots = static_cast<const int32_t*>(data(a[8], "slot_map", kInt, B * n_new, dev));
    const Space ws = workspace(a[10], dev);
    if (ws.p && ws.bytes < 4) refuse("workspace: it does not hold the status word");
    const rtp_stream_t st = stream_of(a[11], dev);
    if (n_new != (int32_t)n_new) refuse("n_new is out of range");
    return unlocked([&] {
      return f_append(desc, cache, k, v, start, slots, (int32_t)n_new, ws.p, st);
    });
  });
}

// (desc, cache, B, Hq, Hkv, device, k_new, v_new, q_pre, seq_lens, out, lse, ws, stream); k_new and
// v_new are None for the step without the append
PyObject* decode_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&] {
    const auto* desc = address<const rtp_layer_desc>(a[0]);
    const auto* cache = address<const rtp_paged_cache>(a[1]);
    const int64_t B = number(a[2]), Hq = number(a[3]), Hkv = number(a[4]), dev = number(a[5]);
    const bool append = a[6] != Py_None || a[7] != Py_None;
    const auto* k = static_cast<const uint16_t*>(data(a[6], "k_new", kBFloat16, B * Hkv * 128, dev, !append));
    const auto* v = static_cast<const uint16_t*>(data(a[7], "v_new", kBFloat16, B * Hkv * 128, dev, !append));
    const auto* q = static_cast<const uint16_t*>(data(a[8], "q_pre", kBFloat16, B * Hq * 128, dev));
    const auto* lens = static_cast<const int32_t*>(data(a[9], "seq_lens", kInt, B, dev));
    auto* out = static_cast<uint16_t*>(data(a[10], "out", kBFloat16, B * Hq * 128, dev));
    auto* lse = static_cast<float*>(data(a[11], "lse", kFloat, B * Hq, dev, true));
    const Space ws = workspace(a[12], dev);
    const rtp_stream_t st = stream_of(a[13], dev);
    return unlocked([&] {
      return append ? f_decode_append(desc, cache, k, v, q, lens, out, lse, ws.p, ws.bytes, st)
                    : f_decode(desc, cache, q, lens, out, lse, ws.p, ws.bytes, st);
    });
  });
}

#define RTP_FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {RTP_FAST(bind), RTP_FAST(reserve), RTP_FAST(append_kv), RTP_FAST(decode_step),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
