// Argument marshalling of the short calls (rotary positions and the 8-bit cache)
// from PyTorch tensors to the C ABI, as a CPython extension module.
//
// A decode step makes these calls once per layer with a few microseconds of GPU
// work each, so the time on the host is what they cost: checking a tensor's shape,
// type, device and contiguity through Python attributes takes 0.5 us a tensor and
// allocating an output 2 us.  Here a check is a few loads.  Nothing is computed: each
// function checks what the library cannot see, allocates what the caller did not
// pass, and calls the entry point of the same name on the tensors' device and
// stream.  The library's functions are handed in by address (bind), so there is
// one copy of it in the process.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/CUDAContext.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>

#include "splitkv.h"

namespace {

// ------------------------------------------------------------ the library

struct Library {
  decltype(&::rope_apply) rope_apply = nullptr;
  decltype(&::kv8_append) kv8_append = nullptr;
  decltype(&::kv8_fetch) kv8_fetch = nullptr;
  decltype(&::attn_splitkv_kv8_plan) plan = nullptr;
  decltype(&::attn_splitkv_kv8_workspace) workspace = nullptr;
  decltype(&::attn_splitkv_decode_kv8) decode = nullptr;
  decltype(&::kv8_evict) evict = nullptr;
};
Library g_lib;
PyObject* g_error = nullptr;  // SkvError

// A Python exception is set (with the error indicator), unwind to the entry.
struct PythonError {};

[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw PythonError();
}

void check(skv_status s, const char* what) {
  if (s == SKV_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(s), what);
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw PythonError();
}

// ------------------------------------------------------------ arguments

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor, not %.100s", name, Py_TYPE(o)->tp_name);
    throw PythonError();
  }
  return THPVariable_Unpack(o);
}

std::string text(at::IntArrayRef shape) {
  std::ostringstream s;
  s << "(";
  for (size_t i = 0; i < shape.size(); ++i) s << (i ? ", " : "") << shape[i];
  s << ")";
  return s.str();
}

// The address of a tensor of exactly this shape, type and device, contiguous.
void* address(const at::Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType dt, int dev) {
  if (t.scalar_type() != dt)
    refuse(std::string(name) + " has dtype " + c10::toString(t.scalar_type()) + ", expected " + c10::toString(dt));
  if (t.sizes() != shape)
    refuse(std::string(name) + " has shape " + text(t.sizes()) + ", expected " + text(shape));
  if (!t.is_cuda() || dev < 0) refuse("tensors must be on a CUDA device");
  if (t.get_device() != dev)
    refuse(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", expected cuda:" + std::to_string(dev));
  if (!t.is_contiguous()) refuse("tensors must be contiguous");
  return t.data_ptr();
}

void* arg(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType dt, int dev) {
  if (o == Py_None) refuse(std::string(name) + " is needed");
  return address(tensor(o, name), name, shape, dt, dev);
}

void* opt(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType dt, int dev) {
  return o == Py_None ? nullptr : address(tensor(o, name), name, shape, dt, dev);
}

int index_of(const at::Tensor& t) { return t.is_cuda() ? static_cast<int>(t.get_device()) : -1; }

skv_dtype half(at::ScalarType dt, const char* name) {
  if (dt == at::kBFloat16) return SKV_BF16;
  if (dt == at::kHalf) return SKV_FP16;
  refuse(std::string(name) + " must be bfloat16 or float16, not " + c10::toString(dt));
}

int small(int64_t x, const char* name) {
  if (x < INT_MIN || x > INT_MAX) refuse(std::string(name) + " is too large");
  return static_cast<int>(x);
}

int integer(PyObject* o, const char* name) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw PythonError();
  return small(x, name);
}

double real(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw PythonError();
  return x;
}

bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw PythonError();
  return x != 0;
}

// Makes the tensors' device current for a call, and the caller's stream (its
// address as an integer; None: the device's current one): what the call allocates
// then belongs to the stream it runs on.  Memory of another stream could still be in
// use there, and would be handed out again there before this call has run; so what the
// caller passes is recorded as in use on the given stream, and what it gets as in use
// on the current one.
class On {
 public:
  On(int dev, PyObject* const* args, Py_ssize_t n) : dev_(static_cast<c10::DeviceIndex>(dev)), device_(dev_) {
    const c10::cuda::CUDAStream now = c10::cuda::getCurrentCUDAStream(dev_);
    handle = reinterpret_cast<skv_stream_t>(now.stream());
    PyObject* stream = args[n - 1];  // the last argument of every call
    if (stream != Py_None) {
      void* p = PyLong_AsVoidPtr(stream);
      if (p == nullptr && PyErr_Occurred()) throw PythonError();
      if (p != now.stream()) {
        caller_ = now;
        stream_.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), dev_));
        handle = reinterpret_cast<skv_stream_t>(static_cast<cudaStream_t>(p));
        for (Py_ssize_t i = 0; i < n; ++i) record(args[i]);
      }
    }
  }
  // a new output (not through the operator dispatch of at::empty)
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType dt) const {
    at::Tensor t = scratch(shape, dt);
    if (caller_) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), *caller_);
    return t;
  }
  // memory that the call alone uses
  at::Tensor scratch(at::IntArrayRef shape, at::ScalarType dt) const {
    return at::Tensor(at::detail::empty_cuda(shape, dt, at::Device(at::kCUDA, dev_), std::nullopt));
  }
  skv_stream_t handle;

 private:
  void record(PyObject* o) const {
    if (PyTuple_Check(o)) {  // a cache
      for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(o); ++i) record(PyTuple_GET_ITEM(o, i));
    } else if (THPVariable_Check(o)) {
      c10::cuda::CUDACachingAllocator::recordStream(THPVariable_Unpack(o).storage().data_ptr(), stream_->current_stream());
    }
  }
  c10::DeviceIndex dev_;
  c10::cuda::CUDAGuard device_;
  std::optional<c10::cuda::CUDAStream> caller_;  // the current stream, where it is not the call's
  std::optional<c10::cuda::CUDAStreamGuard> stream_;
};

// ------------------------------------------------------------ the cache

struct Cache {
  void *k, *v;
  float *ks, *vs;
  int64_t B, Hkv, capacity, D;
  int block;
  skv_code code;
  at::ScalarType type;
};

// The four tensors of a KV8Cache, checked, on device dev.
Cache cache_of(PyObject* o, int dev, const char* name) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) {
    PyErr_Format(PyExc_TypeError, "%s must be a KV8Cache, not %.100s", name, Py_TYPE(o)->tp_name);
    throw PythonError();
  }
  const at::Tensor& k = tensor(PyTuple_GET_ITEM(o, 0), "cache.k");
  const at::Tensor& ks = tensor(PyTuple_GET_ITEM(o, 2), "cache.k_scale");
  Cache c;
  c.type = k.scalar_type();
  if ((c.type != at::kChar && c.type != at::kFloat8_e4m3fn) || k.dim() != 4 || ks.dim() != 3 || ks.size(2) == 0 ||
      k.size(2) == 0 || k.size(2) % ks.size(2) != 0)
    refuse(std::string(name) + ": codes are int8 or float8_e4m3fn [B, Hkv, capacity, D], scales float32 "
                               "[B, Hkv, capacity / block]");
  c.code = c.type == at::kChar ? SKV_INT8 : SKV_E4M3;
  c.B = k.size(0);
  c.Hkv = k.size(1);
  c.capacity = k.size(2);
  c.D = k.size(3);
  c.block = small(c.capacity / ks.size(2), "block");
  const int64_t blocks[3] = {c.B, c.Hkv, ks.size(2)};
  c.k = address(k, "cache.k", k.sizes(), c.type, dev);
  c.v = arg(PyTuple_GET_ITEM(o, 1), "cache.v", k.sizes(), c.type, dev);
  c.ks = static_cast<float*>(address(ks, "cache.k_scale", blocks, at::kFloat, dev));
  c.vs = static_cast<float*>(arg(PyTuple_GET_ITEM(o, 3), "cache.v_scale", blocks, at::kFloat, dev));
  small(c.B, "B");
  small(c.Hkv, "Hkv");
  small(c.capacity, "capacity");
  small(c.D, "D");
  return c;
}

int cache_device(PyObject* o) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) return -1;
  return index_of(tensor(PyTuple_GET_ITEM(o, 0), "cache.k"));
}

// ------------------------------------------------------------ entry points
// Each body runs inside this: Python errors pass through, C++ ones (an
// allocation that fails) become PyTorch's own exceptions.
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F body) {
  HANDLE_TH_ERRORS
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", got, want);
    return nullptr;
  }
  try {
    return body();
  } catch (const PythonError&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* pair(PyObject* a, PyObject* b) {  // takes both references
  PyObject* t = (a != nullptr && b != nullptr) ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return t;
}

// a given output, or the one allocated for it
PyObject* result(PyObject* given, const at::Tensor& made) {
  if (given != Py_None) return Py_NewRef(given);
  if (!made.defined()) return Py_NewRef(Py_None);
  return THPVariable_Wrap(made);
}

bool needs_gradient(PyObject* o) { return o != Py_None && THPVariable_Check(o) && THPVariable_Unpack(o).requires_grad(); }

// Tells autograd that a tensor of the caller's was written.
void written(PyObject* o) {
  if (o == Py_None) return;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// rope_apply(q, k, positions, inv_freq, layout, interleaved, factor, inverse, q_out, k_out, stream)
// None, and nothing done, where autograd has to record it.
PyObject* py_rope_apply(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    if (at::GradMode::is_enabled())
      for (const int i : {0, 1, 3, 8, 9})
        if (needs_gradient(a[i])) return Py_NewRef(Py_None);
    const at::Tensor& q = tensor(a[0], "q");
    const int layout = integer(a[4], "layout");
    if (q.dim() != (layout == SKV_TND ? 3 : 4)) refuse("q has " + std::to_string(q.dim()) + " dimensions, not the layout's");
    const int dev = index_of(q);
    const at::ScalarType dt = q.scalar_type();
    const skv_dtype code = half(dt, "q");
    int64_t B = 1, S, Hq, Hkv = 0;
    const int64_t D = q.size(-1);
    if (layout == SKV_HND) {
      B = q.size(0);
      Hq = q.size(1);
      S = q.size(2);
    } else {
      if (layout == SKV_NHD) B = q.size(0);
      S = q.size(-3);
      Hq = q.size(-2);
    }
    const void* pq = address(q, "q", q.sizes(), dt, dev);
    const void* pk = nullptr;
    at::DimVector k_shape;
    if (a[1] != Py_None) {
      const at::Tensor& k = tensor(a[1], "k");
      k_shape = at::DimVector(q.sizes());
      const size_t at = layout == SKV_HND ? 1 : k_shape.size() - 2;
      if (k.dim() == q.dim()) k_shape[at] = Hkv = k.size(static_cast<int64_t>(at));
      pk = address(k, "k", k_shape, dt, dev);
    } else if (a[9] != Py_None) {
      refuse("k_out without k");
    }
    const int64_t pos2[2] = {B, S};
    const auto* pp = static_cast<const int32_t*>(
        arg(a[2], "positions", layout == SKV_TND ? at::IntArrayRef(pos2 + 1, 1) : at::IntArrayRef(pos2, 2), at::kInt, dev));
    const at::Tensor& f = tensor(a[3], "inv_freq");
    const int64_t nf[1] = {f.numel()};
    const auto* pf = static_cast<const double*>(address(f, "inv_freq", nf, at::kDouble, dev));
    const On on(dev, a, n);
    at::Tensor qo, ko;
    void* pqo = opt(a[8], "q_out", q.sizes(), dt, dev);
    void* pko = opt(a[9], "k_out", k_shape, dt, dev);
    if (pqo == nullptr && a[8] == Py_None) {
      qo = on.empty(q.sizes(), dt);
      pqo = qo.data_ptr();
    }
    if (a[1] != Py_None && a[9] == Py_None) {
      ko = on.empty(k_shape, dt);
      pko = ko.data_ptr();
    }
    if (B * S > 0) {
      check(g_lib.rope_apply(pq, pk, pqo, pko, pp, pf, small(B, "B"), small(Hq, "Hq"), small(Hkv, "Hkv"), small(S, "S"),
                             small(D, "D"), small(2 * nf[0], "inv_freq"), static_cast<float>(real(a[6])), code,
                             static_cast<skv_layout>(layout), truth(a[5]), truth(a[7]), on.handle),
            "rope_apply");
      written(a[8]);
      written(a[9]);
    }
    return pair(result(a[8], qo), result(a[9], ko));
  });
}

// kv8_append(cache, k, v, start, num_new, layout, cu_seqlens, max_seqlen, stream)
PyObject* py_kv8_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor& k = tensor(a[1], "k");
    const int dev = index_of(k), layout = integer(a[5], "layout");
    const at::ScalarType dt = k.scalar_type();
    const Cache c = cache_of(a[0], dev, "cache");
    int64_t S, T = 0;
    at::DimVector shape;
    if (layout == SKV_TND) {
      if (a[6] == Py_None || a[7] == Py_None || a[4] != Py_None || k.dim() != 3)
        refuse("TND rows are [tokens, heads, D], with cu_seqlens and max_seqlen and without num_new");
      T = k.size(0);
      S = std::min<int64_t>(integer(a[7], "max_seqlen"), T);  // no sequence is longer than all rows
      shape = {T, c.Hkv, c.D};
    } else {
      if (a[6] != Py_None || a[7] != Py_None || k.dim() != 4)
        refuse("HND and NHD rows are 4-D, without cu_seqlens and max_seqlen");
      S = k.size(layout == SKV_HND ? 2 : 1);
      shape = layout == SKV_HND ? at::DimVector{c.B, c.Hkv, S, c.D} : at::DimVector{c.B, S, c.Hkv, c.D};
    }
    const void* pk = address(k, "k", shape, dt, dev);
    const void* pv = arg(a[2], "v", shape, dt, dev);
    const int64_t b[1] = {c.B}, b1[1] = {c.B + 1};
    const auto* ps = static_cast<const int32_t*>(arg(a[3], "start", b, at::kInt, dev));
    const auto* pn = static_cast<const int32_t*>(opt(a[4], "num_new", b, at::kInt, dev));
    const auto* pc = static_cast<const int32_t*>(opt(a[6], "cu_seqlens", b1, at::kInt, dev));
    const skv_dtype code = half(dt, "k");
    const On on(dev, a, n);
    if (S != 0 && (T != 0 || layout != SKV_TND)) {
      check(g_lib.kv8_append(pk, pv, c.k, c.v, c.ks, c.vs, ps, pn, pc, static_cast<int>(c.B), static_cast<int>(c.Hkv),
                             small(S, "S"), small(T, "tokens"), static_cast<int>(c.capacity), static_cast<int>(c.D), c.block,
                             code, c.code, static_cast<skv_layout>(layout), on.handle),
            "kv8_append");
    }
    return Py_NewRef(Py_None);
  });
}

// kv8_fetch(cache, n, dtype, start, kv_len, layout, k_out, v_out, stream)
PyObject* py_kv8_fetch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const int dev = cache_device(a[0]), rows = integer(a[1], "n"), layout = integer(a[5], "layout");
    const Cache c = cache_of(a[0], dev, "cache");
    if ((layout != SKV_HND && layout != SKV_NHD) || rows < 0) refuse("kv8_fetch takes HND or NHD, and n >= 0");
    at::ScalarType dt = at::kBFloat16;
    if (a[2] != Py_None) {
      if (!THPDtype_Check(a[2])) {
        PyErr_SetString(PyExc_TypeError, "dtype must be a torch.dtype");
        throw PythonError();
      }
      dt = reinterpret_cast<THPDtype*>(a[2])->scalar_type;
    } else if (a[6] != Py_None) {
      dt = tensor(a[6], "k_out").scalar_type();
    }
    const skv_dtype code = half(dt, "dtype");
    const at::DimVector shape =
        layout == SKV_HND ? at::DimVector{c.B, c.Hkv, rows, c.D} : at::DimVector{c.B, rows, c.Hkv, c.D};
    const int64_t b[1] = {c.B};
    const auto* ps = static_cast<const int32_t*>(opt(a[3], "start", b, at::kInt, dev));
    const auto* pl = static_cast<const int32_t*>(opt(a[4], "kv_len", b, at::kInt, dev));
    const On on(dev, a, n);
    at::Tensor ko, vo;
    void* pk = opt(a[6], "k_out", shape, dt, dev);
    void* pv = opt(a[7], "v_out", shape, dt, dev);
    if (a[6] == Py_None) {
      ko = on.empty(shape, dt);
      pk = ko.data_ptr();
    }
    if (a[7] == Py_None) {
      vo = on.empty(shape, dt);
      pv = vo.data_ptr();
    }
    if (rows != 0) {
      check(g_lib.kv8_fetch(c.k, c.v, c.ks, c.vs, pk, pv, ps, pl, static_cast<int>(c.B), static_cast<int>(c.Hkv), rows,
                            static_cast<int>(c.capacity), static_cast<int>(c.D), c.block, code, c.code,
                            static_cast<skv_layout>(layout), on.handle),
            "kv8_fetch");
    }
    return pair(result(a[6], ko), result(a[7], vo));
  });
}

// decode_kv8(q, cache, scale, kv_len, causal, weights, num_ctas, out, lse, return_lse, workspace, stream)
PyObject* py_decode_kv8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    const int dev = index_of(q);
    const at::ScalarType dt = q.scalar_type();
    const Cache c = cache_of(a[1], dev, "cache");
    if (q.dim() != 4) refuse("decode q is [B, Hq, Lq, D]");
    const int64_t Hq = q.size(1), Lq = q.size(2);
    const int64_t shape[4] = {c.B, Hq, Lq, c.D};
    const void* pq = address(q, "q", shape, dt, dev);
    const skv_dtype code = half(dt, "q");
    const int64_t b[1] = {c.B}, bhn[3] = {c.B, c.Hkv, c.capacity};
    const auto* pn = static_cast<const int32_t*>(opt(a[3], "kv_len", b, at::kInt, dev));
    auto* pw = static_cast<float*>(opt(a[5], "weights", bhn, at::kFloat, dev));
    const int iB = static_cast<int>(c.B), iHq = small(Hq, "Hq"), iHkv = static_cast<int>(c.Hkv), iLq = small(Lq, "Lq"),
              iN = static_cast<int>(c.capacity), iD = static_cast<int>(c.D);
    int ctas = integer(a[6], "num_ctas");
    check(g_lib.plan(iB, iHq, iHkv, iLq, iN, iD, at::cuda::getDeviceProperties(static_cast<c10::DeviceIndex>(dev))->multiProcessorCount,
                     ctas, &ctas),
          "attn_splitkv_decode_kv8");
    const On on(dev, a, n);
    at::Tensor out, lse, ws;
    void* po = opt(a[7], "out", shape, dt, dev);
    if (a[7] == Py_None) {
      out = on.empty(shape, dt);
      po = out.data_ptr();
    }
    const bool want_lse = truth(a[9]);
    auto* pl = want_lse ? static_cast<float*>(opt(a[8], "lse", at::IntArrayRef(shape, 3), at::kFloat, dev)) : nullptr;
    if (want_lse && a[8] == Py_None) {
      lse = on.empty(at::IntArrayRef(shape, 3), at::kFloat);
      pl = static_cast<float*>(lse.data_ptr());
    }
    void* pws = nullptr;
    size_t bytes = 0;
    if (a[10] != Py_None) {
      const at::Tensor& w = tensor(a[10], "workspace");
      if (index_of(w) != dev || !w.is_contiguous()) refuse("workspace must be contiguous, on the device of q");
      pws = w.data_ptr();
      bytes = w.nbytes();
    } else {
      bytes = g_lib.workspace(iB, iHq, iHkv, iLq, iN, iD, ctas, pw != nullptr);
      if (bytes > 0) {
        const int64_t size[1] = {static_cast<int64_t>(bytes)};
        ws = on.scratch(size, at::kByte);
        pws = ws.data_ptr();
      }
    }
    const float scale = a[2] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(c.D))) : static_cast<float>(real(a[2]));
    check(g_lib.decode(pq, c.k, c.v, c.ks, c.vs, po, pl, pw, iB, iHq, iHkv, iLq, iN, iD, c.block, scale, code, c.code, pn,
                       truth(a[4]), ctas, pws, bytes, on.handle),
          "attn_splitkv_decode_kv8");
    return pair(result(a[7], out), want_lse ? result(a[8], lse) : Py_NewRef(Py_None));
  });
}

// kv8_evict(cache, to, weights, to_weights, kv_len, budget, sink, recent, kept, new_len, stream)
PyObject* py_kv8_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const int dev = cache_device(a[0]);
    const Cache c = cache_of(a[0], dev, "cache"), t = cache_of(a[1], dev, "to");
    if (t.B != c.B || t.Hkv != c.Hkv || t.D != c.D || t.block != c.block || t.code != c.code)
      refuse("the two caches differ in more than their capacity");
    const int budget = integer(a[5], "budget"), sink = integer(a[6], "sink"), recent = integer(a[7], "recent");
    if (budget < 1 || budget > t.capacity || sink < 0 || recent < 0 || static_cast<int64_t>(sink) + recent > budget)
      refuse("budget " + std::to_string(budget) + " must fit the capacity " + std::to_string(t.capacity) +
             " and hold sink " + std::to_string(sink) + " + recent " + std::to_string(recent));
    const int64_t b[1] = {c.B}, from[3] = {c.B, c.Hkv, c.capacity}, to[3] = {c.B, c.Hkv, t.capacity},
                  bhk[3] = {c.B, c.Hkv, budget};
    const auto* pw = static_cast<const float*>(arg(a[2], "weights", from, at::kFloat, dev));
    auto* pt = static_cast<float*>(arg(a[3], "to_weights", to, at::kFloat, dev));
    const auto* pn = static_cast<const int32_t*>(opt(a[4], "kv_len", b, at::kInt, dev));
    const On on(dev, a, n);
    at::Tensor kept, len;
    auto* pk = static_cast<int32_t*>(opt(a[8], "kept", bhk, at::kInt, dev));
    auto* pl = static_cast<int32_t*>(opt(a[9], "new_len", b, at::kInt, dev));
    if (a[8] == Py_None) {
      kept = on.empty(bhk, at::kInt);
      pk = static_cast<int32_t*>(kept.data_ptr());
    }
    if (a[9] == Py_None) {
      len = on.empty(b, at::kInt);
      pl = static_cast<int32_t*>(len.data_ptr());
    }
    check(g_lib.evict(c.k, c.v, c.ks, c.vs, pw, pn, t.k, t.v, t.ks, t.vs, pt, pk, pl, static_cast<int>(c.B),
                      static_cast<int>(c.Hkv), static_cast<int>(c.capacity), static_cast<int>(t.capacity),
                      static_cast<int>(c.D), c.block, c.code, budget, sink, recent, on.handle),
          "kv8_evict");
    return pair(result(a[8], kept), result(a[9], len));
  });
}

// bind(SkvError, addresses): the seven functions of Library, in its order
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    void* f[7];
    for (int i = 0; i < 7; ++i) {
      f[i] = PyLong_AsVoidPtr(a[i + 1]);
      if (f[i] == nullptr) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a function's address is missing");
        throw PythonError();
      }
    }
    Library l;
    l.rope_apply = reinterpret_cast<decltype(l.rope_apply)>(f[0]);
    l.kv8_append = reinterpret_cast<decltype(l.kv8_append)>(f[1]);
    l.kv8_fetch = reinterpret_cast<decltype(l.kv8_fetch)>(f[2]);
    l.plan = reinterpret_cast<decltype(l.plan)>(f[3]);
    l.workspace = reinterpret_cast<decltype(l.workspace)>(f[4]);
    l.decode = reinterpret_cast<decltype(l.decode)>(f[5]);
    l.evict = reinterpret_cast<decltype(l.evict)>(f[6]);
    g_lib = l;
    Py_XSETREF(g_error, Py_NewRef(a[0]));
    return Py_NewRef(Py_None);
  });
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(py_##name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(rope_apply), FAST(kv8_append), FAST(kv8_fetch), FAST(decode_kv8),
                         FAST(kv8_evict),  FAST(bind),       {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_skv_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__skv_torch() { return PyModule_Create(&module); }
