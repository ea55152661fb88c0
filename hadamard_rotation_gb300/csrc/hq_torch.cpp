// hq_torch.cpp -- the Python calls of the products, norms and caches over torch tensors, in C++.
//
// These calls take the GPU as little as 4 us (a token through the norms), and checking a dozen tensors,
// allocating outputs and marshalling 25 arguments takes Python 10 to 30 us.  Here it is done through
// torch's C++ interface; what is computed and refused is the C ABI's (include/hq.h), which this module
// calls like any other program.  api.py has the Python functions with their documentation.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <exception>
#include <string>

#include "hq.h"

// Which torch and Python this file was compiled for: build.py looks for it in the built module.
#ifdef HQ_BUILT_FOR
__attribute__((used)) static const char built_for[] = HQ_BUILT_FOR;
#endif

namespace {

// A refusal: becomes a Python ValueError.
struct Refused : std::exception {
  std::string text;
  explicit Refused(std::string t) : text(std::move(t)) {}
  const char* what() const noexcept override { return text.c_str(); }
};
struct PythonError {};  // a Python exception is set

using Shape = at::IntArrayRef;

std::string shape_text(Shape s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

const char* type_text(at::ScalarType t) {
  switch (t) {
    case at::kByte: return "torch.uint8";
    case at::kChar: return "torch.int8";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    default: return "a type that is not supported";
  }
}

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// The tensor that must be there, of this shape and type, contiguous, on CUDA device `index`.
const at::Tensor& given(PyObject* o, Shape shape, at::ScalarType type, int index, const char* name) {
  const at::Tensor* t = tensor(o);
  if (!t || t->sizes() != shape || t->scalar_type() != type || !t->is_cuda() || t->get_device() != index ||
      !t->is_contiguous())
    throw Refused(std::string(name) + " must be a contiguous " + type_text(type) + " tensor of shape " +
                  shape_text(shape) + " on cuda:" + std::to_string(index));
  return *t;
}

template <typename T>
const T* at_given(PyObject* o, Shape shape, at::ScalarType type, int index, const char* name) {
  return static_cast<const T*>(given(o, shape, type, index, name).const_data_ptr());
}

const at::Tensor& cuda_tensor(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o);
  if (!t || !t->is_cuda()) throw Refused(std::string(name) + " must be a CUDA tensor (libhq has no CPU path)");
  return *t;
}

// Codes: uint8 of `dims` dimensions.
const at::Tensor& codes(PyObject* o, int dims, const char* name) {
  const at::Tensor& t = cuda_tensor(o, name);
  if (t.dim() != dims || t.scalar_type() != at::kByte)
    throw Refused(std::string(name) + " must be a " + std::to_string(dims) + "-D uint8 tensor of codes");
  return t;
}

bool supported(at::ScalarType t) { return t == at::kFloat || t == at::kBFloat16; }
hq_dtype dtype_of(at::ScalarType t) { return t == at::kFloat ? HQ_F32 : HQ_BF16; }
int64_t tiles_bytes(int64_t rows, int64_t cols) { return (rows + 127) / 128 * ((cols + 3) / 4) * 512; }

// The stream of a call: the one given (of the tensors' device), or that device's current one.
struct Stream {
  c10::cuda::CUDAStream current;
  cudaStream_t handle;
  Stream(PyObject* o, int index) : current(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index))) {
    handle = current.stream();
    if (o == Py_None) return;
    PyObject* d = PyObject_GetAttrString(o, "device_index");
    PyObject* s = d ? PyObject_GetAttrString(o, "cuda_stream") : nullptr;
    if (!d || !s) {
      Py_XDECREF(d);
      throw PythonError();
    }
    const long device = PyLong_AsLong(d);
    handle = static_cast<cudaStream_t>(PyLong_AsVoidPtr(s));
    Py_DECREF(d);
    Py_DECREF(s);
    if (PyErr_Occurred()) throw PythonError();
    if (device != index)
      throw Refused("stream is on cuda:" + std::to_string(device) + ", the tensors on cuda:" + std::to_string(index));
  }
};

// New memory for a call.  It comes from the memory of the call's stream: that of another stream may still be
// in use there by what was freed last.  A result is handed to the current stream as well.
at::Tensor empty(Shape shape, at::ScalarType type, const at::Tensor& like, const Stream& stream, bool result = true) {
  if (stream.handle == stream.current.stream()) return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
  const c10::cuda::CUDAStreamGuard guard(
      c10::cuda::getStreamFromExternal(stream.handle, static_cast<c10::DeviceIndex>(like.get_device())));
  at::Tensor t = at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
  if (result && t.numel()) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), stream.current);
  return t;
}

// A workspace for one call, freed when the call returns: later work on its stream may have it then.
at::Tensor workspace(int64_t bytes, const at::Tensor& like, const Stream& stream) {
  if (bytes < 0) throw Refused("sizes that the library refuses (include/hq.h)");
  return bytes == 0 ? at::Tensor() : empty({bytes}, at::kByte, like, stream, false);
}

// `out` as given, or a new tensor of type `out_dtype`.
at::Tensor output(PyObject* out, PyObject* out_dtype, Shape shape, const at::Tensor& like, const Stream& stream) {
  if (out == Py_None) {
    if (!THPDtype_Check(out_dtype) || !supported(reinterpret_cast<THPDtype*>(out_dtype)->scalar_type))
      throw Refused("out_dtype must be float32 or bfloat16");
    return empty(shape, reinterpret_cast<THPDtype*>(out_dtype)->scalar_type, like, stream);
  }
  const at::Tensor* t = tensor(out);
  if (!t || !supported(t->scalar_type())) throw Refused("out must be a float32 or bfloat16 tensor");
  return given(out, shape, t->scalar_type(), like.get_device(), "out");
}

void* addr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// Calls the C ABI with the tensors' device current and without the interpreter lock; a status that
// is not OK becomes the package's HQError.
template <typename F>
void run(int index, const char* name, F call) {
  hq_status st;
  {
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
    PyThreadState* save = PyEval_SaveThread();
    st = call();
    PyEval_RestoreThread(save);
  }
  if (st == HQ_OK) return;
  PyObject* lib = PyImport_ImportModule("hadamard_rotation_gb300._lib");
  PyObject* r = lib ? PyObject_CallMethod(lib, "check", "is", static_cast<int>(st), name) : nullptr;
  Py_XDECREF(lib);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, hq_status_string(st));
  throw PythonError();
}

PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  PyObject* o = THPVariable_Wrap(t);
  if (!o) throw PythonError();
  return o;
}

PyObject* tuple(std::initializer_list<PyObject*> items) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (r) PyTuple_SET_ITEM(r, i++, o);
    else Py_DECREF(o);
  }
  if (!r) throw PythonError();
  return r;
}

// Runs a call's body; C++ exceptions become Python's.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F body) {
  try {
    if (n != want) throw Refused("wrong number of arguments");
    return body();
  } catch (const PythonError&) {
    return nullptr;
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (xq, xs, x_sg, wq, ws, w_sg, offsets, out, out_dtype, stream); MXFP4 has None for the two scales.
template <bool MX>
PyObject* grouped_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const at::Tensor &xq = codes(a[0], 2, "xq"), &wq = codes(a[3], 3, "wq");
    const int index = static_cast<int>(xq.get_device());
    const int64_t M = xq.size(0), K = 2 * xq.size(1), E = wq.size(0), N = wq.size(1), block = MX ? 32 : 16;
    const auto* q = at_given<uint8_t>(a[0], {M, K / 2}, at::kByte, index, "xq");
    const auto* s = at_given<uint8_t>(a[1], {M, K / block}, at::kByte, index, "xs");
    const auto* g = MX ? nullptr : at_given<float>(a[2], {1}, at::kFloat, index, "x_sg");
    const auto* w = at_given<uint8_t>(a[3], {E, N, K / 2}, at::kByte, index, "wq");
    const auto* t = at_given<uint8_t>(a[4], {E, tiles_bytes(N, K / block)}, at::kByte, index, "ws");
    const auto* h = MX ? nullptr : at_given<float>(a[5], {E}, at::kFloat, index, "w_sg");
    const auto* o = at_given<int32_t>(a[6], {E + 1}, at::kInt, index, "offsets");
    const Stream stream(a[9], index);
    const at::Tensor out = output(a[7], a[8], {M, N}, xq, stream);
    const at::Tensor work = workspace(hq_grouped_gemm_workspace_bytes(M, N, K, E), xq, stream);
    run(index, MX ? "hq_grouped_gemm_mxfp4" : "hq_grouped_gemm_nvfp4", [&] {
      const hq_dtype dt = dtype_of(out.scalar_type());
      return MX ? hq_grouped_gemm_mxfp4(q, s, w, t, o, M, N, K, E, out.data_ptr(), dt, addr(work), stream.handle)
                : hq_grouped_gemm_nvfp4(q, s, g, w, t, h, o, M, N, K, E, out.data_ptr(), dt, addr(work), stream.handle);
    });
    return wrap(out);
  });
}

// (gq, gs, g_sg, xq, xs, x_sg, offsets, out, out_dtype, stream)
template <bool MX>
PyObject* grouped_wgrad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&] {
    const at::Tensor &gq = codes(a[0], 2, "gq"), &xq = codes(a[3], 2, "xq");
    const at::Tensor* off = tensor(a[6]);
    if (!off || off->dim() != 1 || off->size(0) < 1) throw Refused("offsets must be a 1-D int32 tensor of E + 1 values");
    const int index = static_cast<int>(gq.get_device());
    const int64_t N = gq.size(0), T = 2 * gq.size(1), K = xq.size(0), E = off->size(0) - 1, block = MX ? 32 : 16;
    const auto* q = at_given<uint8_t>(a[0], {N, T / 2}, at::kByte, index, "gq");
    const auto* s = at_given<uint8_t>(a[1], {tiles_bytes(N, T / block)}, at::kByte, index, "gs");
    const auto* g = MX ? nullptr : at_given<float>(a[2], {1}, at::kFloat, index, "g_sg");
    const auto* x = at_given<uint8_t>(a[3], {K, T / 2}, at::kByte, index, "xq");
    const auto* t = at_given<uint8_t>(a[4], {tiles_bytes(K, T / block)}, at::kByte, index, "xs");
    const auto* h = MX ? nullptr : at_given<float>(a[5], {1}, at::kFloat, index, "x_sg");
    const auto* o = at_given<int32_t>(a[6], {E + 1}, at::kInt, index, "offsets");
    const Stream stream(a[9], index);
    const at::Tensor out = output(a[7], a[8], {E, N, K}, gq, stream);
    run(index, MX ? "hq_grouped_wgrad_mxfp4" : "hq_grouped_wgrad_nvfp4", [&] {
      const hq_dtype dt = dtype_of(out.scalar_type());
      return MX ? hq_grouped_wgrad_mxfp4(q, s, x, t, o, T, N, K, E, out.data_ptr(), dt, stream.handle)
                : hq_grouped_wgrad_nvfp4(q, s, g, x, t, h, o, T, N, K, E, out.data_ptr(), dt, stream.handle);
    });
    return wrap(out);
  });
}

// (xq, xs, x_sg, wq, ws, w_sg, x, lora_a, lora_b, scaling, row_adapter, out, out_dtype, stream)
template <bool MX>
PyObject* lora_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&] {
    const at::Tensor &xq = codes(a[0], 2, "xq"), &wq = codes(a[3], 2, "wq");
    const int index = static_cast<int>(xq.get_device());
    const int64_t M = xq.size(0), K = 2 * xq.size(1), N = wq.size(0), block = MX ? 32 : 16;
    const at::Tensor *x = tensor(a[6]), *la = tensor(a[7]);
    if (!x || x->sizes() != Shape({M, K}) || x->scalar_type() != at::kBFloat16 || !x->is_cuda() ||
        x->get_device() != index || x->stride(1) != 1)
      throw Refused("x must be a bfloat16 tensor of shape " + shape_text({M, K}) + " on cuda:" + std::to_string(index) +
                    " with contiguous rows");
    if (!la || la->dim() != 3) throw Refused("lora_a must be [adapters, R, K]");
    const int64_t count = la->size(0), R = la->size(1);
    const auto* q = at_given<uint8_t>(a[0], {M, K / 2}, at::kByte, index, "xq");
    const auto* s = at_given<uint8_t>(a[1], {M, K / block}, at::kByte, index, "xs");
    const auto* g = MX ? nullptr : at_given<float>(a[2], {1}, at::kFloat, index, "x_sg");
    const auto* w = at_given<uint8_t>(a[3], {N, K / 2}, at::kByte, index, "wq");
    const auto* t = at_given<uint8_t>(a[4], {tiles_bytes(N, K / block)}, at::kByte, index, "ws");
    const auto* h = MX ? nullptr : at_given<float>(a[5], {1}, at::kFloat, index, "w_sg");
    const auto* pa = at_given<void>(a[7], {count, R, K}, at::kBFloat16, index, "lora_a");
    const auto* pb = at_given<void>(a[8], {count, N, R}, at::kBFloat16, index, "lora_b");
    const auto* sc = at_given<float>(a[9], {count}, at::kFloat, index, "scaling");
    const auto* id = at_given<int32_t>(a[10], {M}, at::kInt, index, "row_adapter");
    const int64_t ldx = M > 1 ? x->stride(0) : K;
    const Stream stream(a[13], index);
    const at::Tensor out = output(a[11], a[12], {M, N}, xq, stream);
    const at::Tensor work = workspace(hq_lora_gemm_workspace_bytes(M, N, K, R), xq, stream);
    run(index, MX ? "hq_lora_gemm_mxfp4" : "hq_lora_gemm_nvfp4", [&] {
      const hq_dtype dt = dtype_of(out.scalar_type());
      const void* px = x->const_data_ptr();
      return MX ? hq_lora_gemm_mxfp4(q, s, w, t, px, ldx, pa, pb, sc, id, M, N, K, count, R, out.data_ptr(), dt,
                                     addr(work), stream.handle)
                : hq_lora_gemm_nvfp4(q, s, g, w, t, h, px, ldx, pa, pb, sc, id, M, N, K, count, R, out.data_ptr(), dt,
                                     addr(work), stream.handle);
    });
    return wrap(out);
  });
}

// (xq, x_scales, wq, w_scales, out, out_dtype, stream)
PyObject* gemm_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const at::Tensor &xq = cuda_tensor(a[0], "xq"), &wq = cuda_tensor(a[2], "wq");
    if (xq.dim() != 2 || wq.dim() != 2) throw Refused("xq must be [M, K] and wq [N, K]");
    const int index = static_cast<int>(xq.get_device());
    const int64_t M = xq.size(0), K = xq.size(1), N = wq.size(0);
    const auto* x = at_given<int8_t>(a[0], {M, K}, at::kChar, index, "xq");
    const auto* xs = at_given<float>(a[1], {M}, at::kFloat, index, "x_scales");
    const auto* w = at_given<int8_t>(a[2], {N, K}, at::kChar, index, "wq");
    const auto* ws = at_given<float>(a[3], {N}, at::kFloat, index, "w_scales");
    const Stream stream(a[6], index);
    const at::Tensor out = output(a[4], a[5], {M, N}, xq, stream);
    run(index, "hq_gemm_int8", [&] {
      return hq_gemm_int8(x, xs, w, ws, M, N, K, out.data_ptr(), dtype_of(out.scalar_type()), stream.handle);
    });
    return wrap(out);
  });
}

// ---- the paged cache -------------------------------------------------------------------------------

long whole(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  return v;
}

// uint8 [pages, kv_heads, page_size / 16, 18 D]
struct Cache {
  const at::Tensor& t;
  int index;
  int64_t pages, kv_heads, page_size, D;
  explicit Cache(PyObject* o) : t(cuda_tensor(o, "cache")) {
    if (t.dim() != 4 || t.scalar_type() != at::kByte || !t.is_contiguous() || t.size(3) % 18 != 0)
      throw Refused("cache must be a contiguous uint8 tensor [pages, kv_heads, page_size / 16, 18 * D]");
    index = static_cast<int>(t.get_device());
    pages = t.size(0), kv_heads = t.size(1), page_size = 16 * t.size(2), D = t.size(3) / 18;
  }
};

// [T, heads, D] with contiguous heads; ld: elements between tokens.
struct Heads {
  const at::Tensor* t;
  int64_t ld;
  Heads(PyObject* o, int64_t tokens, int64_t heads, const Cache& cache, const char* name) : t(tensor(o)) {
    if (!t || t->dim() != 3 || (tokens >= 0 && t->size(0) != tokens) || (heads >= 0 && t->size(1) != heads) ||
        t->size(2) != cache.D || !supported(t->scalar_type()) || !t->is_cuda() || t->get_device() != cache.index ||
        t->stride(2) != 1 || (t->size(1) > 1 && t->stride(1) != cache.D))
      throw Refused(std::string(name) + " must be a bfloat16 or float32 tensor [T, " +
                    (heads >= 0 ? std::to_string(heads) : std::string("heads")) + ", " + std::to_string(cache.D) +
                    "] on cuda:" + std::to_string(cache.index) + " with contiguous heads");
    ld = t->size(0) > 1 ? t->stride(0) : t->size(1) * cache.D;
  }
  // `out`, contiguous, reaches into what lies between its first and last element.
  bool meets(const at::Tensor& out) const {
    if (t->numel() == 0 || out.numel() == 0) return false;
    const auto *a = static_cast<const char*>(t->const_data_ptr()), *b = static_cast<const char*>(out.const_data_ptr());
    const int64_t span = (t->size(0) - 1) * ld + t->size(1) * t->size(2);
    return a < b + out.numel() * out.element_size() && b < a + span * t->element_size();
  }
};

// (q, k, v, cos, sin, positions, slots, kv_amax, cache, group, interleaved, q_out, stream)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const Cache cache(a[8]);
    const Heads k(a[1], -1, cache.kv_heads, cache, "k");
    const int64_t T = k.t->size(0);
    const Heads v(a[2], T, cache.kv_heads, cache, "v");
    const at::ScalarType type = k.t->scalar_type();
    const void* pq = nullptr;
    int64_t ld_q = 0, heads = 0;
    if (a[0] != Py_None) {
      const Heads q(a[0], T, -1, cache, "q");
      if (q.t->scalar_type() != type) throw Refused("q, k and v must be of one type");
      pq = q.t->const_data_ptr(), ld_q = q.ld, heads = q.t->size(1);
    }
    if (v.t->scalar_type() != type) throw Refused("q, k and v must be of one type");
    const float *cos = nullptr, *sin = nullptr;
    const int32_t* positions = nullptr;
    int64_t rows = 0, rotary = 0;
    if (a[3] != Py_None || a[4] != Py_None || a[5] != Py_None) {
      const at::Tensor* c = tensor(a[3]);
      if (!c || c->dim() != 2) throw Refused("cos, sin and positions are given together; cos must be [rows, rotary / 2]");
      rows = c->size(0), rotary = 2 * c->size(1);
      cos = at_given<float>(a[3], {rows, rotary / 2}, at::kFloat, cache.index, "cos");
      sin = at_given<float>(a[4], {rows, rotary / 2}, at::kFloat, cache.index, "sin");
      positions = at_given<int32_t>(a[5], {T}, at::kInt, cache.index, "positions");
    }
    const auto* slots = at_given<int64_t>(a[6], {T}, at::kLong, cache.index, "slots");
    const auto* amax = at_given<float>(a[7], {2}, at::kFloat, cache.index, "kv_amax");
    const int group = static_cast<int>(std::min(std::max(whole(a[9]), -1l), 257l));  // (others: refused by the library)
    const int pairs = PyObject_IsTrue(a[10]);
    if (pairs < 0) throw PythonError();
    const Stream stream(a[12], cache.index);
    at::Tensor out;
    if (a[0] == Py_None) {
      if (a[11] != Py_None) throw Refused("q_out without q");
    } else {
      out = a[11] == Py_None ? empty({T, heads, cache.D}, at::kBFloat16, cache.t, stream)
                             : given(a[11], {T, heads, cache.D}, at::kBFloat16, cache.index, "q_out");
      if (a[11] != Py_None && (k.meets(out) || v.meets(out) || Heads(a[0], T, -1, cache, "q").meets(out)))
        throw Refused("q_out may not overlap q, k or v");
    }
    run(cache.index, "hq_kv_append_nvfp4", [&] {
      return hq_kv_append_nvfp4(pq, ld_q, k.t->const_data_ptr(), k.ld, v.t->const_data_ptr(), v.ld, dtype_of(type), T, heads,
                                cache.kv_heads, cache.D, cos, sin, rows, rotary, pairs, positions, slots, group, amax,
                                addr(out), static_cast<uint8_t*>(cache.t.data_ptr()), cache.pages, cache.page_size,
                                stream.handle);
    });
    return wrap(out);
  });
}

// (cache, slots, kv_amax, group, out_dtype, k, v, stream)
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&] {
    const Cache cache(a[0]);
    const at::Tensor* s = tensor(a[1]);
    if (!s || s->dim() != 1) throw Refused("slots must be a 1-D int64 tensor");
    const int64_t T = s->size(0);
    const auto* slots = at_given<int64_t>(a[1], {T}, at::kLong, cache.index, "slots");
    const auto* amax = at_given<float>(a[2], {2}, at::kFloat, cache.index, "kv_amax");
    const int group = static_cast<int>(std::min(std::max(whole(a[3]), -1l), 257l));
    const Stream stream(a[7], cache.index);
    const at::Tensor k = output(a[5], a[4], {T, cache.kv_heads, cache.D}, cache.t, stream);
    const at::Tensor v = output(a[6], a[4], {T, cache.kv_heads, cache.D}, cache.t, stream);
    if (k.scalar_type() != v.scalar_type()) throw Refused("k and v must be of one type");
    run(cache.index, "hq_kv_read_nvfp4", [&] {
      return hq_kv_read_nvfp4(static_cast<const uint8_t*>(cache.t.const_data_ptr()), cache.pages, cache.page_size,
                              cache.kv_heads, cache.D, slots, T, amax, group, k.data_ptr(), v.data_ptr(),
                              dtype_of(k.scalar_type()), stream.handle);
    });
    return tuple({wrap(k), wrap(v)});
  });
}

// (q, cache, page_table, kv_len, q_start, kv_amax, scale, group, window, max_q, out, return_lse, stream)
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const Cache cache(a[1]);
    const Heads q(a[0], -1, -1, cache, "q");
    if (q.t->scalar_type() != at::kBFloat16) throw Refused("q must be bfloat16");
    const int64_t T = q.t->size(0), heads = q.t->size(1);
    const at::Tensor* table = tensor(a[2]);
    if (!table || table->dim() != 2 || table->scalar_type() != at::kInt || !table->is_cuda() ||
        table->get_device() != cache.index || (table->size(1) > 1 && table->stride(1) != 1))
      throw Refused("page_table must be an int32 tensor [S, pages] on cuda:" + std::to_string(cache.index) +
                    " with contiguous rows");
    const int64_t S = table->size(0), pages = table->size(1), ld = S > 1 ? table->stride(0) : pages;
    const auto* lens = at_given<int32_t>(a[3], {S}, at::kInt, cache.index, "kv_len");
    const auto* starts = at_given<int32_t>(a[4], {S + 1}, at::kInt, cache.index, "q_start");
    const auto* amax = at_given<float>(a[5], {2}, at::kFloat, cache.index, "kv_amax");
    const double scale = PyFloat_AsDouble(a[6]);
    if (scale == -1.0 && PyErr_Occurred()) throw PythonError();
    const int group = static_cast<int>(std::min(std::max(whole(a[7]), -1l), 257l));
    const long window = whole(a[8]), max_q = whole(a[9]);
    if (window < 0) throw Refused("window must be 0 (none) or positive");
    const int with_lse = PyObject_IsTrue(a[11]);
    if (with_lse < 0) throw PythonError();
    const Stream stream(a[12], cache.index);
    const at::Tensor out = a[10] == Py_None ? empty({T, heads, cache.D}, at::kBFloat16, cache.t, stream)
                                            : given(a[10], {T, heads, cache.D}, at::kBFloat16, cache.index, "out");
    if (a[10] != Py_None && q.meets(out)) throw Refused("out may not overlap q");
    at::Tensor lse;
    if (with_lse) lse = empty({T, heads}, at::kFloat, cache.t, stream);
    const at::Tensor work = workspace(hq_kv_attention_workspace_bytes(heads, cache.kv_heads, cache.D, T, max_q < 0 ? T : max_q), cache.t, stream);
    run(cache.index, "hq_kv_attention_nvfp4", [&] {
      return hq_kv_attention_nvfp4(q.t->const_data_ptr(), q.ld, T, heads, static_cast<const uint8_t*>(cache.t.const_data_ptr()),
                                   cache.pages, cache.page_size, cache.kv_heads, cache.D,
                                   static_cast<const int32_t*>(table->const_data_ptr()), ld, pages, lens, starts, S,
                                   max_q < 0 ? T : max_q, amax, static_cast<float>(scale), window, group, out.data_ptr(),
                                   static_cast<float*>(addr(lse)), addr(work), stream.handle);
    });
    return with_lse ? tuple({wrap(out), wrap(lse)}) : wrap(out);
  });
}

// ---- norms ------------------------------------------------------------------------------------------

const at::Tensor& norm_input(PyObject* o, const char* name) {
  const at::Tensor& t = cuda_tensor(o, name);
  if (t.dim() != 2 || !supported(t.scalar_type()))
    throw Refused(std::string(name) + " must be a 2-D float32 or bfloat16 tensor [M, D]");
  return t;
}

// A tensor shaped and typed like `like`, rows contiguous, or absent.
struct Rows {
  const void* p = nullptr;
  int64_t ld;
  Rows(PyObject* o, const at::Tensor& like, const char* name) {
    ld = like.size(1);
    if (o == Py_None) return;
    const at::Tensor* t = tensor(o);
    if (!t || t->sizes() != like.sizes() || t->scalar_type() != like.scalar_type() || !t->is_cuda() ||
        t->get_device() != like.get_device() || t->stride(1) != 1)
      throw Refused(std::string(name) + " must be a " + type_text(like.scalar_type()) + " tensor of shape " +
                    shape_text(like.sizes()) + " on cuda:" + std::to_string(like.get_device()) +
                    " with contiguous rows");
    p = t->const_data_ptr();
    if (t->size(0) > 1) ld = t->stride(0);
  }
};

struct NormParams {
  const void *w_post = nullptr, *w_pre = nullptr, *gate = nullptr;
  at::ScalarType type = at::kFloat;
  hq_gate_kind kind = HQ_GATE_NONE;
  int64_t ld_gate = 0;

  NormParams(const at::Tensor& h, bool has_y, PyObject* post_w, PyObject* g, PyObject* pre_w, bool post, bool pre) {
    const int64_t M = h.size(0), D = h.size(1);
    const int index = static_cast<int>(h.get_device());
    bool typed = false;
    auto vector = [&](PyObject* o, Shape shape, const char* name) -> const void* {
      if (o == Py_None) return nullptr;
      const at::Tensor* t = tensor(o);
      if (!t || !supported(t->scalar_type())) throw Refused(std::string(name) + " must be a float32 or bfloat16 tensor");
      if (!typed) type = t->scalar_type();  // one type for all of them
      typed = true;
      return given(o, shape, type, index, name).const_data_ptr();
    };
    if (post_w != Py_None && !post) throw Refused("w_post without a post norm");
    if (pre_w != Py_None && !pre) throw Refused("w_pre without pre_norm");
    w_post = vector(post_w, {D}, "w_post");
    w_pre = vector(pre_w, {D}, "w_pre");
    if (g == Py_None) return;
    if (!has_y) throw Refused("gate without y");
    const at::Tensor* t = tensor(g);
    if (!t) throw Refused("gate must be a tensor");
    if (t->dim() == 1) {
      kind = HQ_GATE_CHANNEL;
      gate = vector(g, {D}, "gate");
    } else if (t->sizes() == Shape({M, 1})) {
      kind = HQ_GATE_TOKEN;
      gate = vector(g, {M, 1}, "gate [M, 1]");
    } else {
      kind = HQ_GATE_FULL;
      const Rows r(g, h, "gate ([D], [M, 1] or [M, D])");
      gate = r.p;
      ld_gate = r.ld;
    }
  }
};

bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw PythonError();
  return r;
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError();
  return static_cast<float>(v);
}

// (h, y, w_post, gate, w_pre, alpha, eps, post_norm, pre_norm, amax_group, h_out, n, stream)
PyObject* block_norm(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 13, [&] {
    const at::Tensor& h = norm_input(a[0], "h");
    const int64_t M = h.size(0), D = h.size(1);
    const int index = static_cast<int>(h.get_device());
    const at::ScalarType type = h.scalar_type();
    const bool has_y = a[1] != Py_None, post = truth(a[7]) && has_y, pre = truth(a[8]);
    const Rows rh(a[0], h, "h"), ry(a[1], h, "y");
    const NormParams p(h, has_y, a[2], a[3], a[4], post, pre);
    const float alpha = number(a[5]), eps = number(a[6]);
    int group = 0;
    if (a[9] != Py_None) {
      const long v = PyLong_AsLong(a[9]);
      if (v == -1 && PyErr_Occurred()) throw PythonError();
      group = v < 0 || v > 256 ? -1 : static_cast<int>(v);  // (-1: refused by the library)
    }
    const Stream stream(a[12], index);
    at::Tensor h_out, n, r_post, r_pre, amax;
    if (has_y) h_out = a[10] == Py_None ? empty({M, D}, type, h, stream) : given(a[10], {M, D}, type, index, "h_out");
    if (pre) n = a[11] == Py_None ? empty({M, D}, type, h, stream) : given(a[11], {M, D}, type, index, "n");
    if (post) r_post = empty({M}, at::kFloat, h, stream);
    if (pre) r_pre = empty({M}, at::kFloat, h, stream);
    if (a[9] != Py_None) amax = empty({1}, at::kFloat, h, stream);
    run(index, "hq_block_norm", [&] {
      return hq_block_norm(rh.p, rh.ld, ry.p, ry.ld, dtype_of(type), M, D, p.w_post, p.w_pre, dtype_of(p.type), p.kind,
                           p.gate, p.ld_gate, (post ? HQ_NORM_POST : 0) | (pre ? HQ_NORM_PRE : 0), alpha, eps,
                           addr(h_out), addr(n), static_cast<float*>(addr(r_post)), static_cast<float*>(addr(r_pre)),
                           group, static_cast<float*>(addr(amax)), stream.handle);
    });
    PyObject* first = has_y ? wrap(h_out) : Py_NewRef(a[0]);
    return amax.defined() ? tuple({first, wrap(n), wrap(r_post), wrap(r_pre), wrap(amax)})
                          : tuple({first, wrap(n), wrap(r_post), wrap(r_pre)});
  });
}

// (dh_out, dn, h_out, y, w_post, gate, w_pre, r_post, r_pre, alpha, post_norm, pre_norm, stream)
PyObject* block_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded(count, 13, [&] {
    const at::Tensor& h = norm_input(a[2], "h_out");
    const int64_t M = h.size(0), D = h.size(1);
    const int index = static_cast<int>(h.get_device());
    const at::ScalarType type = h.scalar_type();
    const bool has_y = a[3] != Py_None, post = truth(a[10]) && has_y, pre = truth(a[11]);
    if (pre && (a[1] == Py_None || a[8] == Py_None)) throw Refused("dn and r_pre are needed with pre_norm");
    if (!pre && (a[1] != Py_None || a[0] == Py_None))
      throw Refused("without pre_norm there is no dn, and dh_out is needed");
    if (post && a[7] == Py_None) throw Refused("r_post is needed with post_norm");
    const Rows rd(a[0], h, "dh_out"), rn(a[1], h, "dn"), rh(a[2], h, "h_out"), ry(a[3], h, "y");
    const NormParams p(h, has_y, a[4], a[5], a[6], post, pre);
    const float* r_post = post ? at_given<float>(a[7], {M}, at::kFloat, index, "r_post") : nullptr;
    const float* r_pre = pre ? at_given<float>(a[8], {M}, at::kFloat, index, "r_pre") : nullptr;
    const float alpha = number(a[9]);
    const Stream stream(a[12], index);
    at::Tensor dh = empty({M, D}, type, h, stream), dy, dw_post, dw_pre, dgate;
    if (has_y) dy = empty({M, D}, type, h, stream);
    if (p.w_post) dw_post = empty({D}, at::kFloat, h, stream);
    if (p.w_pre) dw_pre = empty({D}, at::kFloat, h, stream);
    if (p.kind != HQ_GATE_NONE)
      dgate = empty(tensor(a[5])->sizes(), p.kind == HQ_GATE_FULL ? type : at::kFloat, h, stream);
    const at::Tensor work = workspace(hq_block_norm_bwd_workspace_bytes(M, D), h, stream);
    run(index, "hq_block_norm_bwd", [&] {
      return hq_block_norm_bwd(rd.p, rd.ld, rn.p, rn.ld, rh.p, rh.ld, ry.p, ry.ld, dtype_of(type), M, D, p.w_post,
                               p.w_pre, dtype_of(p.type), p.kind, p.gate, p.ld_gate,
                               (post ? HQ_NORM_POST : 0) | (pre ? HQ_NORM_PRE : 0), r_post, r_pre, alpha, addr(dh),
                               addr(dy), static_cast<float*>(addr(dw_post)), addr(dgate),
                               static_cast<float*>(addr(dw_pre)), addr(work), stream.handle);
    });
    return tuple({wrap(dh), wrap(dy), wrap(dw_post), wrap(dgate), wrap(dw_pre)});
  });
}

#define HQ_METHOD(name, function) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(function)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    HQ_METHOD("grouped_gemm_nvfp4", grouped_gemm<false>),
    HQ_METHOD("grouped_gemm_mxfp4", grouped_gemm<true>),
    HQ_METHOD("grouped_wgrad_nvfp4", grouped_wgrad<false>),
    HQ_METHOD("grouped_wgrad_mxfp4", grouped_wgrad<true>),
    HQ_METHOD("lora_gemm_nvfp4", lora_gemm<false>),
    HQ_METHOD("lora_gemm_mxfp4", lora_gemm<true>),
    HQ_METHOD("gemm_int8", gemm_int8),
    HQ_METHOD("kv_append", kv_append),
    HQ_METHOD("kv_read", kv_read),
    HQ_METHOD("kv_attention", kv_attention),
    HQ_METHOD("block_norm", block_norm),
    HQ_METHOD("block_norm_bwd", block_norm_bwd),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", "The products, norms and caches of libhq over torch tensors.", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls(void) { return PyModule_Create(&module); }
