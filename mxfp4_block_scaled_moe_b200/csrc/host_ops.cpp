// The host side of the operators whose kernels take a few microseconds: argument checks on torch
// tensors, the outputs' allocation and the C ABI call, as one native step. The same in Python
// took 8 to 14 us a call (attribute reads, ctypes' argument conversion), longer than most of
// the kernels. Argument marshalling only: the module is handed the C ABI's entry points by
// binding.py and calls them on the tensors' device and its current stream.
//
// Every function takes positional arguments, all of them; binding.py gives them their names,
// defaults and documentation. A tensor that does not fit raises ValueError; a refusal by the
// C ABI goes through the callable given to setup(), which raises.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>
#include <stdexcept>
#include <string>
#include <vector>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mxfp4_moe.h"

namespace {

using at::Tensor;

struct TypeError : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct PythonError {};   // the Python error is set already

// ------------------------------------------------------------------ entry points ---
decltype(&rmsnorm_residual) p_norm;
decltype(&fp8_linear_fused) p_linear;
decltype(&mxfp4_kv_append) p_append;
decltype(&mxfp4_kv_attention) p_attention;
decltype(&mxfp4_kv_attention_workspace) p_workspace;
decltype(&mxfp4_dequantize) p_dequantize;
PyObject* g_fail;   // g_fail(rc, name) raises

void check_rc(int rc, const char* name) {
  if (rc == MXMOE_OK) return;
  PyObject* r = PyObject_CallFunction(g_fail, "is", rc, name);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) throw std::runtime_error(std::string(name) + " failed");
  throw PythonError();
}

// ------------------------------------------------------------------- arguments -----
const Tensor* optional(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw TypeError(std::string(name) + " must be a torch.Tensor");
  return &THPVariable_Unpack(o);
}
const Tensor& tensor(PyObject* o, const char* name) {
  const Tensor* t = optional(o, name);
  if (!t) throw TypeError(std::string(name) + " must be a torch.Tensor");
  return *t;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError();
  return v;
}
int whole(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  if (v < INT32_MIN || v > INT32_MAX) throw std::invalid_argument(std::string(name) + " is out of range");
  return static_cast<int>(v);
}
int size32(int64_t v, const char* name) {
  if (v > INT32_MAX) throw std::invalid_argument(std::string(name) + " is out of range");
  return static_cast<int>(v);
}

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

int device_of(const Tensor& t, const char* name) {
  if (!t.is_cuda()) throw std::invalid_argument(std::string(name) + " must be a CUDA tensor");
  return static_cast<int>(t.get_device());
}

[[noreturn]] void refuse(const Tensor& t, at::ScalarType type, const at::IntArrayRef* shape, int dev, const char* name) {
  const std::string n(name);
  if (!t.is_cuda()) throw std::invalid_argument(n + " must be a CUDA tensor");
  if (t.get_device() != dev)
    throw std::invalid_argument(n + " is on cuda:" + std::to_string(t.get_device()) + ", the other tensors on cuda:" +
                                std::to_string(dev));
  if (t.scalar_type() != type)
    throw std::invalid_argument(n + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
  if (shape && t.sizes() != *shape)
    throw std::invalid_argument(n + " must have shape " + text(*shape) + ", got " + text(t.sizes()));
  throw std::invalid_argument(n + " must be contiguous");
}

// device pointer of a dense tensor of that type, shape and device
template <class T>
T* dense(const Tensor& t, at::ScalarType type, at::IntArrayRef shape, int dev, const char* name) {
  if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev || t.sizes() != shape || !t.is_contiguous())
    refuse(t, type, &shape, dev, name);
  return static_cast<T*>(t.data_ptr());
}
template <class T>
T* dense(const Tensor* t, at::ScalarType type, at::IntArrayRef shape, int dev, const char* name) {
  return t ? dense<T>(*t, type, shape, dev, name) : nullptr;
}

// a dense tensor of that type and device, of any shape
void check_dense(const Tensor& t, at::ScalarType type, int dev, const char* name) {
  if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
    refuse(t, type, nullptr, dev, name);
}
void check_count(const Tensor& t, int64_t count, const char* name) {
  if (t.numel() != count)
    throw std::invalid_argument(std::string(name) + " must have " + std::to_string(count) + " elements, got " + text(t.sizes()));
}

void check_bf16(const Tensor& t, int dev, const char* name) {
  if (t.scalar_type() != at::kBFloat16 || !t.is_cuda() || t.get_device() != dev)
    refuse(t, at::kBFloat16, nullptr, dev, name);
}

// the row stride of a bf16 tensor (..., H): a dense tensor of any rank, or two-dimensional rows
// cut from wider ones
int64_t row_stride(const Tensor& t, int64_t H, int dev, const char* name) {
  check_bf16(t, dev, name);
  if (t.is_contiguous()) return H;
  if (t.dim() != 2 || t.stride(1) != 1)
    throw std::invalid_argument(std::string(name) + " must be contiguous, or two-dimensional with contiguous rows");
  return t.stride(0);
}

// the token stride of a bf16 tensor (..., heads, D): heads dense, tokens one stride apart
int64_t token_stride(const Tensor& t, int dev, const char* name) {
  check_bf16(t, dev, name);
  const auto size = t.sizes(), stride = t.strides();
  const int64_t nd = t.dim(), row = size[nd - 2] * size[nd - 1];
  if (t.is_contiguous()) return row;
  if (stride[nd - 1] != 1 || (size[nd - 2] != 1 && stride[nd - 2] != size[nd - 1]))
    throw std::invalid_argument(std::string(name) + ": each token's heads must be dense");
  int64_t step = -1, n = 1;
  for (int64_t d = nd - 3; d >= 0; --d) {
    if (size[d] == 1) continue;
    if (step < 0)
      step = stride[d];
    else if (stride[d] != step * n)
      throw std::invalid_argument(std::string(name) + ": the tokens must be one stride apart");
    n *= size[d];
  }
  return step < 0 ? row : step;
}

Tensor fresh(at::IntArrayRef shape, const Tensor& like, at::ScalarType type) {
  return at::empty(shape, like.options().dtype(type).requires_grad(false).memory_format(at::MemoryFormat::Contiguous));
}

// `call(stream)` with the tensors' device current
template <class Call>
void on_device(int dev, const char* name, Call call) {
  c10::cuda::OptionalCUDAGuard guard;
  if (c10::cuda::current_device() != dev) guard.set_index(static_cast<c10::DeviceIndex>(dev));
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = call(stream);
  Py_END_ALLOW_THREADS
  check_rc(rc, name);
}

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

// Runs a function's body; C++ exceptions end here.
template <class Body>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, Body body) {
  try {
    if (got != want) throw TypeError("takes " + std::to_string(want) + " arguments, got " + std::to_string(got));
    return body();
  } catch (const PythonError&) {
  } catch (const TypeError& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

// --------------------------------------------------------------------- operators ---

// x, weight, residual, eps, act_scale, sum_out, q, y, fp8 -> (y, q, scale, sum)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const Tensor& x = tensor(a[0], "x");
    const Tensor *residual = optional(a[2], "residual"), *given_sum = optional(a[5], "sum_out"),
                 *given_q = optional(a[6], "q"), *given_y = optional(a[7], "y");
    const bool fp8 = a[8] == Py_True;
    const int dev = device_of(x, "x");
    if (x.dim() < 1) throw std::invalid_argument("x must have at least one dimension");
    const auto shape = x.sizes();
    const int64_t H = shape.back(), T = H ? x.numel() / H : 0;
    const int64_t ldx = row_stride(x, H, dev, "x");
    const uint16_t* w = dense<uint16_t>(tensor(a[1], "weight"), at::kBFloat16, {H}, dev, "weight");
    const uint16_t* r = nullptr;
    int64_t ldr = H;
    Tensor sum, q, y, scale;
    if (residual) {
      if (residual->sizes() != shape)
        throw std::invalid_argument("residual must have x's shape " + text(shape) + ", got " + text(residual->sizes()));
      ldr = row_stride(*residual, H, dev, "residual");
      r = static_cast<const uint16_t*>(residual->data_ptr());
      if (given_sum) dense<void>(*given_sum, at::kBFloat16, shape, dev, "sum_out");
      sum = given_sum ? *given_sum : fresh(shape, x, at::kBFloat16);
    } else if (given_sum) {
      throw std::invalid_argument("sum_out goes with a residual");
    }
    if (given_y) dense<void>(*given_y, at::kBFloat16, shape, dev, "y");
    if (given_y || !fp8) y = given_y ? *given_y : fresh(shape, x, at::kBFloat16);
    float s = 0.f;
    const bool fixed = a[4] != Py_None;
    if (fp8) {
      if (given_q) dense<void>(*given_q, at::kByte, shape, dev, "q");
      q = given_q ? *given_q : fresh(shape, x, at::kByte);
      if (fixed) s = static_cast<float>(number(a[4]));
      else scale = fresh(shape.slice(0, shape.size() - 1), x, at::kFloat);
    }
    const float eps = static_cast<float>(number(a[3]));
    const int T32 = size32(T, "T"), H32 = size32(H, "H");
    on_device(dev, "rmsnorm_residual", [&](void* st) {
      const auto ptr = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
      return p_norm(static_cast<const uint16_t*>(x.data_ptr()), ldx, r, ldr, w, eps, T32, H32,
                    static_cast<uint16_t*>(ptr(sum)), static_cast<uint16_t*>(ptr(y)), static_cast<uint8_t*>(ptr(q)),
                    static_cast<float*>(ptr(scale)), fp8 && fixed ? &s : nullptr, st);
    });
    return Py_BuildValue("(NNNN)", wrap(y), wrap(q), wrap(scale), wrap(sum));
  });
}

// xq, wq, s_x, s_w, bias, act, residual, out -> out
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const Tensor &xq = tensor(a[0], "xq"), &wq = tensor(a[1], "wq");
    const int dev = device_of(xq, "xq");
    if (xq.dim() != 2 || wq.dim() != 2) throw std::invalid_argument("xq and wq must be two-dimensional");
    const int64_t T = xq.size(0), K = xq.size(1), N = wq.size(0);
    const uint8_t* x = dense<uint8_t>(xq, at::kByte, {T, K}, dev, "xq");
    const uint8_t* w = dense<uint8_t>(wq, at::kByte, {N, K}, dev, "wq");
    const float *sx = nullptr, *sw = nullptr;
    float sx_all = 1.f, sw_all = 1.f;
    if (THPVariable_Check(a[2])) sx = dense<float>(tensor(a[2], "s_x"), at::kFloat, {T}, dev, "s_x");
    else sx_all = static_cast<float>(number(a[2]));
    if (THPVariable_Check(a[3])) sw = dense<float>(tensor(a[3], "s_w"), at::kFloat, {N}, dev, "s_w");
    else sw_all = static_cast<float>(number(a[3]));
    const float* bias = dense<float>(optional(a[4], "bias"), at::kFloat, {N}, dev, "bias");
    const int act = whole(a[5], "act");
    const uint16_t* residual = dense<uint16_t>(optional(a[6], "residual"), at::kBFloat16, {T, N}, dev, "residual");
    const Tensor* given = optional(a[7], "out");
    if (given) dense<void>(*given, at::kBFloat16, {T, N}, dev, "out");
    const Tensor out = given ? *given : fresh({T, N}, xq, at::kBFloat16);
    const int T32 = size32(T, "T"), K32 = size32(K, "K"), N32 = size32(N, "N");
    on_device(dev, "fp8_linear_fused", [&](void* st) {
      return p_linear(x, T32, K32, w, N32, sx, sx_all, sw, sw_all, bias, act, residual,
                      static_cast<uint16_t*>(out.data_ptr()), st);
    });
    return wrap(out);
  });
}

struct Cache {
  uint8_t *k_blocks, *k_scales, *v_blocks, *v_scales;
  int64_t pages;
  int Hkv, page_size, D;
  Cache(PyObject* const* a, int dev) {
    const Tensor& kb = tensor(a[0], "k_blocks");
    if (kb.dim() != 4)
      throw std::invalid_argument("k_blocks must be (num_pages, Hkv, page_size, D/2), got " + text(kb.sizes()));
    const auto shape = kb.sizes();
    const int64_t sc[4] = {shape[0], shape[1], shape[2], shape[3] / 16};
    k_blocks = dense<uint8_t>(kb, at::kByte, shape, dev, "k_blocks");
    k_scales = dense<uint8_t>(tensor(a[1], "k_scales"), at::kByte, sc, dev, "k_scales");
    v_blocks = dense<uint8_t>(tensor(a[2], "v_blocks"), at::kByte, shape, dev, "v_blocks");
    v_scales = dense<uint8_t>(tensor(a[3], "v_scales"), at::kByte, sc, dev, "v_scales");
    pages = shape[0];
    Hkv = size32(shape[1], "Hkv");
    page_size = size32(shape[2], "page_size");
    D = size32(2 * shape[3], "D");
  }
};

// k, v, slots, k_blocks, k_scales, v_blocks, v_scales
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const int dev = device_of(k, "k");
    const Cache c(a + 3, dev);
    const int64_t T = k.dim() == 3 ? k.size(0) : -1;
    const int64_t want[3] = {T, c.Hkv, c.D};
    if (T < 0 || k.sizes() != at::IntArrayRef(want) || v.sizes() != at::IntArrayRef(want))
      throw std::invalid_argument("k and v must be (T, " + std::to_string(c.Hkv) + ", " + std::to_string(c.D) + "), got " +
                                  text(k.sizes()) + " and " + text(v.sizes()));
    const int64_t ldk = token_stride(k, dev, "k"), ldv = token_stride(v, dev, "v");
    const int64_t* slots = dense<int64_t>(tensor(a[2], "slots"), at::kLong, {T}, dev, "slots");
    const int T32 = size32(T, "T");
    on_device(dev, "mxfp4_kv_append", [&](void* st) {
      return p_append(static_cast<const uint16_t*>(k.data_ptr()), ldk, static_cast<const uint16_t*>(v.data_ptr()), ldv,
                      slots, T32, c.Hkv, c.D, c.k_blocks, c.k_scales, c.v_blocks, c.v_scales, c.pages, c.page_size, st);
    });
    Py_RETURN_NONE;
  });
}

// q, k_blocks, k_scales, v_blocks, v_scales, block_table, seq_lens, scale, window, sinks, out,
// workspace -> out
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const Tensor& q = tensor(a[0], "q");
    const int dev = device_of(q, "q");
    const Cache c(a + 1, dev);
    const auto shape = q.sizes();
    if ((shape.size() != 3 && shape.size() != 4) || shape.back() != c.D)
      throw std::invalid_argument("q must be (B, Lq, Hq, " + std::to_string(c.D) + ") or (B, Hq, " + std::to_string(c.D) +
                                  "), got " + text(shape));
    const int64_t ldq = token_stride(q, dev, "q");
    const int B = size32(shape[0], "B"), Lq = shape.size() == 4 ? size32(shape[1], "Lq") : 1,
              Hq = size32(shape[shape.size() - 2], "Hq");
    const Tensor& table = tensor(a[5], "block_table");
    if (table.dim() != 2) throw std::invalid_argument("block_table must be (B, max_pages), got " + text(table.sizes()));
    const int max_pages = size32(table.size(1), "max_pages");
    const int32_t* rows = dense<int32_t>(table, at::kInt, {B, table.size(1)}, dev, "block_table");
    const int32_t* lens = dense<int32_t>(tensor(a[6], "seq_lens"), at::kInt, {B}, dev, "seq_lens");
    const float scale = a[7] == Py_None ? 1.f / std::sqrt(static_cast<float>(c.D)) : static_cast<float>(number(a[7]));
    const int window = whole(a[8], "window");
    const float* sinks = dense<float>(optional(a[9], "sinks"), at::kFloat, {Hq}, dev, "sinks");
    const Tensor *given = optional(a[10], "out"), *given_ws = optional(a[11], "workspace");
    if (given) dense<void>(*given, at::kBFloat16, shape, dev, "out");
    if (given_ws) dense<void>(*given_ws, at::kByte, given_ws->sizes(), dev, "workspace");
    const Tensor out = given ? *given : fresh(shape, q, at::kBFloat16);
    Tensor ws = given_ws ? *given_ws : Tensor();
    if (!given_ws) {
      int64_t bytes = 0;
      c10::cuda::OptionalCUDAGuard guard;
      if (c10::cuda::current_device() != dev) guard.set_index(static_cast<c10::DeviceIndex>(dev));
      check_rc(p_workspace(B, Lq, Hq, c.Hkv, c.D, &bytes), "mxfp4_kv_attention_workspace");
      ws = fresh({bytes}, q, at::kByte);
    }
    on_device(dev, "mxfp4_kv_attention", [&](void* st) {
      return p_attention(static_cast<const uint16_t*>(q.data_ptr()), ldq, c.k_blocks, c.k_scales, c.v_blocks, c.v_scales,
                         c.pages, c.page_size, rows, max_pages, lens, sinks, B, Lq, Hq, c.Hkv, c.D, scale, window,
                         static_cast<uint16_t*>(out.data_ptr()), ws.data_ptr(), ws.numel(), st);
    });
    return wrap(out);
  });
}

// blocks, scales, out, fp32 (else bf16) -> out. scales and a given out may have any shape of the right
// number of elements. Everything is checked before the first pointer is taken.
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    const Tensor &blocks = tensor(a[0], "blocks"), &scales = tensor(a[1], "scales");
    const int dev = device_of(blocks, "blocks");
    check_dense(blocks, at::kByte, dev, "blocks");
    check_dense(scales, at::kByte, dev, "scales");
    if (blocks.dim() < 1) throw std::invalid_argument("blocks must have at least one dimension");
    const int64_t half = blocks.sizes().back(), rows = half ? blocks.numel() / half : 0;
    check_count(scales, rows * (half / 16), "scales");
    const bool f32 = a[3] == Py_True;
    const at::ScalarType type = f32 ? at::kFloat : at::kBFloat16;
    const Tensor* given = optional(a[2], "out");
    if (given) {
      check_dense(*given, type, dev, "out");
      check_count(*given, rows * 2 * half, "out");
    }
    std::vector<int64_t> shape(blocks.sizes().begin(), blocks.sizes().end());
    shape.back() = 2 * half;
    const Tensor out = given ? *given : fresh(shape, blocks, type);
    const auto *b = static_cast<const uint8_t*>(blocks.data_ptr()), *s = static_cast<const uint8_t*>(scales.data_ptr());
    on_device(dev, "mxfp4_dequantize", [&](void* st) {
      return p_dequantize(b, s, rows, 2 * half, out.data_ptr(), f32 ? MXMOE_OUT_F32 : MXMOE_OUT_BF16, st);
    });
    return wrap(out);
  });
}

// setup(fail, {entry point: address})
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 2, [&]() -> PyObject* {
    const auto address = [&](const char* name) {
      PyObject* v = PyDict_GetItemString(a[1], name);
      void* p = v ? PyLong_AsVoidPtr(v) : nullptr;
      if (!p) throw std::runtime_error(std::string("no entry point ") + name);
      return p;
    };
    p_norm = reinterpret_cast<decltype(p_norm)>(address("rmsnorm_residual"));
    p_linear = reinterpret_cast<decltype(p_linear)>(address("fp8_linear_fused"));
    p_append = reinterpret_cast<decltype(p_append)>(address("mxfp4_kv_append"));
    p_attention = reinterpret_cast<decltype(p_attention)>(address("mxfp4_kv_attention"));
    p_workspace = reinterpret_cast<decltype(p_workspace)>(address("mxfp4_kv_attention_workspace"));
    p_dequantize = reinterpret_cast<decltype(p_dequantize)>(address("mxfp4_dequantize"));
    Py_INCREF(a[0]);
    Py_XSETREF(g_fail, a[0]);
    Py_RETURN_NONE;
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<setup>("setup"),   method<norm>("norm"),           method<linear>("linear"),
                         method<append>("append"), method<attention>("attention"), method<dequantize>("dequantize"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch's C++ interface holds for one version of it: binding.py compares `built_for` with the versions that run,
// and build.py finds it in the file
const char built_for[] = "built for: " MXMOE_BUILT_FOR;

PyMODINIT_FUNC PyInit__host_ops(void) {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", built_for + sizeof("built for: ") - 1) < 0) Py_CLEAR(m);
  return m;
}
