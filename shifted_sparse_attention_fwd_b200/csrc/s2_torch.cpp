// Python binding of the serving entries, for torch tensors: checks a call's tensors, allocates its
// outputs and passes addresses to libs2attn.so. A decoding step is a few microseconds of GPU work;
// the same checks and allocations in Python take 10 us a call, here under 2.
//
// The library's functions are handed over as addresses by the Python side, which loads the library
// (bind). Wrong tensors raise ValueError before anything is allocated or launched; a status other than
// S2ATTN_OK is returned as an int, and the Python side raises it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <climits>
#include <cmath>
#include <initializer_list>
#include <optional>
#include <stdexcept>
#include <string>
#include <utility>

#include "../../include/s2attn.h"

namespace {

decltype(&s2attn_rope_append_f64) g_append = nullptr;
decltype(&s2attn_decode) g_decode = nullptr;
decltype(&s2attn_decode_workspace_size) g_decode_space = nullptr;
decltype(&s2attn_prompt_fwd) g_prompt = nullptr;

using at::Tensor;
using Sizes = std::initializer_list<int64_t>;

[[noreturn]] void refuse(const char* name, const std::string& text) {
  throw std::invalid_argument(std::string(name) + ": " + text);
}

std::string type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "bfloat16";
    case at::kFloat: return "float32";
    case at::kHalf: return "float16";
    case at::kDouble: return "float64";
    case at::kInt: return "int32";
    case at::kLong: return "int64";
    case at::kByte: return "uint8";
    default: return c10::toString(t);
  }
}

// A Python argument as a tensor; None is an undefined tensor.
const Tensor& tensor(PyObject* o, const char* name, bool may_be_none = false) {
  static const Tensor none;
  if (o == Py_None && may_be_none) return none;
  if (!THPVariable_Check(o)) refuse(name, "expected a tensor");
  return THPVariable_Unpack(o);
}

void check(const Tensor& t, const char* name, at::ScalarType type, Sizes shape, int device) {
  if (t.scalar_type() != type)
    refuse(name, "expected " + type_name(type) + ", got " + type_name(t.scalar_type()));
  if (t.sizes() != at::IntArrayRef(shape)) {
    std::string want, got;
    for (int64_t n : shape) want += (want.empty() ? "" : ", ") + std::to_string(n);
    for (int64_t n : t.sizes()) got += (got.empty() ? "" : ", ") + std::to_string(n);
    refuse(name, "expected shape (" + want + "), got (" + got + ")");
  }
  if (!t.is_cuda()) refuse(name, "expected a CUDA tensor");
  if (t.get_device() != device)
    refuse(name, "expected a tensor on CUDA device " + std::to_string(device) + ", got one on " +
                     std::to_string(t.get_device()));
}
void check_packed(const Tensor& t, const char* name, at::ScalarType type, Sizes shape, int device) {
  check(t, name, type, shape, device);
  if (!t.is_contiguous()) refuse(name, "expected a contiguous tensor");
}

// There is no backward. A graph that would end here is refused rather than cut in silence: a tensor that
// requires grad while gradients are recorded, or that carries a forward-mode tangent.
void refuse_gradients(std::initializer_list<std::pair<const Tensor*, const char*>> tensors) {
  for (const auto& [t, name] : tensors) {
    // (a tensor without autograd data, as in serving, has neither)
    if (!t->defined() || t->unsafeGetTensorImpl()->autograd_meta() == nullptr) continue;
    if (c10::GradMode::is_enabled() && t->requires_grad())
      refuse(name, "requires grad, and the serving entries have no backward (call them under torch.no_grad())");
    if (c10::AutogradState::get_tls_state().get_fw_grad_mode() && t->_fw_grad(0).defined())
      refuse(name, "has a forward-mode tangent, and the serving entries have no derivative");
  }
}

// What a call writes in place counts as changed, for a graph that holds it (tensors of inference mode keep no count).
int written(int status, std::initializer_list<const Tensor*> tensors) {
  if (status != S2ATTN_OK) return status;
  for (const Tensor* t : tensors)
    if (t->defined() && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
  return status;
}

// Shape of the tensor that gives a call its sizes.
void want_axes(const Tensor& t, const char* name, int64_t n) {
  if (t.dim() != n) refuse(name, "expected " + std::to_string(n) + " axes, got " + std::to_string(t.dim()));
  for (int64_t x : t.sizes())
    if (x > INT_MAX) refuse(name, "an axis is longer than 2^31 - 1");
}

// Row stride of a checked bf16 [rows, heads, d] tensor (strides of axes of length 1 do not count).
long long row_stride(const Tensor& t, const char* name) {
  const int64_t H = t.size(1), d = t.size(2);
  if (t.is_contiguous()) return H * d;
  if (t.stride(2) != 1 || (H > 1 && t.stride(1) != d)) refuse(name, "expected contiguous (heads, d) blocks");
  return t.size(0) > 1 ? t.stride(0) : H * d;
}
long long rows(const Tensor& t, const char* name, Sizes shape, int device) {
  check(t, name, at::kBFloat16, shape, device);
  return row_stride(t, name);
}
// {page, token} strides of a bf16 [pages, page_size, Hkv, d] cache.
void cache(const Tensor& t, const char* name, Sizes shape, int device, long long* out) {
  check(t, name, at::kBFloat16, shape, device);
  const int64_t H = t.size(2), d = t.size(3);
  if (t.is_contiguous()) {
    out[1] = H * d;
    out[0] = t.size(1) * H * d;
    return;
  }
  if (t.stride(3) != 1 || (H > 1 && t.stride(2) != d)) refuse(name, "expected contiguous (Hkv, d) blocks");
  out[1] = t.size(1) > 1 ? t.stride(1) : H * d;
  out[0] = t.size(0) > 1 ? t.stride(0) : t.size(1) * out[1];
}

Tensor empty(at::IntArrayRef shape, at::ScalarType type, int device) {
  return at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(device)),
                                std::nullopt);
}

// For the length of a call: its device and, where one is given, its stream are the current ones, so that
// what is allocated belongs to the stream that the call runs on.
struct Place {
  c10::cuda::OptionalCUDAGuard device;
  c10::cuda::OptionalCUDAStreamGuard given;
  void* stream;
  Place(int index, PyObject* handle) {
    if (index < 0) throw std::invalid_argument("expected CUDA tensors");
    if (handle == Py_None) {
      device.set_index(static_cast<c10::DeviceIndex>(index));
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
      return;
    }
    stream = PyLong_AsVoidPtr(handle);
    if (PyErr_Occurred()) throw std::invalid_argument("stream: expected a handle");
    given.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream),
                                                        static_cast<c10::DeviceIndex>(index)));
  }
};

int device_of(const Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(name, "expected a CUDA tensor");
  return static_cast<int>(t.get_device());
}

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw std::invalid_argument("expected a number");
  return x;
}

// A call of no rows has nothing to launch (the library takes at least one); its other arguments are checked as
// the library checks them.
int check_heads(int64_t Hq, int64_t Hkv, int64_t d) {
  if (Hq <= 0 || Hkv <= 0 || d <= 0 || Hq % Hkv != 0) return S2ATTN_ERR_INVALID_ARG;
  return d == 64 || d == 128 ? S2ATTN_OK : S2ATTN_ERR_UNSUPPORTED;
}
bool positive(double x) { return x > 0.0 && std::isfinite(x); }

void* data(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// What each function returns: the status if it is not OK, else the new tensors or None.
PyObject* answer(int status) {
  if (status != S2ATTN_OK) return PyLong_FromLong(status);
  Py_RETURN_NONE;
}
PyObject* answer(int status, const Tensor& a, const Tensor& b) {
  if (status != S2ATTN_OK) return PyLong_FromLong(status);
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = THPVariable_Wrap(b);
  return x && y ? Py_BuildValue("(NN)", x, y) : nullptr;
}

template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& call) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return call();
  } catch (const std::invalid_argument& e) {
    PyErr_Clear();
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    PyErr_Clear();
    PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// rope_append(fresh, q, q_rot, k, k_rot, v, k_cache, v_cache, table, lens, cu, base, pi_scale, stream):
// fresh: q_rot and k_rot are allocated here and returned.
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const bool fresh = a[0] == Py_True;
    const Tensor &q = tensor(a[1], "q", true), &k = tensor(a[3], "k"), &v = tensor(a[5], "v");
    const Tensor &kc = tensor(a[6], "k_cache"), &vc = tensor(a[7], "v_cache"), &table = tensor(a[8], "block_table");
    const Tensor &lens = tensor(a[9], "cache_lens"), &cu = tensor(a[10], "cu_seqlens", true);
    Tensor q_rot = tensor(a[2], "q_rot", true), k_rot = tensor(a[4], "k_rot", true);
    if (!fresh && q.defined() != q_rot.defined()) throw std::invalid_argument("q and q_rot go together");
    want_axes(k, "k", 3);
    want_axes(kc, "k_cache", 4);
    want_axes(table, "block_table", 2);
    const int dev = device_of(k, "k");
    const int64_t T = k.size(0), Hkv = k.size(1), d = k.size(2), B = table.size(0), width = table.size(1);
    int64_t Hq = Hkv;
    if (q.defined()) {
      want_axes(q, "q", 3);
      Hq = q.size(1);
    }
    long long st[9];
    st[2] = rows(k, "k", {T, Hkv, d}, dev);
    st[4] = rows(v, "v", {T, Hkv, d}, dev);
    st[0] = st[1] = Hq * d;
    st[3] = Hkv * d;
    if (q.defined()) st[0] = rows(q, "q", {T, Hq, d}, dev);
    if (q_rot.defined()) st[1] = rows(q_rot, "q_rot", {T, Hq, d}, dev);
    if (k_rot.defined()) st[3] = rows(k_rot, "k_rot", {T, Hkv, d}, dev);
    cache(kc, "k_cache", {kc.size(0), kc.size(1), Hkv, d}, dev, st + 5);
    cache(vc, "v_cache", {kc.size(0), kc.size(1), Hkv, d}, dev, st + 7);
    check_packed(table, "block_table", at::kInt, {B, width}, dev);
    check_packed(lens, "cache_lens", at::kInt, {B}, dev);
    if (cu.defined()) check_packed(cu, "cu_seqlens", at::kInt, {B + 1}, dev);
    refuse_gradients({{&q, "q"}, {&q_rot, "q_rot"}, {&k, "k"}, {&k_rot, "k_rot"}, {&v, "v"}, {&kc, "k_cache"},
                      {&vc, "v_cache"}});
    const double base = number(a[11]), pi = number(a[12]);
    const Place at_(dev, a[13]);
    if (fresh) {
      if (q.defined()) q_rot = empty({T, Hq, d}, at::kBFloat16, dev);
      k_rot = empty({T, Hkv, d}, at::kBFloat16, dev);
    }
    if (T == 0) {   // of as many sequences as there are, if none of them has new rows
      int status = check_heads(Hq, Hkv, d);
      if ((!cu.defined() && B != 0) || !positive(base - 1.0) || !positive(pi)) status = S2ATTN_ERR_INVALID_ARG;
      return fresh ? answer(status, q_rot, k_rot) : answer(status);
    }
    int status = g_append(
        data(q), data(q_rot), data(k), data(k_rot), data(v), data(kc), data(vc), static_cast<const int*>(data(table)),
        static_cast<const int*>(data(cu)), static_cast<const int*>(data(lens)), static_cast<int>(T),
        static_cast<int>(B), static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(d),
        static_cast<int>(kc.size(0)), static_cast<int>(kc.size(1)), static_cast<int>(width),
        base, pi, st, at_.stream);
    status = fresh ? written(status, {&kc, &vc}) : written(status, {&q_rot, &k_rot, &kc, &vc});
    return fresh ? answer(status, q_rot, k_rot) : answer(status);
  });
}

// decode(fresh, q, k_cache, v_cache, table, lens, o, lse, scale, workspace, stream): fresh: o and lse are
// allocated here and returned. scale None: 1 / sqrt(d); workspace None: allocated for the call.
PyObject* py_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const bool fresh = a[0] == Py_True;
    const Tensor &q = tensor(a[1], "q"), &kc = tensor(a[2], "k_cache"), &vc = tensor(a[3], "v_cache");
    const Tensor &table = tensor(a[4], "block_table"), &lens = tensor(a[5], "cache_lens");
    Tensor o = tensor(a[6], "o", fresh), lse = tensor(a[7], "lse", true), space = tensor(a[9], "workspace", true);
    want_axes(q, "q", 3);
    want_axes(kc, "k_cache", 4);
    want_axes(table, "block_table", 2);
    const int64_t B = q.size(0), Hq = q.size(1), d = q.size(2), Hkv = kc.size(2), width = table.size(1);
    if (q.scalar_type() != at::kBFloat16) refuse("q", "expected bfloat16, got " + type_name(q.scalar_type()));
    const int dev = device_of(q, "q");
    long long st[6];
    st[0] = rows(q, "q", {B, Hq, d}, dev);
    st[1] = Hq * d;
    if (!fresh) st[1] = rows(o, "o", {B, Hq, d}, dev);
    cache(kc, "k_cache", {kc.size(0), kc.size(1), Hkv, d}, dev, st + 2);
    cache(vc, "v_cache", {kc.size(0), kc.size(1), Hkv, d}, dev, st + 4);
    check_packed(table, "block_table", at::kInt, {B, width}, dev);
    check_packed(lens, "cache_lens", at::kInt, {B}, dev);
    if (lse.defined()) check_packed(lse, "lse", at::kFloat, {B, Hq}, dev);
    if (space.defined()) check_packed(space, "workspace", at::kByte, {space.numel()}, dev);
    refuse_gradients({{&q, "q"}, {&kc, "k_cache"}, {&vc, "v_cache"}, {&o, "o"}, {&lse, "lse"}});
    const double scale = a[8] == Py_None ? 1.0 / std::sqrt(static_cast<double>(d)) : number(a[8]);
    const Place at_(dev, a[10]);
    if (fresh) {
      o = empty({B, Hq, d}, at::kBFloat16, dev);
      lse = empty({B, Hq}, at::kFloat, dev);
    }
    if (B == 0) {
      const int status = positive(static_cast<float>(scale)) ? check_heads(Hq, Hkv, d) : S2ATTN_ERR_INVALID_ARG;
      return fresh ? answer(status, o, lse) : answer(status);
    }
    if (!space.defined())
      space = empty({static_cast<int64_t>(g_decode_space(static_cast<int>(B), static_cast<int>(Hq),
                                                         static_cast<int>(Hkv), static_cast<int>(d)))},
                    at::kByte, dev);
    int status =
        g_decode(data(q), data(kc), data(vc), static_cast<const int*>(data(table)),
                 static_cast<const int*>(data(lens)), data(o), static_cast<float*>(data(lse)), static_cast<int>(B),
                 static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(d), static_cast<int>(kc.size(0)),
                 static_cast<int>(kc.size(1)), static_cast<int>(width), static_cast<float>(scale), st, data(space),
                 static_cast<size_t>(space.numel()), at_.stream);
    if (!fresh) status = written(status, {&o, &lse});
    return fresh ? answer(status, o, lse) : answer(status);
  });
}

// prompt_fwd(fresh, q, k, v, o, lse, cu_seqlens, scale, stream): cu_seqlens is a CPU tensor.
PyObject* py_prompt(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const bool fresh = a[0] == Py_True;
    const Tensor &q = tensor(a[1], "q"), &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
    Tensor o = tensor(a[4], "o", fresh), lse = tensor(a[5], "lse", fresh);
    const Tensor& cu = tensor(a[6], "cu_seqlens");
    want_axes(q, "q", 3);
    want_axes(k, "k", 3);
    const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2), Hkv = k.size(1);
    const int dev = device_of(q, "q");
    long long st[4];
    st[0] = rows(q, "q", {T, Hq, d}, dev);
    st[1] = rows(k, "k", {T, Hkv, d}, dev);
    st[2] = rows(v, "v", {T, Hkv, d}, dev);
    st[3] = Hq * d;
    if (!fresh) {
      st[3] = rows(o, "o", {T, Hq, d}, dev);
      check_packed(lse, "lse", at::kFloat, {Hq, T}, dev);
    }
    if (cu.is_cuda() || cu.scalar_type() != at::kInt || cu.dim() != 1 || !cu.is_contiguous())
      refuse("cu_seqlens", "expected a contiguous int32 CPU tensor of one axis, or a sequence of ints");
    refuse_gradients({{&q, "q"}, {&k, "k"}, {&v, "v"}, {&o, "o"}, {&lse, "lse"}});
    const double scale = a[7] == Py_None ? 1.0 / std::sqrt(static_cast<double>(d)) : number(a[7]);
    const Place at_(dev, a[8]);
    if (fresh) {
      o = empty({T, Hq, d}, at::kBFloat16, dev);
      lse = empty({Hq, T}, at::kFloat, dev);
    }
    if (T == 0) {   // sequences of no rows
      int status = positive(static_cast<float>(scale)) ? check_heads(Hq, Hkv, d) : S2ATTN_ERR_INVALID_ARG;
      if (cu.numel() == 0) status = S2ATTN_ERR_INVALID_ARG;
      for (int64_t i = 0; i < cu.numel(); ++i)
        if (cu.const_data_ptr<int>()[i] != 0) status = S2ATTN_ERR_INVALID_ARG;
      return fresh ? answer(status, o, lse) : answer(status);
    }
    int status =
        g_prompt(data(q), data(k), data(v), data(o), static_cast<float*>(data(lse)), static_cast<const int*>(data(cu)),
                 static_cast<int>(cu.numel()) - 1, static_cast<int>(T), static_cast<int>(Hq), static_cast<int>(Hkv),
                 static_cast<int>(d), static_cast<float>(scale), st, at_.stream);
    if (!fresh) status = written(status, {&o, &lse});
    return fresh ? answer(status, o, lse) : answer(status);
  });
}

PyObject* py_bind(PyObject*, PyObject* args) {
  unsigned long long f[4];
  if (!PyArg_ParseTuple(args, "KKKK", f, f + 1, f + 2, f + 3)) return nullptr;
  g_append = reinterpret_cast<decltype(g_append)>(f[0]);
  g_decode = reinterpret_cast<decltype(g_decode)>(f[1]);
  g_decode_space = reinterpret_cast<decltype(g_decode_space)>(f[2]);
  g_prompt = reinterpret_cast<decltype(g_prompt)>(f[3]);
  Py_RETURN_NONE;
}

template <class F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef g_methods[] = {
    {"bind", py_bind, METH_VARARGS, nullptr},
    {"rope_append", fast(&py_append), METH_FASTCALL, nullptr},
    {"decode", fast(&py_decode), METH_FASTCALL, nullptr},
    {"prompt_fwd", fast(&py_prompt), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_s2torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__s2torch() {
  PyObject* m = PyModule_Create(&g_module);
  if (m && PyModule_AddStringConstant(m, "TORCH_VERSION", TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
