// Native marshalling of the block operators' Python calls: torch tensors to
// the addresses, sizes and stream that the C ABI of include/nvfp4.h takes.  A
// decode step makes hundreds of these calls back to back, each a few
// microseconds of GPU work; the same checks and argument conversion through
// ctypes took 4.5 us a call, as long as the launch itself.
//
// Checks only: every tensor is on one GPU, of its type, large enough, and
// contiguous or (where the call takes a row stride) a matrix with unit column
// stride.  The call is made on that GPU's current stream, or on the stream
// given.  Addresses of the C functions come from the loaded library
// (setup), so nothing is linked twice.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdint>
#include <cstdio>

namespace {

// nvfp4_status values that refusals here share with the C ABI
constexpr int kErrNull = 1, kErrShape = 2;

PyObject* g_error = nullptr;  // Nvfp4Error(status, fn, message)
const char* (*g_last_error)() = nullptr;

typedef const void* cp;
typedef int (*epilogue_fn)(cp, cp, cp, cp, cp, cp, int32_t, cp, int64_t, float, void*, int64_t, int64_t, int64_t, int64_t,
                           void*, size_t, void*);
typedef int (*gated_fn)(cp, cp, cp, cp, cp, cp, int32_t, void*, int64_t, int64_t, int64_t, int64_t, void*, size_t, void*);
typedef int (*gated_quantize_fn)(cp, cp, cp, cp, cp, cp, int32_t, cp, void*, void*, int64_t, int64_t, int64_t, void*,
                                 size_t, void*);
typedef int (*ffn_fn)(cp, cp, cp, cp, cp, cp, int32_t, cp, cp, cp, cp, cp, cp, int64_t, float, void*, int64_t, int64_t,
                      int64_t, int64_t, void*, size_t, void*);
typedef int (*norm_fn)(cp, int64_t, cp, cp, cp, int64_t, cp, int64_t, float, cp, cp, float, int32_t, void*, int64_t, void*,
                       int64_t, cp, void*, void*, int64_t, int64_t, void*);
epilogue_fn g_epilogue;
gated_fn g_gated;
gated_quantize_fn g_gated_quantize;
ffn_fn g_ffn;
norm_fn g_norm;

enum Type { kBytes, kBf16, kF32 };

// a * b of sizes: 0 if one is negative (the library refuses those), saturating
int64_t prod(int64_t a, int64_t b) {
  if (a <= 0 || b <= 0) return 0;
  return a > INT64_MAX / b ? INT64_MAX : a * b;
}

// Other Python threads run while one exists: a launch may wait for room in the
// GPU's queue, and what it waits for may need the interpreter (a host function
// on the stream).
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// One call being marshalled.  The first thing found wrong is raised as a
// Python exception and `failed` set; later steps then do nothing.
struct Call {
  const char* fn;
  PyObject* const* args;
  Py_ssize_t nargs;
  bool failed = false;
  int device = -1;
  c10::Device on = c10::Device(c10::DeviceType::CUDA, 0);

  Call(const char* fn_, PyObject* const* args_, Py_ssize_t nargs_, Py_ssize_t want) : fn(fn_), args(args_), nargs(nargs_) {
    if (nargs != want) {
      PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", fn, want, nargs);
      failed = true;
    }
  }

  void refuse(int status, const char* message) {
    if (failed) return;
    failed = true;
    PyObject* e = PyObject_CallFunction(g_error, "iss", status, fn, message);
    if (!e) return;
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }

  int64_t integer(int i) {
    if (failed) return 0;
    const int64_t v = PyLong_AsLongLong(args[i]);
    if (v == -1 && PyErr_Occurred()) failed = true;
    return v;
  }
  int32_t integer32(int i) {
    const int64_t v = integer(i);
    return v < INT32_MIN ? INT32_MIN : v > INT32_MAX ? INT32_MAX : (int32_t)v;  // out-of-range enums stay refused
  }
  float real(int i) {
    if (failed) return 0.0f;
    const double v = PyFloat_AsDouble(args[i]);
    if (v == -1.0 && PyErr_Occurred()) failed = true;
    return (float)v;
  }

  // The tensor at i, on the call's GPU and of its type (nullptr for None or a refusal).
  const at::Tensor* tensor(int i, const char* name, Type type) {
    if (failed || args[i] == Py_None) return nullptr;
    char msg[160];
    if (!THPVariable_Check(args[i]) || !THPVariable_Unpack(args[i]).is_cuda()) {
      snprintf(msg, sizeof msg, "%s must be a GPU tensor", name);
      refuse(kErrNull, msg);
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(args[i]);
    if (device < 0) {
      device = t.get_device();
      on = t.device();
    } else if (t.get_device() != device) {
      snprintf(msg, sizeof msg, "%s is on GPU %d, the call's other tensors on GPU %d", name, (int)t.get_device(), device);
      refuse(kErrShape, msg);
      return nullptr;
    }
    const at::ScalarType s = t.scalar_type();
    if ((type == kF32 && s != at::kFloat) ||
        (type == kBf16 && s != at::kBFloat16 && s != at::kShort && s != at::kUInt16)) {
      snprintf(msg, sizeof msg, "%s is torch.%s, not torch.%s", name, c10::toString(s), type == kF32 ? "float32" : "bfloat16");
      refuse(kErrShape, msg);
      return nullptr;
    }
    return &t;
  }

  // Address of a contiguous tensor of at least nbytes (None: NULL).
  void* flat(int i, int64_t nbytes, const char* name, Type type = kBytes) {
    const at::Tensor* t = tensor(i, name, type);
    return t ? contiguous(*t, nbytes, name) : nullptr;
  }

  void* contiguous(const at::Tensor& t, int64_t nbytes, const char* name) {
    char msg[160];
    if (!t.is_contiguous()) {
      snprintf(msg, sizeof msg, "%s must be contiguous", name);
      refuse(kErrShape, msg);
      return nullptr;
    }
    if ((int64_t)t.nbytes() < nbytes) {
      snprintf(msg, sizeof msg, "%s holds %lld bytes, the call needs %lld", name, (long long)t.nbytes(), (long long)nbytes);
      refuse(kErrShape, msg);
      return nullptr;
    }
    return t.data_ptr();
  }

  // Address and row stride of a bf16 [rows][cols] matrix (None: NULL): 2-D
  // with unit column stride, or contiguous (stride 0: the row length).
  void* rows(int i, int64_t nrows, int64_t cols, const char* name, int64_t* ld) {
    *ld = 0;
    const at::Tensor* t = tensor(i, name, kBf16);
    if (!t) return nullptr;
    if (t->dim() != 2 || (t->is_contiguous() && t->size(1) == cols)) return contiguous(*t, prod(2, prod(nrows, cols)), name);
    char msg[160];
    if (t->size(0) < nrows || t->size(1) != cols) {
      snprintf(msg, sizeof msg, "%s is %lld x %lld, the call needs %lld x %lld", name, (long long)t->size(0),
               (long long)t->size(1), (long long)nrows, (long long)cols);
      refuse(kErrShape, msg);
      return nullptr;
    }
    if (t->stride(0) < cols || (cols > 1 && t->stride(1) != 1)) {
      snprintf(msg, sizeof msg, "%s needs unit column stride and a row stride of at least %lld", name, (long long)cols);
      refuse(kErrShape, msg);
      return nullptr;
    }
    *ld = t->stride(0);
    return t->data_ptr();
  }

  void* workspace(int i, size_t* bytes) {
    *bytes = 0;
    const at::Tensor* t = tensor(i, "workspace", kBytes);
    if (!t) return nullptr;
    *bytes = t->nbytes();
    return contiguous(*t, 0, "workspace");
  }

  // call(stream) on the tensors' GPU, without the interpreter lock (the
  // caller's arguments keep the tensors alive); None or the raised exception.
  template <class F>
  PyObject* run(int stream_arg, F&& call) {
    if (failed) return nullptr;
    void* stream = nullptr;
    if (args[stream_arg] != Py_None) {
      stream = PyLong_AsVoidPtr(args[stream_arg]);
      if (PyErr_Occurred()) return nullptr;
    }
    if (args[stream_arg] == Py_None && device >= 0)
      stream = c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
    int status;
    {
      const Unlocked unlocked;
      if (device >= 0 && device != c10::hip::current_device()) {
        const c10::DeviceGuard guard(on);
        status = call(stream);
      } else {
        status = call(stream);
      }
    }
    if (status != 0) {
      refuse(status, g_last_error());
      return nullptr;
    }
    Py_RETURN_NONE;
  }
};

// (a, a_sf, b, b_sf, alpha, bias, act, residual, beta, d, M, N, K, workspace, stream)
PyObject* gemm_epilogue(PyObject* const* args, Py_ssize_t nargs) {
  Call c("nvfp4_gemm_epilogue", args, nargs, 15);
  if (c.failed) return nullptr;
  const int64_t M = c.integer(10), N = c.integer(11), K = c.integer(12);
  const int64_t mk = prod(M, K), nk = prod(N, K);
  void *a = c.flat(0, mk / 2, "a"), *a_sf = c.flat(1, mk / 16, "a_sf");
  void *b = c.flat(2, nk / 2, "b"), *b_sf = c.flat(3, nk / 16, "b_sf");
  void *alpha = c.flat(4, 4, "alpha", kF32), *bias = c.flat(5, prod(2, N), "bias", kBf16);
  const int32_t act = c.integer32(6);
  int64_t ldr, ldd;
  void* res = c.rows(7, M, N, "residual", &ldr);
  const float beta = c.real(8);
  void* d = c.rows(9, M, N, "d", &ldd);
  size_t wsb;
  void* ws = c.workspace(13, &wsb);
  return c.run(14, [&](void* s) {
    return g_epilogue(a, a_sf, b, b_sf, alpha, bias, act, res, ldr, beta, d, ldd, M, N, K, ws, wsb, s);
  });
}

// (a, a_sf, b, b_sf, alpha, bias, act, h, M, I, K, workspace, stream)
PyObject* gemm_gated(PyObject* const* args, Py_ssize_t nargs) {
  Call c("nvfp4_gemm_gated", args, nargs, 13);
  if (c.failed) return nullptr;
  const int64_t M = c.integer(8), I = c.integer(9), K = c.integer(10);
  const int64_t mk = prod(M, K), ik = prod(I, K);
  void *a = c.flat(0, mk / 2, "a"), *a_sf = c.flat(1, mk / 16, "a_sf");
  void *b = c.flat(2, ik, "b"), *b_sf = c.flat(3, ik / 8, "b_sf");
  void *alpha = c.flat(4, 8, "alpha", kF32), *bias = c.flat(5, prod(4, I), "bias", kBf16);
  const int32_t act = c.integer32(6);
  int64_t ldh;
  void* h = c.rows(7, M, I, "h", &ldh);
  size_t wsb;
  void* ws = c.workspace(11, &wsb);
  return c.run(12, [&](void* s) { return g_gated(a, a_sf, b, b_sf, alpha, bias, act, h, ldh, M, I, K, ws, wsb, s); });
}

// (a, a_sf, b, b_sf, alpha, bias, act, gs, q, sf, M, I, K, workspace, stream)
PyObject* gemm_gated_quantize(PyObject* const* args, Py_ssize_t nargs) {
  Call c("nvfp4_gemm_gated_quantize", args, nargs, 15);
  if (c.failed) return nullptr;
  const int64_t M = c.integer(10), I = c.integer(11), K = c.integer(12);
  const int64_t mk = prod(M, K), ik = prod(I, K), mi = prod(M, I);
  void *a = c.flat(0, mk / 2, "a"), *a_sf = c.flat(1, mk / 16, "a_sf");
  void *b = c.flat(2, ik, "b"), *b_sf = c.flat(3, ik / 8, "b_sf");
  void *alpha = c.flat(4, 8, "alpha", kF32), *bias = c.flat(5, prod(4, I), "bias", kBf16);
  const int32_t act = c.integer32(6);
  void *gs = c.flat(7, 4, "gs", kF32), *q = c.flat(8, mi / 2, "q"), *sf = c.flat(9, mi / 16, "sf");
  size_t wsb;
  void* ws = c.workspace(13, &wsb);
  return c.run(14, [&](void* s) {
    return g_gated_quantize(a, a_sf, b, b_sf, alpha, bias, act, gs, q, sf, M, I, K, ws, wsb, s);
  });
}

// (a, a_sf, w_gu, w_gu_sf, alpha_gu, bias_gu, act, gs_h, w_d, w_d_sf, alpha_d, bias_d, residual, beta, d, M, H, I,
//  workspace, stream)
PyObject* ffn(PyObject* const* args, Py_ssize_t nargs) {
  Call c("nvfp4_ffn", args, nargs, 20);
  if (c.failed) return nullptr;
  const int64_t M = c.integer(15), H = c.integer(16), I = c.integer(17);
  const int64_t mh = prod(M, H), hi = prod(H, I);
  void *a = c.flat(0, mh / 2, "a"), *a_sf = c.flat(1, mh / 16, "a_sf");
  void *gu = c.flat(2, hi, "w_gu"), *gu_sf = c.flat(3, hi / 8, "w_gu_sf");
  void *al = c.flat(4, 8, "alpha_gu", kF32), *bgu = c.flat(5, prod(4, I), "bias_gu", kBf16);
  const int32_t act = c.integer32(6);
  void* gs = c.flat(7, 4, "gs_h", kF32);
  void *dn = c.flat(8, hi / 2, "w_d"), *dn_sf = c.flat(9, hi / 16, "w_d_sf");
  void *ald = c.flat(10, 4, "alpha_d", kF32), *bd = c.flat(11, prod(2, H), "bias_d", kBf16);
  int64_t ldr, ldd;
  void* res = c.rows(12, M, H, "residual", &ldr);
  const float beta = c.real(13);
  void* d = c.rows(14, M, H, "d", &ldd);
  size_t wsb;
  void* ws = c.workspace(18, &wsb);
  return c.run(19, [&](void* s) {
    return g_ffn(a, a_sf, gu, gu_sf, al, bgu, act, gs, dn, dn_sf, ald, bd, res, ldr, beta, d, ldd, M, H, I, ws, wsb, s);
  });
}

// (x, post_weight, post_bias, gate, gate_group, residual, beta, weight, bias, eps, kind, r, y, gs, q, sf, T, H, stream)
PyObject* residual_norm(PyObject* const* args, Py_ssize_t nargs) {
  Call c("nvfp4_residual_norm", args, nargs, 19);
  if (c.failed) return nullptr;
  const int64_t T = c.integer(16), H = c.integer(17), group = c.integer(4);
  const int64_t h2 = prod(2, H), th = prod(T, H);
  const int64_t gates = group < 0 || T <= 0 ? 0 : group == 0 ? 1 : (T - 1) / group + 1;
  int64_t ldx, ldres, ldr, ldy;
  void *x = c.rows(0, T, H, "x", &ldx);
  void *pw = c.flat(1, h2, "post_weight", kBf16), *pb = c.flat(2, h2, "post_bias", kBf16);
  void *gate = c.flat(3, prod(gates, h2), "gate", kBf16), *res = c.rows(5, T, H, "residual", &ldres);
  const float beta = c.real(6);
  void *w = c.flat(7, h2, "weight", kBf16), *b = c.flat(8, h2, "bias", kBf16);
  const float eps = c.real(9);
  const int32_t kind = c.integer32(10);
  void *r = c.rows(11, T, H, "r", &ldr), *y = c.rows(12, T, H, "y", &ldy);
  void *gs = c.flat(13, 4, "gs", kF32), *q = c.flat(14, th / 2, "q"), *sf = c.flat(15, th / 16, "sf");
  return c.run(18, [&](void* s) {
    return g_norm(x, ldx, pw, pb, gate, group, res, ldres, beta, w, b, eps, kind, r, ldr, y, ldy, gs, q, sf, T, H, s);
  });
}

// setup(error class, last_error, epilogue, gated, gated_quantize, ffn, norm): addresses as integers
PyObject* setup(PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 7) {
    PyErr_SetString(PyExc_TypeError, "setup takes 7 arguments");
    return nullptr;
  }
  void* p[6];
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i + 1]);
    if (PyErr_Occurred()) return nullptr;
  }
  Py_INCREF(args[0]);
  Py_XDECREF(g_error);
  g_error = args[0];
  g_last_error = (const char* (*)())p[0];
  g_epilogue = (epilogue_fn)p[1];
  g_gated = (gated_fn)p[2];
  g_gated_quantize = (gated_quantize_fn)p[3];
  g_ffn = (ffn_fn)p[4];
  g_norm = (norm_fn)p[5];
  Py_RETURN_NONE;
}

// A Python entry point: no C++ exception leaves it (torch throws for tensors
// without storage, sparse ones for instance).
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  try {
    return F(args, nargs);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyMethodDef kMethods[] = {
    {"setup", (PyCFunction)(void (*)())entry<setup>, METH_FASTCALL, nullptr},
    {"gemm_epilogue", (PyCFunction)(void (*)())entry<gemm_epilogue>, METH_FASTCALL, nullptr},
    {"gemm_gated", (PyCFunction)(void (*)())entry<gemm_gated>, METH_FASTCALL, nullptr},
    {"gemm_gated_quantize", (PyCFunction)(void (*)())entry<gemm_gated_quantize>, METH_FASTCALL, nullptr},
    {"ffn", (PyCFunction)(void (*)())entry<ffn>, METH_FASTCALL, nullptr},
    {"residual_norm", (PyCFunction)(void (*)())entry<residual_norm>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", "Argument marshalling of the block operators.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__binding() {
  PyObject* m = PyModule_Create(&kModule);
  // the torch whose headers this was compiled against: another one may lay its tensors out differently
  if (m && PyModule_AddStringConstant(m, "torch_version", NVFP4_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
