// Native marshalling of the Python calls of the block operators and of the
// mixture-of-experts operators on MXFP4 operands: torch tensors to the
// addresses, sizes and stream that the C ABI of include/nvfp4.h takes.  A
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
typedef int (*route_fn)(cp, int32_t, int64_t, cp, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, float, void*,
                        void*, int64_t, int32_t, void*);
typedef int (*sort_fn)(cp, int32_t, void*, void*, void*, int64_t, int32_t, int32_t, void*, size_t, void*);
typedef int (*mx_quantize_fn)(cp, int64_t, int64_t, int32_t, void*, void*, void*);
typedef int (*mx_quantize_rows_fn)(cp, cp, int32_t, void*, void*, int64_t, int64_t, int64_t, void*);
typedef int (*mx_grouped_fn)(cp, cp, cp, cp, cp, cp, cp, cp, void*, int64_t, int64_t, int64_t, int64_t, int32_t, void*,
                             void*);
typedef int (*mx_gated_fn)(cp, cp, cp, cp, cp, cp, cp, cp, int32_t, int32_t, void*, void*, int64_t, int64_t, int64_t,
                           int64_t, int32_t, void*, void*);
typedef int (*mx_moe_fn)(cp, cp, cp, cp, cp, cp, cp, int32_t, int32_t, cp, cp, cp, cp, cp, cp, void*, int64_t, int64_t,
                         int64_t, int32_t, int32_t, void*, size_t, void*, void*);
epilogue_fn g_epilogue;
gated_fn g_gated;
gated_quantize_fn g_gated_quantize;
ffn_fn g_ffn;
norm_fn g_norm;
route_fn g_route;
sort_fn g_sort;
mx_quantize_fn g_mx_quantize;
mx_quantize_rows_fn g_mx_quantize_rows;
mx_grouped_fn g_mx_grouped;
mx_gated_fn g_mx_gated;
mx_moe_fn g_mx_moe;

enum Type { kBytes, kBf16, kF32, kI32, kF32OrBf16 };
const char* const kTypeNames[] = {"bytes", "bfloat16", "float32", "int32", "float32 or torch.bfloat16"};

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
    if ((type == kF32 && s != at::kFloat) || (type == kI32 && s != at::kInt) ||
        (type == kF32OrBf16 && s != at::kFloat && s != at::kBFloat16) ||
        (type == kBf16 && s != at::kBFloat16 && s != at::kShort && s != at::kUInt16)) {
      snprintf(msg, sizeof msg, "%s is torch.%s, not torch.%s", name, c10::toString(s), kTypeNames[type]);
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

  // Address and row stride of a [rows][cols] matrix (None: NULL): 2-D
  // with unit column stride, or contiguous (stride 0: the row length).
  void* rows(int i, int64_t nrows, int64_t cols, const char* name, int64_t* ld, Type type = kBf16) {
    *ld = 0;
    const at::Tensor* t = tensor(i, name, type);
    if (!t) return nullptr;
    if (t->dim() != 2 || (t->is_contiguous() && t->size(1) == cols))
      return contiguous(*t, prod((int64_t)t->element_size(), prod(nrows, cols)), name);
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

// The mixture-of-experts operators ------------------------------------------

// (logits, bias, score, n_group, topk_group, group_top, top_k, renormalize, scale, ids, weights, T, E, stream)
PyObject* moe_route(PyObject* const* args, Py_ssize_t nargs) {
  Call c("nvfp4_moe_route", args, nargs, 14);
  if (c.failed) return nullptr;
  const int64_t T = c.integer(11), top_k = c.integer(6);
  const int32_t E = c.integer32(12), k = c.integer32(6);
  int64_t ldl;
  const at::Tensor* t = c.tensor(0, "logits", kF32OrBf16);
  const bool bf16 = t && t->scalar_type() == at::kBFloat16;
  void* logits = c.rows(0, T, E, "logits", &ldl, kF32OrBf16);
  void* bias = c.flat(1, prod(4, E), "bias", kF32);
  const int32_t score = c.integer32(2), groups = c.integer32(3), top_groups = c.integer32(4), group_top = c.integer32(5);
  const int32_t renormalize = c.integer32(7) != 0;
  const float scale = c.real(8);
  void* ids = c.flat(9, prod(4, prod(T, top_k)), "ids", kI32);
  void* weights = c.flat(10, prod(4, prod(T, top_k)), "weights", kF32);
  return c.run(13, [&](void* s) {
    return g_route(logits, bf16, ldl, bias, score, groups, top_groups, group_top, k, renormalize, scale, ids, weights, T, E, s);
  });
}

// (ids, first, offsets, row_token, token_rows, T, E, top_k, workspace, stream)
PyObject* moe_sort(PyObject* const* args, Py_ssize_t nargs) {
  Call c("nvfp4_moe_sort", args, nargs, 10);
  if (c.failed) return nullptr;
  const int64_t T = c.integer(5), top_k = c.integer(7);
  const int32_t E = c.integer32(6), k = c.integer32(7), first = c.integer32(1);
  const int64_t rows4 = prod(4, prod(T, top_k));
  void *ids = c.flat(0, rows4, "ids", kI32), *offsets = c.flat(2, prod(4, (int64_t)E + 1), "offsets", kI32);
  void *row_token = c.flat(3, rows4, "row_token", kI32), *token_rows = c.flat(4, rows4, "token_rows", kI32);
  size_t wsb;
  void* ws = c.workspace(8, &wsb);
  return c.run(9, [&](void* s) { return g_sort(ids, first, offsets, row_token, token_rows, T, E, k, ws, wsb, s); });
}

// (x, R, K, rule, q, sf, stream)
PyObject* mx_quantize(PyObject* const* args, Py_ssize_t nargs) {
  Call c("nvfp4_mx_quantize", args, nargs, 7);
  if (c.failed) return nullptr;
  const int64_t R = c.integer(1), K = c.integer(2), n = prod(R, K);
  void* x = c.flat(0, prod(4, n), "x", kF32);
  const int32_t rule = c.integer32(3);
  void *q = c.flat(4, n / 2, "q"), *sf = c.flat(5, n / 32, "sf");
  return c.run(6, [&](void* s) { return g_mx_quantize(x, R, K, rule, q, sf, s); });
}

// (x, row_token, rule, q, sf, rows, T, K, stream)
PyObject* mx_quantize_rows(PyObject* const* args, Py_ssize_t nargs) {
  Call c("nvfp4_mx_quantize_rows_bf16", args, nargs, 9);
  if (c.failed) return nullptr;
  const int64_t rows = c.integer(5), T = c.integer(6), K = c.integer(7), n = prod(rows, K);
  void *x = c.flat(0, prod(2, prod(T, K)), "x", kBf16), *tok = c.flat(1, prod(4, rows), "row_token", kI32);
  const int32_t rule = c.integer32(2);
  void *q = c.flat(3, n / 2, "q"), *sf = c.flat(4, n / 32, "sf");
  return c.run(8, [&](void* s) { return g_mx_quantize_rows(x, tok, rule, q, sf, rows, T, K, s); });
}

// (a, a_sf, row_token, b, b_sf, offsets, alpha, bias, d, rows, T, N, K, E, status, stream)
PyObject* mx_grouped_gemm(PyObject* const* args, Py_ssize_t nargs) {
  Call c("nvfp4_mx_grouped_gemm", args, nargs, 16);
  if (c.failed) return nullptr;
  const int64_t rows = c.integer(9), T = c.integer(10), N = c.integer(11), K = c.integer(12);
  const int32_t E = c.integer32(13);
  const int64_t tk = prod(T, K), en = prod(E, N), enk = prod(en, K);
  void *a = c.flat(0, tk / 2, "a"), *a_sf = c.flat(1, tk / 32, "a_sf");
  void* tok = c.flat(2, prod(4, rows), "row_token", kI32);
  void *b = c.flat(3, enk / 2, "b"), *b_sf = c.flat(4, enk / 32, "b_sf");
  void* offsets = c.flat(5, prod(4, (int64_t)E + 1), "offsets", kI32);
  void *alpha = c.flat(6, prod(4, E), "alpha", kF32), *bias = c.flat(7, prod(2, en), "bias", kBf16);
  void *d = c.flat(8, prod(2, prod(rows, N)), "d", kBf16), *status = c.flat(14, 4, "status", kI32);
  return c.run(15, [&](void* s) {
    return g_mx_grouped(a, a_sf, tok, b, b_sf, offsets, alpha, bias, d, rows, T, N, K, E, status, s);
  });
}

// (a, a_sf, row_token, b, b_sf, offsets, alpha, bias, act, rule, q, sf, rows, T, I, K, E, status, stream)
PyObject* mx_grouped_gated_quantize(PyObject* const* args, Py_ssize_t nargs) {
  Call c("nvfp4_mx_grouped_gated_quantize", args, nargs, 19);
  if (c.failed) return nullptr;
  const int64_t rows = c.integer(12), T = c.integer(13), I = c.integer(14), K = c.integer(15);
  const int32_t E = c.integer32(16);
  const int64_t tk = prod(T, K), ei = prod(E, I), eik = prod(ei, K), ri = prod(rows, I);
  void *a = c.flat(0, tk / 2, "a"), *a_sf = c.flat(1, tk / 32, "a_sf");
  void* tok = c.flat(2, prod(4, rows), "row_token", kI32);
  void *b = c.flat(3, eik, "b"), *b_sf = c.flat(4, eik / 16, "b_sf");
  void* offsets = c.flat(5, prod(4, (int64_t)E + 1), "offsets", kI32);
  void *alpha = c.flat(6, prod(8, E), "alpha", kF32), *bias = c.flat(7, prod(4, ei), "bias", kBf16);
  const int32_t act = c.integer32(8), rule = c.integer32(9);
  void *q = c.flat(10, ri / 2, "q"), *sf = c.flat(11, ri / 32, "sf"), *status = c.flat(17, 4, "status", kI32);
  return c.run(18, [&](void* s) {
    return g_mx_gated(a, a_sf, tok, b, b_sf, offsets, alpha, bias, act, rule, q, sf, rows, T, I, K, E, status, s);
  });
}

// (x, row_token, offsets, w_gu, w_gu_sf, alpha_gu, bias_gu, act, rule, w_d, w_d_sf, alpha_d, bias_d, token_rows,
//  token_weight, out, T, H, I, E, top_k, workspace, status, stream)
PyObject* mx_moe_ffn(PyObject* const* args, Py_ssize_t nargs) {
  Call c("nvfp4_mx_moe_ffn", args, nargs, 24);
  if (c.failed) return nullptr;
  const int64_t T = c.integer(16), H = c.integer(17), I = c.integer(18), top_k = c.integer(20);
  const int32_t E = c.integer32(19), k = c.integer32(20);
  const int64_t th = prod(T, H), rows = prod(T, top_k), eh = prod(E, H), ei = prod(E, I), ehi = prod(eh, I);
  void *x = c.flat(0, prod(2, th), "x", kBf16), *tok = c.flat(1, prod(4, rows), "row_token", kI32);
  void* offsets = c.flat(2, prod(4, (int64_t)E + 1), "offsets", kI32);
  void *gu = c.flat(3, ehi, "w_gu"), *gu_sf = c.flat(4, ehi / 16, "w_gu_sf");
  void *al = c.flat(5, prod(8, E), "alpha_gu", kF32), *bgu = c.flat(6, prod(4, ei), "bias_gu", kBf16);
  const int32_t act = c.integer32(7), rule = c.integer32(8);
  void *dn = c.flat(9, ehi / 2, "w_d"), *dn_sf = c.flat(10, ehi / 32, "w_d_sf");
  void *ald = c.flat(11, prod(4, E), "alpha_d", kF32), *bd = c.flat(12, prod(2, eh), "bias_d", kBf16);
  void *tr = c.flat(13, prod(4, rows), "token_rows", kI32), *tw = c.flat(14, prod(4, rows), "token_weight", kF32);
  void* out = c.flat(15, prod(2, th), "out", kBf16);
  size_t wsb;
  void* ws = c.workspace(21, &wsb);
  void* status = c.flat(22, 4, "status", kI32);
  return c.run(23, [&](void* s) {
    return g_mx_moe(x, tok, offsets, gu, gu_sf, al, bgu, act, rule, dn, dn_sf, ald, bd, tr, tw, out, T, H, I, E, k, ws, wsb,
                    status, s);
  });
}

// Addresses at args[from ..], as integers; false with a Python exception set.
bool addresses(PyObject* const* args, int from, int count, void** p) {
  for (int i = 0; i < count; ++i) {
    p[i] = PyLong_AsVoidPtr(args[from + i]);
    if (PyErr_Occurred()) return false;
  }
  return true;
}

// setup(error class, last_error, epilogue, gated, gated_quantize, ffn, norm): addresses as integers
PyObject* setup(PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 7) {
    PyErr_SetString(PyExc_TypeError, "setup takes 7 arguments");
    return nullptr;
  }
  void* p[6];
  if (!addresses(args, 1, 6, p)) return nullptr;
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

// setup_experts(moe_route, moe_sort, mx_quantize, mx_quantize_rows_bf16, mx_grouped_gemm,
// mx_grouped_gated_quantize, mx_moe_ffn): addresses as integers, after setup
PyObject* setup_experts(PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != 7) {
    PyErr_SetString(PyExc_TypeError, "setup_experts takes 7 arguments");
    return nullptr;
  }
  void* p[7];
  if (!addresses(args, 0, 7, p)) return nullptr;
  g_route = (route_fn)p[0];
  g_sort = (sort_fn)p[1];
  g_mx_quantize = (mx_quantize_fn)p[2];
  g_mx_quantize_rows = (mx_quantize_rows_fn)p[3];
  g_mx_grouped = (mx_grouped_fn)p[4];
  g_mx_gated = (mx_gated_fn)p[5];
  g_mx_moe = (mx_moe_fn)p[6];
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
    {"setup_experts", (PyCFunction)(void (*)())entry<setup_experts>, METH_FASTCALL, nullptr},
    {"moe_route", (PyCFunction)(void (*)())entry<moe_route>, METH_FASTCALL, nullptr},
    {"moe_sort", (PyCFunction)(void (*)())entry<moe_sort>, METH_FASTCALL, nullptr},
    {"mx_quantize", (PyCFunction)(void (*)())entry<mx_quantize>, METH_FASTCALL, nullptr},
    {"mx_quantize_rows", (PyCFunction)(void (*)())entry<mx_quantize_rows>, METH_FASTCALL, nullptr},
    {"mx_grouped_gemm", (PyCFunction)(void (*)())entry<mx_grouped_gemm>, METH_FASTCALL, nullptr},
    {"mx_grouped_gated_quantize", (PyCFunction)(void (*)())entry<mx_grouped_gated_quantize>, METH_FASTCALL, nullptr},
    {"mx_moe_ffn", (PyCFunction)(void (*)())entry<mx_moe_ffn>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", "Argument marshalling of the block and mixture-of-experts operators.", -1, kMethods,
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
