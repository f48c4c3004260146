// marshal.cpp -- the Python side of the operators around a QKV projection:
// checks torch tensors, makes missing outputs with torch's allocator, and
// passes addresses and the stream through the C ABI (include/nts.h).  No step
// of the computation runs here.
//
// These calls serve single tokens, where the host's share of a call is the
// larger one: marshalled in Python, a rotation of one token that makes its
// outputs took 26 us of host time, so it takes 5.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <optional>

#include "nts.h"

namespace {

constexpr int64_t kBlock = 128;

PyObject* g_check = nullptr;   // _lib.check: raises NtsError for a status

// A Python exception that is already set.
struct PyError {};

[[noreturn]] void refuse(const char* fmt, const char* name, const char* more = "") {
  PyErr_Format(PyExc_ValueError, fmt, name, more);
  throw PyError();
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kLong: return "torch.int64";
    case at::kByte: return "torch.uint8";
    default: return "another type";
  }
}

bool given(PyObject* o) { return o != nullptr && o != Py_None; }

const at::Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

// The device of a call: that of its first tensor, which has to be the current one.
int device_of(const char* name, const at::Tensor& t) {
  if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
  const int dev = t.get_device();
  if (dev != (int)c10::cuda::current_device()) refuse("%s must be on the current device", name);
  return dev;
}

void check_place(const char* name, const at::Tensor& t, at::ScalarType type, int dev) {
  if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
  if (t.get_device() != dev) refuse("%s must be on the current device", name);
  if (t.scalar_type() != type) refuse("%s must be %s", name, type_name(type));
}

// A contiguous tensor on the call's device.
const at::Tensor& flat(const char* name, PyObject* o, at::ScalarType type, int dev) {
  const at::Tensor& t = tensor(name, o);
  check_place(name, t, type, dev);
  if (!t.is_contiguous()) refuse("%s must be contiguous", name);
  return t;
}

const at::Tensor& matrix(const char* name, const at::Tensor& t) {
  if (t.dim() != 2) refuse("%s must be a matrix", name);
  return t;
}

// The stream of a call.  What the call makes belongs to that stream, so that
// memory that torch hands out again is free there; when it is not the current
// one, torch also waits for the current stream, where the results are used, before
// it hands an output on.  The legacy handle is the default stream under another
// name.  The per-thread stream has no pool of torch's: what a call makes there
// would come from the current stream's pool, where earlier work may still use
// the memory and later work may be given it while the kernel writes.  Only when
// the current stream is the default one does CUDA order the two both ways;
// otherwise the call makes nothing (`pool` is false).
struct On {
  int dev;
  void* handle;
  bool foreign = false, pool = true;
  std::optional<c10::cuda::CUDAStream> user;
  c10::cuda::OptionalCUDAStreamGuard guard;

  On(PyObject* o, int device) : dev(device) {
    const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev);
    handle = current.stream();
    if (!given(o)) return;
    PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
    if (h == nullptr) throw PyError();
    handle = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (handle == nullptr && PyErr_Occurred()) throw PyError();
    const cudaStream_t s = static_cast<cudaStream_t>(handle);
    const bool main = s == nullptr || s == cudaStreamLegacy;
    if (s == current.stream() || (main && current.stream() == nullptr)) return;
    foreign = s == cudaStreamPerThread;
    pool = !foreign || current.stream() == nullptr;
    if (foreign) return;
    user = current;
    guard.reset_stream(main
                           ? c10::cuda::getDefaultCUDAStream((c10::DeviceIndex)dev)
                           : c10::cuda::getStreamFromExternal(s, (c10::DeviceIndex)dev));
  }
};

at::Tensor scratch(at::IntArrayRef shape, at::ScalarType type, const On& on) {
  return at::Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (int8_t)on.dev),
                                           std::nullopt));
}

at::Tensor fresh(const char* name, at::IntArrayRef shape, at::ScalarType type, const On& on) {
  if (!on.pool)
    refuse("%s is needed on the per-thread stream, as another than the default stream is current",
           name);
  at::Tensor t = scratch(shape, type, on);
  if (on.user && t.numel() != 0)
    c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), *on.user);
  return t;
}

// The caller's output buffer, checked, or a new one.
at::Tensor output(const char* name, PyObject* o, at::IntArrayRef shape, at::ScalarType type,
                  const On& on) {
  if (!given(o)) return fresh(name, shape, type, on);
  const at::Tensor& t = flat(name, o, type, on.dev);
  if (t.sizes() != shape) refuse("%s has the wrong shape", name);
  return t;
}

// A bf16 matrix with contiguous rows and any row stride.
struct Rows {
  at::Tensor t;
  int64_t ld;
};

Rows rows(const char* name, PyObject* o, int dev, const at::Tensor* like = nullptr) {
  const at::Tensor& t = tensor(name, o);
  check_place(name, t, at::kBFloat16, dev);
  matrix(name, t);
  if (like != nullptr && t.sizes() != like->sizes()) refuse("%s has the wrong shape", name);
  if (t.size(1) > 1 && t.stride(1) != 1) refuse("%s must have contiguous rows", name);
  return {t, t.size(0) > 1 ? t.stride(0) : t.size(1)};
}

Rows rows_out(const char* name, PyObject* o, const On& on, const at::Tensor& like) {
  if (given(o)) return rows(name, o, on.dev, &like);
  return {fresh(name, like.sizes(), at::kBFloat16, on), like.size(1)};
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError();
  return v;
}

float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyError();
  return (float)v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PyError();
  return v != 0;
}

// Runs a call of the library without the interpreter lock; NtsError on a failure.
template <typename F>
void call(F f) {
  int status;
  Py_BEGIN_ALLOW_THREADS
  status = f();
  Py_END_ALLOW_THREADS
  if (status == NTS_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "i", status);
  Py_XDECREF(r);
  if (r != nullptr) PyErr_SetString(PyExc_RuntimeError, "a status that raised nothing");
  throw PyError();
}

PyObject* wrap(const at::Tensor& t) {
  PyObject* o = THPVariable_Wrap(t);
  if (o == nullptr) throw PyError();
  return o;
}

// A tuple of tensors; an undefined one stands for None.
template <typename... T>
PyObject* tuple_of(const T&... t) {
  PyObject* r = PyTuple_New(sizeof...(T));
  if (r == nullptr) throw PyError();
  Py_ssize_t i = 0;
  for (const at::Tensor* x : {&t...}) {
    PyObject* o;
    if (x->defined()) {
      o = THPVariable_Wrap(*x);
    } else {
      Py_INCREF(Py_None);
      o = Py_None;
    }
    if (o == nullptr) {
      Py_DECREF(r);
      throw PyError();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
float* fptr(const at::Tensor& t) { return static_cast<float*>(ptr(t)); }

// ------------------------------------------------------------- rotation

// What a rotation and its gradient share.
struct RopeArgs {
  int dev;
  Rows q, k;
  float *gq, *gk, *table;
  int64_t* pos;
  int64_t P, T, nq, nk, d, rot;

  RopeArgs(PyObject* oq, PyObject* ogq, PyObject* ok, PyObject* ogk, PyObject* opos,
           PyObject* otable, PyObject* od) {
    dev = device_of("q", tensor("q", oq));
    q = rows("q", oq, dev);
    k = rows("k", ok, dev);
    d = integer(od);
    T = q.t.size(0);
    if (d <= 0 || q.t.size(1) % d != 0 || k.t.size(1) % d != 0)
      refuse("q and k must hold whole heads of %s values", "head_dim");
    if (k.t.size(0) != T) refuse("q and k must have the same number of %s", "tokens");
    const at::Tensor& tg = flat("gamma_q", ogq, at::kFloat, dev);
    const at::Tensor& tk = flat("gamma_k", ogk, at::kFloat, dev);
    if (tg.numel() != d) refuse("%s must hold head_dim values", "gamma_q");
    if (tk.numel() != d) refuse("%s must hold head_dim values", "gamma_k");
    const at::Tensor& tp = flat("positions", opos, at::kLong, dev);
    if (tp.numel() != T) refuse("%s must hold one position per token", "positions");
    const at::Tensor& tt = matrix("table", flat("table", otable, at::kFloat, dev));
    gq = fptr(tg);
    gk = fptr(tk);
    table = fptr(tt);
    pos = static_cast<int64_t*>(tp.data_ptr());
    P = tt.size(0);
    rot = tt.size(1);
    nq = q.t.size(1) / d;
    nk = k.t.size(1) / d;
  }
};

// q, gamma_q, k, gamma_k, positions, table, head_dim, eps, interleaved, out_q,
// out_k, rinv_q, rinv_k, want_rinv, stream
PyObject* qknorm_rope(PyObject* const* a) {
  const RopeArgs r(a[0], a[1], a[2], a[3], a[4], a[5], a[6]);
  const float eps = real(a[7]);
  const int il = truth(a[8]);
  const On on(a[14], r.dev);
  const Rows yq = rows_out("out_q", a[9], on, r.q.t), yk = rows_out("out_k", a[10], on, r.k.t);
  const bool want = truth(a[13]);
  at::Tensor rq, rk;
  if (want || given(a[11])) rq = output("rinv_q", a[11], {r.T, r.nq}, at::kFloat, on);
  if (want || given(a[12])) rk = output("rinv_k", a[12], {r.T, r.nk}, at::kFloat, on);
  call([&] {
    return nts_qknorm_rope(ptr(r.q.t), r.q.ld, r.gq, ptr(yq.t), yq.ld, fptr(rq), ptr(r.k.t),
                           r.k.ld, r.gk, ptr(yk.t), yk.ld, fptr(rk), r.pos, r.table, r.P, r.T, r.nq,
                           r.nk, r.d, r.rot, il, eps, on.handle);
  });
  return tuple_of(yq.t, yk.t, rq, rk);
}

// dyq, dyk, q, gamma_q, k, gamma_k, positions, table, head_dim, eps,
// interleaved, out_dq, out_dk, dgamma_q, dgamma_k, workspace, stream
PyObject* qknorm_rope_backward(PyObject* const* a) {
  const RopeArgs r(a[2], a[3], a[4], a[5], a[6], a[7], a[8]);
  const float eps = real(a[9]);
  const int il = truth(a[10]);
  const Rows dyq = rows("dyq", a[0], r.dev, &r.q.t), dyk = rows("dyk", a[1], r.dev, &r.k.t);
  const On on(a[16], r.dev);
  const Rows dq = rows_out("out_dq", a[11], on, r.q.t);
  const Rows dk = rows_out("out_dk", a[12], on, r.k.t);
  const at::Tensor dgq = output("dgamma_q", a[13], {r.d}, at::kFloat, on);
  const at::Tensor dgk = output("dgamma_k", a[14], {r.d}, at::kFloat, on);
  at::Tensor ws;
  if (given(a[15])) {
    ws = flat("workspace", a[15], at::kByte, r.dev);
  } else {
    int64_t bytes = 0;
    call([&] { return nts_qknorm_rope_backward_workspace(r.d, &bytes); });
    if (on.foreign) refuse("a %s is needed on the per-thread stream", "workspace");
    ws = scratch({bytes}, at::kByte, on);
  }
  call([&] {
    return nts_qknorm_rope_backward(ptr(dyq.t), dyq.ld, ptr(dyk.t), dyk.ld, ptr(r.q.t), r.q.ld,
                                    r.gq, ptr(r.k.t), r.k.ld, r.gk, r.pos, r.table, r.P, ptr(dq.t),
                                    dq.ld, ptr(dk.t), dk.ld, fptr(dgq), fptr(dgk), ptr(ws),
                                    ws.numel(), r.T, r.nq, r.nk, r.d, r.rot, il, eps, on.handle);
  });
  return tuple_of(dq.t, dk.t, dgq, dgk);
}

// ---------------------------------------------------------------- casts

int64_t blocks(int64_t n, int64_t per = kBlock) { return (n + per - 1) / per; }

// x, gamma, eps, codes, scales, rinv, want_rinv, stream
PyObject* rmsnorm_blockcast(PyObject* const* a) {
  const int dev = device_of("x", tensor("x", a[0]));
  const at::Tensor& x = matrix("x", flat("x", a[0], at::kBFloat16, dev));
  const int64_t T = x.size(0), D = x.size(1);
  float* gamma = nullptr;
  if (given(a[1])) {
    const at::Tensor& g = flat("gamma", a[1], at::kFloat, dev);
    if (g.numel() != D) refuse("%s must hold D values", "gamma");
    gamma = fptr(g);
  }
  const float eps = real(a[2]);
  const On on(a[7], dev);
  const at::Tensor codes = output("codes", a[3], {T, D}, at::kByte, on);
  const at::Tensor scales = output("scales", a[4], {T, blocks(D)}, at::kFloat, on);
  at::Tensor rinv;
  if (truth(a[6]) || given(a[5])) rinv = output("rinv", a[5], {T}, at::kFloat, on);
  call([&] {
    return nts_rmsnorm_blockcast(ptr(x), gamma, static_cast<uint8_t*>(ptr(codes)), fptr(scales),
                                 fptr(rinv), T, D, eps, on.handle);
  });
  return tuple_of(codes, scales, rinv);
}

// x, block_rows, codes, scales, stream
PyObject* blockcast(PyObject* const* a) {
  const int dev = device_of("x", tensor("x", a[0]));
  const at::Tensor& x = matrix("x", flat("x", a[0], at::kBFloat16, dev));
  const int64_t T = x.size(0), D = x.size(1), per = integer(a[1]);
  if (per != 1 && per != kBlock) refuse("%s must be 1 or 128", "block_rows");
  const On on(a[4], dev);
  const at::Tensor codes = output("codes", a[2], {T, D}, at::kByte, on);
  const at::Tensor scales = output("scales", a[3], {blocks(T, per), blocks(D)}, at::kFloat, on);
  call([&] {
    return nts_blockcast(ptr(x), static_cast<uint8_t*>(ptr(codes)), fptr(scales), T, D, (int)per,
                         on.handle);
  });
  return tuple_of(codes, scales, at::Tensor());
}

// x, codes, scales, stream
PyObject* blockcast_t(PyObject* const* a) {
  const int dev = device_of("x", tensor("x", a[0]));
  const at::Tensor& x = matrix("x", flat("x", a[0], at::kBFloat16, dev));
  const int64_t T = x.size(0), D = x.size(1);
  const On on(a[3], dev);
  const at::Tensor codes = output("codes", a[1], {D, (T + 15) / 16 * 16}, at::kByte, on);
  const at::Tensor scales = output("scales", a[2], {D, blocks(T)}, at::kFloat, on);
  call([&] {
    return nts_blockcast_t(ptr(x), static_cast<uint8_t*>(ptr(codes)), fptr(scales), T, D, on.handle);
  });
  return tuple_of(codes, scales, at::Tensor());
}

// -------------------------------------------------------------- product

const at::Tensor& operand(const char* name, PyObject* o, int dev) {
  const at::Tensor& t = tensor(name, o);
  const bool fp8 = t.scalar_type() == at::kFloat8_e4m3fn;
  return matrix(name, flat(name, o, fp8 ? at::kFloat8_e4m3fn : at::kByte, dev));
}

// a_codes, a_scales, w_codes, w_scales, out, fp32 (when there is no out), stream
PyObject* gemm_blockscaled(PyObject* const* a) {
  const int dev = device_of("a_codes", tensor("a_codes", a[0]));
  const at::Tensor& x = operand("a_codes", a[0], dev);
  const at::Tensor& w = operand("w_codes", a[2], dev);
  const at::Tensor& sx = flat("a_scales", a[1], at::kFloat, dev);
  const at::Tensor& sw = flat("w_scales", a[3], at::kFloat, dev);
  const int64_t M = x.size(0), K = x.size(1), N = w.size(0), kb = blocks(K);
  if (w.size(1) != K) refuse("a_codes and w_codes must have the same %s", "K");
  if (sx.sizes() != at::IntArrayRef({M, kb})) refuse("%s must have shape [M, ceil(K/128)]", "a_scales");
  int per;
  if (sw.sizes() == at::IntArrayRef({blocks(N), kb}))
    per = (int)kBlock;
  else if (sw.sizes() == at::IntArrayRef({N, kb}))
    per = 1;
  else
    refuse("%s must have shape [ceil(N/128), ceil(K/128)] or [N, ceil(K/128)]", "w_scales");
  bool fp32 = truth(a[5]);
  if (given(a[4])) {
    const at::ScalarType t = tensor("out", a[4]).scalar_type();
    if (t != at::kFloat && t != at::kBFloat16) refuse("%s must be bfloat16 or float32", "out");
    fp32 = t == at::kFloat;
  }
  const On on(a[6], dev);
  const at::Tensor y = output("out", a[4], {M, N}, fp32 ? at::kFloat : at::kBFloat16, on);
  call([&] {
    return nts_gemm_blockscaled(static_cast<uint8_t*>(ptr(x)), fptr(sx),
                                static_cast<uint8_t*>(ptr(w)), fptr(sw), per, ptr(y),
                                fp32 ? NTS_OUT_FP32 : NTS_OUT_BF16, M, N, K, on.handle);
  });
  return wrap(y);
}

// ------------------------------------------------------------- the module

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const PyError&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_check(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XSETREF(g_check, f);
  Py_RETURN_NONE;
}

#define ENTRY(name, n) \
  {#name, (PyCFunction)(void (*)(void))entry<name, n>, METH_FASTCALL, nullptr}

PyMethodDef g_methods[] = {ENTRY(qknorm_rope, 15),
                           ENTRY(qknorm_rope_backward, 17),
                           ENTRY(rmsnorm_blockcast, 8),
                           ENTRY(blockcast, 5),
                           ENTRY(blockcast_t, 4),
                           ENTRY(gemm_blockscaled, 7),
                           {"set_check", set_check, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "marshal_nts", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_marshal_nts(void) { return PyModule_Create(&g_module); }
