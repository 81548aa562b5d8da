// Python binding of the cache and scoring operators: checks torch tensors,
// allocates the results, and calls the C entry points of libmk.so on the
// current stream.  Marshalling only, in C++ because a call on a few tokens is
// as long as its host side: the same checks in Python with ctypes took 12 us of 18.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "mk_cache.h"

namespace {

PyObject* g_error = nullptr;  // MkError(code, what)

PyObject* refuse(int code, const std::string& what) {
  if (PyObject* e = PyObject_CallFunction(g_error, "is", code, what.c_str())) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}
struct Refused {
  int code;
  std::string what;
};
void require(bool ok, const char* op, const char* name, const char* wanted) {
  if (!ok) throw Refused{MK_ERR_INVALID_ARG, std::string(op) + ": " + name + ": " + wanted};
}

// An argument as a tensor; None: an undefined one where that is allowed.
at::Tensor tensor(PyObject* o, const char* op, const char* name, bool optional = false) {
  if (o == Py_None && optional) return {};
  require(THPVariable_Check(o), op, name, "a tensor is wanted");
  return THPVariable_Unpack(o);
}
long integer(PyObject* o, const char* op, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    require(false, op, name, "an integer is wanted");
  }
  require(v >= INT_MIN && v <= INT_MAX, op, name, "out of range");
  return v;
}
double number(PyObject* o, const char* op, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    require(false, op, name, "a number is wanted");
  }
  return v;
}
bool on(const at::Tensor& t, int device) { return t.is_cuda() && t.get_device() == device; }
const int32_t* ints(const at::Tensor& t, int64_t n, int device, const char* op, const char* name) {
  if (!t.defined()) return nullptr;
  require(t.scalar_type() == at::kInt && t.dim() == 1 && t.size(0) == n && on(t, device) && t.is_contiguous(), op, name,
          "a contiguous int32 tensor of the right length on the right device is wanted");
  return static_cast<const int32_t*>(t.const_data_ptr());
}
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, int device) {
  return at::detail::empty_cuda(sizes, type, c10::nullopt, at::Device(at::kCUDA, (c10::DeviceIndex)device), c10::nullopt, c10::nullopt);
}
void called(int rc, const char* what) {
  if (rc != MK_OK) throw Refused{rc, what};
}
mk_cache* handle(PyObject* o) {
  mk_cache* c = static_cast<mk_cache*>(PyLong_AsVoidPtr(o));
  if (!c) PyErr_Clear();
  require(c != nullptr, "Cache", "handle", "the cache is closed");
  return c;
}
int dtype_code(const at::Tensor& t, const char* op) {
  require(t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kFloat, op, "dtype", "bf16 or fp32 is wanted");
  return t.scalar_type() == at::kBFloat16 ? MK_DTYPE_BF16 : MK_DTYPE_FP32;
}

// append(handle, layer, k, v, seq_lens, q, starts, positions, q_norm, k_norm, q_out) -> q_out or None
PyObject* do_append(PyObject* const* a) {
  constexpr const char* kOp = "append";
  mk_cache* c = handle(a[0]);
  const mk_cache_desc& d = c->d;
  const int dev = c->device;
  const at::Tensor k = tensor(a[2], kOp, "k"), v = tensor(a[3], kOp, "v"), lens = tensor(a[4], kOp, "seq_lens"),
                   q = tensor(a[5], kOp, "q", true), starts = tensor(a[6], kOp, "starts", true),
                   positions = tensor(a[7], kOp, "positions", true), q_norm = tensor(a[8], kOp, "q_norm", true),
                   k_norm = tensor(a[9], kOp, "k_norm", true);
  at::Tensor q_out = tensor(a[10], kOp, "q_out", true);
  mk_append_args p = {};
  p.dtype = dtype_code(k, kOp);
  require(k.dim() == 3 && k.size(0) <= INT_MAX, kOp, "k", "a tensor [n][n_kv][hd] is wanted");
  const int64_t n = k.size(0);
  auto rows = [&](const at::Tensor& t, int heads, const char* name, int64_t& stride) {
    require(t.dim() == 3 && t.size(0) == n && t.size(1) == heads && t.size(2) == d.head_dim && t.scalar_type() == k.scalar_type() &&
                on(t, dev) && (n == 0 || (t.stride(2) == 1 && (t.stride(1) == d.head_dim || heads == 1))),
            kOp, name, "[n][heads][hd] of one type, the heads of a token contiguous, on the cache's device is wanted");
    stride = t.stride(0);
    return t.const_data_ptr();
  };
  p.k = rows(k, d.n_kv_heads, "k", p.k_stride);
  p.v = rows(v, d.n_kv_heads, "v", p.v_stride);
  if (q.defined()) {
    p.q = rows(q, d.n_q_heads, "q", p.q_stride);
    if (q_out.defined())
      require(q_out.sizes() == q.sizes() && q_out.scalar_type() == at::kBFloat16 && on(q_out, dev) && q_out.is_contiguous(), kOp,
              "q_out", "a contiguous bf16 tensor of q's shape is wanted");
    else
      q_out = empty({n, d.n_q_heads, d.head_dim}, at::kBFloat16, dev);
    p.q_out = q_out.mutable_data_ptr();
  } else {
    require(!q_out.defined(), kOp, "q_out", "there is no q");
  }
  require(starts.defined() || n == d.batch, kOp, "starts", "without them one token a sequence is wanted");
  p.starts = ints(starts, (int64_t)d.batch + 1, dev, kOp, "starts");
  p.seq_lens = ints(lens, d.batch, dev, kOp, "seq_lens");
  p.positions = ints(positions, n, dev, kOp, "positions");
  auto gain = [&](const at::Tensor& t, const char* name) -> const void* {
    if (!t.defined()) return nullptr;
    require(t.dim() == 1 && t.size(0) == d.head_dim && t.scalar_type() == at::kBFloat16 && on(t, dev) && t.is_contiguous(), kOp, name,
            "a contiguous bf16 tensor [hd] on the cache's device is wanted");
    return t.const_data_ptr();
  };
  p.q_norm = gain(q_norm, "q_norm");
  p.k_norm = gain(k_norm, "k_norm");
  p.n_tokens = (int32_t)n;
  called(mk_cache_append(c, (int)integer(a[1], kOp, "layer"), &p, c10::cuda::getCurrentCUDAStream(dev).stream()), "mk_cache_append");
  if (!q_out.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(q_out);
}

// attend(handle, layer, q, seq_lens, prefix_len, scale, out, lse, workspace) -> (out, lse)
PyObject* do_attend(PyObject* const* a) {
  constexpr const char* kOp = "attend";
  mk_cache* c = handle(a[0]);
  const mk_cache_desc& d = c->d;
  const int dev = c->device;
  const at::Tensor q = tensor(a[2], kOp, "q"), lens = tensor(a[3], kOp, "seq_lens");
  at::Tensor out = tensor(a[6], kOp, "out", true), lse = tensor(a[7], kOp, "lse", true), ws = tensor(a[8], kOp, "workspace", true);
  const double scale = number(a[5], kOp, "scale");
  require(scale == 0 || (float)scale != 0.f, kOp, "scale", "0, or a number that is not 0 in fp32, is wanted");
  const int64_t shape[3] = {d.batch, d.n_q_heads, d.head_dim};
  auto whole = [&](const at::Tensor& t, int dims, at::ScalarType type, const char* name) {
    require(t.sizes() == at::IntArrayRef(shape, dims) && t.scalar_type() == type && on(t, dev) && t.is_contiguous(), kOp, name,
            "a contiguous tensor of the right shape and type ([B][n_q][hd] bf16, [B][n_q] fp32) on the cache's device is wanted");
  };
  whole(q, 3, at::kBFloat16, "q");
  const int32_t* len = ints(lens, d.batch, dev, kOp, "seq_lens");
  const size_t need = mk_cache_attend_bytes(c);
  if (out.defined()) whole(out, 3, at::kBFloat16, "out");
  else out = empty(at::IntArrayRef(shape, 3), at::kBFloat16, dev);
  if (lse.defined()) whole(lse, 2, at::kFloat, "lse");
  else lse = empty(at::IntArrayRef(shape, 2), at::kFloat, dev);
  if (ws.defined()) require(on(ws, dev) && ws.is_contiguous(), kOp, "workspace", "a contiguous tensor on the cache's device is wanted");
  else ws = empty({(int64_t)need}, at::kByte, dev);
  called(mk_cache_attend(c, (int)integer(a[1], kOp, "layer"), q.const_data_ptr(), len, (int)integer(a[4], kOp, "prefix_len"), (float)scale,
                         out.mutable_data_ptr(), static_cast<float*>(lse.mutable_data_ptr()), ws.mutable_data_ptr(), ws.nbytes(),
                         c10::cuda::getCurrentCUDAStream(dev).stream()),
         "mk_cache_attend");
  PyObject* r = PyTuple_New(2);
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(out));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(lse));
  return r;
}

// token_logprobs(logits, tokens, top_k) -> (logprob, entropy, ids, logprobs of the ids)
PyObject* do_logprobs(PyObject* const* a) {
  constexpr const char* kOp = "token_logprobs";
  const at::Tensor x = tensor(a[0], kOp, "logits"), tokens = tensor(a[1], kOp, "tokens");
  const int64_t k = integer(a[2], kOp, "top_k");
  require(x.is_cuda() && x.dim() == 2 && (x.stride(1) == 1 || x.size(1) == 1) && x.size(0) <= INT_MAX && x.size(1) <= INT_MAX, kOp,
          "logits", "device logits [n][vocab] with contiguous rows are wanted");
  const int dev = x.get_device(), code = dtype_code(x, kOp);
  const int64_t n = x.size(0);
  const int32_t* tok = ints(tokens, n, dev, kOp, "tokens");
  require(k >= 0 && k <= 32, kOp, "top_k", "0 to 32 are wanted");
  const at::Tensor logprob = empty({n}, at::kFloat, dev), entropy = empty({n}, at::kFloat, dev), ids = empty({n, k}, at::kInt, dev),
                   best = empty({n, k}, at::kFloat, dev);
  called(mk_token_logprobs(x.const_data_ptr(), code, x.stride(0), (int)n, (int)x.size(1), tok, static_cast<float*>(logprob.mutable_data_ptr()),
                           static_cast<float*>(entropy.mutable_data_ptr()), (int)k, static_cast<int32_t*>(ids.mutable_data_ptr()),
                           static_cast<float*>(best.mutable_data_ptr()), dev, c10::cuda::getCurrentCUDAStream(dev).stream()),
         "mk_token_logprobs");
  PyObject* r = PyTuple_New(4);
  const at::Tensor* all[4] = {&logprob, &entropy, &ids, &best};
  for (int i = 0; i < 4; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(*all[i]));
  return r;
}

template <PyObject* (*Do)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are wanted", N);
    return nullptr;
  }
  try {
    return Do(a);
  } catch (const Refused& r) {
    return refuse(r.code, r.what);
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"append", (PyCFunction)(void (*)(void))entry<do_append, 11>, METH_FASTCALL, nullptr},
    {"attend", (PyCFunction)(void (*)(void))entry<do_attend, 9>, METH_FASTCALL, nullptr},
    {"token_logprobs", (PyCFunction)(void (*)(void))entry<do_logprobs, 3>, METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_mk_torch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mk_torch() { return PyModule_Create(&kModule); }
