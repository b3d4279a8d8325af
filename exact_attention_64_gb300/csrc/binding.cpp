// Python entry points of the calls that generation makes once per token
// (paged_decode, cache_append, cache_evict, key_weights, rotary_*): argument checks,
// output and workspace tensors, and the C ABI call, in one step of native code.
// Such a call takes a few microseconds on the GPU, and marshalling it in Python
// took about three times as long. Like the rest of the binding it only
// marshals; every check of values is the C ABI's own.
#include <Python.h>

#include <ATen/Functions.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <string>

#include "../../include/fa2.h"

namespace {

using at::Tensor;

[[noreturn]] void value_error(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw python_error();
}

// FA2Error(func, code) of the package.
[[noreturn]] void status_error(const char* func, int code) {
  PyObject* mod = PyImport_ImportModule("exact_attention_64_gb300");
  PyObject* cls = mod != nullptr ? PyObject_GetAttrString(mod, "FA2Error") : nullptr;
  PyObject* err = cls != nullptr ? PyObject_CallFunction(cls, "si", func, code) : nullptr;
  if (err != nullptr) PyErr_SetObject(cls, err);
  Py_XDECREF(err);
  Py_XDECREF(cls);
  Py_XDECREF(mod);
  throw python_error();
}

const Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) value_error(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

using Sizes = std::initializer_list<int64_t>;

// A contiguous tensor of this shape and type on CUDA device `dev`: its address.
template <class T = void>
T* need(const char* name, const Tensor& t, Sizes shape, at::ScalarType type, int dev) {
  const auto s = t.sizes();
  const bool same = s.size() == shape.size() && std::equal(s.begin(), s.end(), shape.begin());
  if (!t.is_cuda() || t.get_device() != dev)
    value_error(std::string(name) + " must be a CUDA tensor on cuda:" + std::to_string(dev < 0 ? 0 : dev));
  if (!same || t.scalar_type() != type) {
    std::string m = std::string(name) + " must have shape (";
    for (const int64_t x : shape) m += std::to_string(x) + ", ";
    if (shape.size() > 0) m.resize(m.size() - 2);
    value_error(m + ") and dtype " + c10::toString(type));
  }
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  return static_cast<T*>(t.data_ptr());
}
template <class T = void>
T* need_opt(const char* name, PyObject* o, Sizes shape, at::ScalarType type, int dev) {
  return o == Py_None ? nullptr : need<T>(name, tensor(name, o), shape, type, dev);
}

// The caller's tensor, or a new one.
Tensor output(const char* name, PyObject* o, Sizes shape, at::ScalarType type, int dev) {
  if (o == Py_None)
    return at::empty(at::IntArrayRef(shape.begin(), shape.size()),
                     at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)));
  const Tensor& t = tensor(name, o);
  need(name, t, shape, type, dev);
  return t;
}

struct Space {
  Tensor t;
  size_t bytes;
};
Space workspace(PyObject* o, size_t need_bytes, const char* func, int dev) {
  if (need_bytes == 0) status_error(func, FA2_ERR_INVALID_ARG);
  if (o == Py_None)
    return {at::empty({static_cast<int64_t>(need_bytes)},
                      at::TensorOptions().dtype(at::kByte).device(at::kCUDA, static_cast<c10::DeviceIndex>(dev))),
            need_bytes};
  const Tensor& t = tensor("workspace", o);
  if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
    value_error("workspace must be a contiguous tensor on cuda:" + std::to_string(dev));
  return {t, t.nbytes()};
}

int dtype_code(const char* name, const Tensor& t) {
  if (t.scalar_type() == at::kHalf) return FA2_FP16;
  if (t.scalar_type() == at::kBFloat16) return FA2_BF16;
  value_error(std::string(name) + " must be float16 or bfloat16");
}

float scale_of(PyObject* o, int64_t d) {
  if (o == Py_None) return static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(x);
}

// Sizes go to the C ABI as int.
int as_int(const char* name, int64_t x) {
  if (x < 0 || x > INT32_MAX) value_error(std::string(name) + " does not fit in 31 bits");
  return static_cast<int>(x);
}

// Runs an entry point on the tensors' device and its current stream.
template <class F>
void run(const char* func, int dev, F call) {
  const c10::cuda::OptionalCUDAGuard guard(
      c10::cuda::current_device() == dev
          ? std::nullopt
          : std::optional<c10::Device>(c10::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev))));
  void* stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  int code = 0;
  Py_BEGIN_ALLOW_THREADS;
  code = call(stream);
  Py_END_ALLOW_THREADS;
  if (code != FA2_OK) status_error(func, code);
}

struct Cache {
  void *k, *v;
  int *table, *lens;
  int pages, Hkv, ps, d, B, width;
  int64_t L;
  int dtype, dev;
  at::ScalarType type;
};

Cache cache_of(PyObject* ko, PyObject* vo, PyObject* to, PyObject* lo) {
  const Tensor &k = tensor("k_cache", ko), &v = tensor("v_cache", vo), &t = tensor("table", to);
  Cache c{};
  if (!k.is_cuda()) value_error("k_cache must be a CUDA tensor");
  if (k.dim() != 4) value_error("expected a [num_pages, Hkv, page_size, d] cache");
  c.dtype = dtype_code("k_cache", k);
  if (t.dim() != 2) value_error("expected a [B, max_pages] table");
  c.dev = k.get_device();
  c.type = k.scalar_type();
  const Sizes shape = {k.size(0), k.size(1), k.size(2), k.size(3)};
  c.pages = as_int("num_pages", k.size(0));
  c.Hkv = as_int("Hkv", k.size(1));
  c.ps = as_int("page_size", k.size(2));
  c.d = as_int("d", k.size(3));
  c.B = as_int("B", t.size(0));
  c.width = as_int("max_pages", t.size(1));
  c.L = t.size(1) * k.size(2);
  c.k = need("k_cache", k, shape, c.type, c.dev);
  c.v = need("v_cache", v, shape, c.type, c.dev);
  c.table = need<int>("table", t, {c.B, c.width}, at::kInt, c.dev);
  c.lens = need<int>("lens", tensor("lens", lo), {c.B}, at::kInt, c.dev);
  return c;
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

// q, k_cache, v_cache, table, lens, scale, weights, weights_out, out, lse, workspace
PyObject* paged_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arity(n, 11)) return nullptr;
  const Cache c = cache_of(a[1], a[2], a[3], a[4]);
  const Tensor& q = tensor("q", a[0]);
  if (q.dim() != 3) value_error("expected a [B, Hq, d] query");
  const int64_t Hq = q.size(1);
  const void* qp = need("q", q, {c.B, Hq, c.d}, c.type, c.dev);
  if (a[6] == Py_None && a[7] != Py_None) value_error("weights_out needs weights");
  float* w = need_opt<float>("weights", a[6], {c.B, c.Hkv, c.L}, at::kFloat, c.dev);
  float* wo = a[7] == Py_None ? w : need_opt<float>("weights_out", a[7], {c.B, c.Hkv, c.L}, at::kFloat, c.dev);
  const float scale = scale_of(a[5], c.d);
  const int hq = as_int("Hq", Hq);
  const Tensor o = output("out", a[8], {c.B, Hq, c.d}, c.type, c.dev);
  const Tensor lse = output("lse", a[9], {c.B, Hq}, at::kFloat, c.dev);
  const Space ws = workspace(a[10], fa2_paged_decode_workspace_size(c.B, hq, c.Hkv, c.d, c.ps, c.width, w != nullptr),
                             "fa2_paged_decode_workspace_size", c.dev);
  void* op = o.data_ptr();
  float* lp = static_cast<float*>(lse.data_ptr());
  void* wp = ws.t.data_ptr();
  run("fa2_paged_decode", c.dev, [&](void* stream) {
    return fa2_paged_decode(qp, c.k, c.v, c.table, c.lens, w, wo, op, lp, c.B, hq, c.Hkv, c.d, c.pages, c.ps, c.width,
                            scale, c.dtype, wp, ws.bytes, stream);
  });
  PyObject* r0 = THPVariable_Wrap(o);
  PyObject* r1 = THPVariable_Wrap(lse);
  PyObject* r = PyTuple_Pack(2, r0, r1);
  Py_XDECREF(r0);
  Py_XDECREF(r1);
  return r;
  END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, table, lens, prefix, prefix_len, scale, out, lse, workspace
PyObject* prefix_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arity(n, 11)) return nullptr;
  const Cache c = cache_of(a[1], a[2], a[3], a[4]);
  const Tensor &q = tensor("q", a[0]), &p = tensor("prefix", a[5]);
  if (q.dim() != 3) value_error("expected a [B, Hq, d] query");
  if (p.dim() != 1) value_error("expected a [prefix_pages] prefix");
  const int64_t Hq = q.size(1);
  const void* qp = need("q", q, {c.B, Hq, c.d}, c.type, c.dev);
  const int hq = as_int("Hq", Hq), pages = as_int("prefix_pages", p.size(0));
  const int* pp = need<int>("prefix", p, {pages}, at::kInt, c.dev);
  const int* pl = need<int>("prefix_len", tensor("prefix_len", a[6]), {1}, at::kInt, c.dev);
  const float scale = scale_of(a[7], c.d);
  const Tensor o = output("out", a[8], {c.B, Hq, c.d}, c.type, c.dev);
  const Tensor lse = output("lse", a[9], {c.B, Hq}, at::kFloat, c.dev);
  const Space ws = workspace(a[10], fa2_prefix_decode_workspace_size(c.B, hq, c.Hkv, c.d, c.ps, c.width),
                             "fa2_prefix_decode_workspace_size", c.dev);
  void* op = o.data_ptr();
  float* lp = static_cast<float*>(lse.data_ptr());
  void* wp = ws.t.data_ptr();
  run("fa2_prefix_decode", c.dev, [&](void* stream) {
    return fa2_prefix_decode(qp, c.k, c.v, c.table, c.lens, pp, pl, op, lp, c.B, hq, c.Hkv, c.d, c.pages, c.ps, c.width,
                             pages, scale, c.dtype, wp, ws.bytes, stream);
  });
  PyObject* r0 = THPVariable_Wrap(o);
  PyObject* r1 = THPVariable_Wrap(lse);
  PyObject* r = PyTuple_Pack(2, r0, r1);
  Py_XDECREF(r0);
  Py_XDECREF(r1);
  return r;
  END_HANDLE_TH_ERRORS
}

// k, v, k_cache, v_cache, table, lens, num_new, weights, new_weights, positions, next_pos, lens_out
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arity(n, 12)) return nullptr;
  const Cache c = cache_of(a[2], a[3], a[4], a[5]);
  const Tensor& k = tensor("k", a[0]);
  if (k.dim() != 4) value_error("expected [B, Hkv, T, d] keys");
  const int64_t T = k.size(2);
  const void* kp = need("k", k, {c.B, c.Hkv, T, c.d}, c.type, c.dev);
  const void* vp = need("v", tensor("v", a[1]), {c.B, c.Hkv, T, c.d}, c.type, c.dev);
  if (a[8] != Py_None && a[7] == Py_None) value_error("new_weights needs weights");
  if ((a[9] == Py_None) != (a[10] == Py_None)) value_error("positions and next_pos go together");
  const int* num = need_opt<int>("num_new", a[6], {c.B}, at::kInt, c.dev);
  float* w = need_opt<float>("weights", a[7], {c.B, c.Hkv, c.L}, at::kFloat, c.dev);
  const float* nw = need_opt<float>("new_weights", a[8], {c.B, c.Hkv, T}, at::kFloat, c.dev);
  int* pos = need_opt<int>("positions", a[9], {c.B, c.Hkv, c.L}, at::kInt, c.dev);
  const int* next = need_opt<int>("next_pos", a[10], {c.B}, at::kInt, c.dev);
  const int t = as_int("T", T);
  const Tensor out = output("lens_out", a[11], {c.B}, at::kInt, c.dev);
  int* lp = static_cast<int*>(out.data_ptr());
  run("fa2_cache_append", c.dev, [&](void* stream) {
    return fa2_cache_append(kp, vp, c.k, c.v, c.table, c.lens, num, w, nw, pos, next, lp, c.B, c.Hkv, t, c.d, c.pages,
                            c.ps, c.width, c.dtype, stream);
  });
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// k_cache, v_cache, table, lens, weights, budget, recent, positions, next_pos, weights_out, positions_out, lens_out,
// workspace
PyObject* cache_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arity(n, 13)) return nullptr;
  const Cache c = cache_of(a[0], a[1], a[2], a[3]);
  const float* w = need<float>("weights", tensor("weights", a[4]), {c.B, c.Hkv, c.L}, at::kFloat, c.dev);
  int64_t budget = PyLong_AsLongLong(a[5]), recent = PyLong_AsLongLong(a[6]);
  if (PyErr_Occurred()) throw python_error();
  if (budget < 1 || recent < 0 || recent > budget) value_error("needs budget >= 1 and 0 <= recent <= budget");
  // No sequence is longer than a table: more changes nothing.
  budget = std::min<int64_t>(budget, INT32_MAX);
  recent = std::min<int64_t>(recent, INT32_MAX);
  float* wo = a[9] == Py_None ? const_cast<float*>(w)
                              : need_opt<float>("weights_out", a[9], {c.B, c.Hkv, c.L}, at::kFloat, c.dev);
  if ((a[7] == Py_None) != (a[8] == Py_None)) value_error("positions and next_pos go together");
  if (a[7] == Py_None && a[10] != Py_None) value_error("positions_out needs positions");
  int* p = need_opt<int>("positions", a[7], {c.B, c.Hkv, c.L}, at::kInt, c.dev);
  int* po = a[10] == Py_None ? p : need_opt<int>("positions_out", a[10], {c.B, c.Hkv, c.L}, at::kInt, c.dev);
  const int* next = need_opt<int>("next_pos", a[8], {c.B}, at::kInt, c.dev);
  const Tensor out = output("lens_out", a[11], {c.B}, at::kInt, c.dev);
  const Space ws = workspace(a[12], fa2_cache_evict_workspace_size(c.B, c.Hkv, c.ps, c.width, static_cast<int>(budget)),
                             "fa2_cache_evict_workspace_size", c.dev);
  int* lp = static_cast<int*>(out.data_ptr());
  void* wp = ws.t.data_ptr();
  run("fa2_cache_evict", c.dev, [&](void* stream) {
    return fa2_cache_evict(c.k, c.v, c.table, c.lens, w, wo, p, po, next, lp, c.B, c.Hkv, c.d, c.pages, c.ps, c.width,
                           static_cast<int>(budget), static_cast<int>(recent), c.dtype, wp, ws.bytes, stream);
  });
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// table, lens, new_lens, refs, free_pages, num_free, page_size, lens_out, workspace
PyObject* cache_resize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arity(n, 9)) return nullptr;
  const Tensor &t = tensor("table", a[0]), &r = tensor("refs", a[3]);
  if (!t.is_cuda()) value_error("table must be a CUDA tensor");
  if (t.dim() != 2) value_error("expected a [B, max_pages] table");
  if (r.dim() != 1) value_error("expected refs of [num_pages]");
  const int dev = t.get_device(), B = as_int("B", t.size(0)), width = as_int("max_pages", t.size(1)),
            pages = as_int("num_pages", r.size(0));
  const int64_t size = PyLong_AsLongLong(a[6]);
  if (PyErr_Occurred()) throw python_error();
  if (size < 1) value_error("page_size must be at least 1");
  const int ps = as_int("page_size", size);
  int* tp = need<int>("table", t, {B, width}, at::kInt, dev);
  const int* lp = need<int>("lens", tensor("lens", a[1]), {B}, at::kInt, dev);
  const int* np = need<int>("new_lens", tensor("new_lens", a[2]), {B}, at::kInt, dev);
  int* rp = need<int>("refs", r, {pages}, at::kInt, dev);
  int* fp = need<int>("free_pages", tensor("free_pages", a[4]), {pages}, at::kInt, dev);
  int* cp = need<int>("num_free", tensor("num_free", a[5]), {1}, at::kInt, dev);
  const Tensor out = output("lens_out", a[7], {B}, at::kInt, dev);
  const Space ws = workspace(a[8], fa2_cache_resize_workspace_size(B, pages, ps, width), "fa2_cache_resize_workspace_size",
                             dev);
  int* op = static_cast<int*>(out.data_ptr());
  void* wp = ws.t.data_ptr();
  run("fa2_cache_resize", dev, [&](void* stream) {
    return fa2_cache_resize(tp, lp, np, rp, fp, cp, op, B, pages, ps, width, wp, ws.bytes, stream);
  });
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// q, k, lse, causal, scale, q_lens, out, workspace
PyObject* key_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arity(n, 8)) return nullptr;
  const Tensor &q = tensor("q", a[0]), &k = tensor("k", a[1]);
  if (q.dim() != 4 || k.dim() != 4) value_error("expected a [B, H, N, d] tensor");
  if (!q.is_cuda()) value_error("q must be a CUDA tensor");
  const int dtype = dtype_code("q", q), dev = q.get_device();
  const at::ScalarType type = q.scalar_type();
  const int64_t B = q.size(0), Hq = q.size(1), N = q.size(2), d = q.size(3), Hkv = k.size(1), Nk = k.size(2);
  const void* qp = need("q", q, {B, Hq, N, d}, type, dev);
  const void* kp = need("k", k, {B, Hkv, Nk, d}, type, dev);
  const float* lp = need<float>("lse", tensor("lse", a[2]), {B, Hq, N}, at::kFloat, dev);
  const int causal = PyObject_IsTrue(a[3]);
  if (causal < 0) throw python_error();
  const float scale = scale_of(a[4], d);
  const int* ql = need_opt<int>("q_lens", a[5], {B}, at::kInt, dev);
  const int b = as_int("B", B), hq = as_int("Hq", Hq), hkv = as_int("Hkv", Hkv), nq = as_int("N", N),
            nk = as_int("N_k", Nk), dd = as_int("d", d);
  const Tensor out = output("out", a[6], {B, Hkv, Nk}, at::kFloat, dev);
  const Space ws = workspace(a[7], fa2_key_weights_workspace_size(), "fa2_key_weights_workspace_size", dev);
  float* op = static_cast<float*>(out.data_ptr());
  void* wp = ws.t.data_ptr();
  run("fa2_key_weights", dev, [&](void* stream) {
    return fa2_key_weights(qp, kp, lp, ql, op, b, hq, hkv, nq, nk, dd, causal, scale, dtype, wp, ws.bytes, stream);
  });
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// A [B, H, N, d] tensor of any strides whose rows are contiguous: its address, and
// its strides of batch, head and token into `st`.
void* need_rows(const char* name, const Tensor& t, Sizes shape, at::ScalarType type, int dev, long long* st) {
  const auto s = t.sizes();
  if (!t.is_cuda() || t.get_device() != dev)
    value_error(std::string(name) + " must be a CUDA tensor on cuda:" + std::to_string(dev < 0 ? 0 : dev));
  if (s.size() != 4 || !std::equal(s.begin(), s.end(), shape.begin()) || t.scalar_type() != type) {
    std::string m = std::string(name) + " must have shape (";
    for (const int64_t x : shape) m += std::to_string(x) + ", ";
    m.resize(m.size() - 2);
    value_error(m + ") and dtype " + c10::toString(type));
  }
  if (t.stride(3) != 1) value_error(std::string(name) + " must have contiguous rows");
  for (int i = 0; i < 3; ++i) st[i] = s[i] > 1 ? t.stride(i) : 0;
  return t.data_ptr();
}

struct Rotary {
  int B, Hq, Hk, N, d, r, pos_mode, interleaved, dtype, wtype, dev;
  at::ScalarType type, weight;
  float eps, amplitude;
  const double* freqs;
  const int* positions;
  void *qw, *kw;
};

float float_of(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(x);
}

// The arguments that both directions share; q and k: the tensors to turn.
Rotary rotary_of(const Tensor& q, PyObject* ko, PyObject* fo, PyObject* po, PyObject* inter, PyObject* qw, PyObject* kw,
                 PyObject* eps, PyObject* amp) {
  if (!q.is_cuda()) value_error("q must be a CUDA tensor");
  if (q.dim() != 4) value_error("expected a [B, H, N, d] tensor");
  Rotary a{};
  a.dtype = dtype_code("q", q);
  a.type = q.scalar_type();
  a.dev = q.get_device();
  a.B = as_int("B", q.size(0));
  a.Hq = as_int("Hq", q.size(1));
  a.N = as_int("N", q.size(2));
  a.d = as_int("d", q.size(3));
  if (ko != Py_None) {
    const Tensor& k = tensor("k", ko);
    if (k.dim() != 4) value_error("expected a [B, H, N, d] tensor");
    a.Hk = as_int("Hkv", k.size(1));
    if (a.Hk == 0) value_error("k has no heads");
  }
  const Tensor& f = tensor("freqs", fo);
  if (f.dim() != 1) value_error("freqs must be one-dimensional");
  a.r = as_int("rotary_dim", 2 * f.size(0));
  a.freqs = need<double>("freqs", f, {f.size(0)}, at::kDouble, a.dev);
  if (po != Py_None) {
    const Tensor& p = tensor("positions", po);
    a.pos_mode = p.dim() == 2 ? 2 : 1;
    a.positions = a.pos_mode == 2 ? need<int>("positions", p, {a.B, a.N}, at::kInt, a.dev)
                                  : need<int>("positions", p, {a.B}, at::kInt, a.dev);
  }
  a.interleaved = PyObject_IsTrue(inter);
  if (a.interleaved < 0) throw python_error();
  if ((qw == Py_None) != (kw == Py_None) && ko != Py_None) value_error("q_weight and k_weight go together");
  if (ko == Py_None && kw != Py_None) value_error("k_weight needs k");
  a.weight = a.type;
  if (qw != Py_None) {
    const Tensor& w = tensor("q_weight", qw);
    if (w.scalar_type() == at::kFloat) a.weight = at::kFloat;
    a.qw = need("q_weight", w, {a.d}, a.weight, a.dev);
    if (kw != Py_None) a.kw = need("k_weight", tensor("k_weight", kw), {a.d}, a.weight, a.dev);
  }
  a.wtype = a.weight == at::kFloat ? FA2_FP32 : a.dtype;
  a.eps = float_of(eps);
  a.amplitude = float_of(amp);
  return a;
}

// The caller's strided tensor, or a new one laid out like `like` (or contiguous).
Tensor rows_output(const char* name, PyObject* o, Sizes shape, const Rotary& a, const Tensor* like, long long* st) {
  const Tensor t = o != Py_None ? tensor(name, o)
                   : like != nullptr
                       ? at::empty_like(*like)
                       : at::empty(at::IntArrayRef(shape.begin(), shape.size()),
                                   at::TensorOptions().dtype(a.type).device(at::kCUDA, static_cast<c10::DeviceIndex>(a.dev)));
  need_rows(name, t, shape, a.type, a.dev, st);
  return t;
}

PyObject* pack_results(std::initializer_list<const Tensor*> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (r == nullptr) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor* t : ts) {
    PyObject* x = Py_None;
    if (t->defined()) x = THPVariable_Wrap(*t);
    else Py_INCREF(x);
    PyTuple_SET_ITEM(r, i++, x);
  }
  return r;
}

// q, k, freqs, positions, interleaved, q_weight, k_weight, eps, amplitude, q_out, k_out
PyObject* rotary_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arity(n, 11)) return nullptr;
  const Tensor& q = tensor("q", a[0]);
  const Rotary r = rotary_of(q, a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8]);
  long long st[12] = {};
  const Sizes qs = {r.B, r.Hq, r.N, r.d}, ks = {r.B, r.Hk, r.N, r.d};
  const void* qp = need_rows("q", q, qs, r.type, r.dev, st);
  const void* kp = r.Hk > 0 ? need_rows("k", tensor("k", a[1]), ks, r.type, r.dev, st + 3) : nullptr;
  if (r.Hk == 0 && a[10] != Py_None) value_error("k_out needs k");
  const Tensor qo = rows_output("q_out", a[9], qs, r, nullptr, st + 6);
  Tensor ko;
  if (r.Hk > 0) ko = rows_output("k_out", a[10], ks, r, nullptr, st + 9);
  void *qop = qo.data_ptr(), *kop = r.Hk > 0 ? ko.data_ptr() : nullptr;
  run("fa2_rotary_fwd", r.dev, [&](void* stream) {
    return fa2_rotary_fwd(qp, kp, r.freqs, r.positions, r.qw, r.kw, qop, kop, st, r.B, r.Hq, r.Hk, r.N, r.d, r.r,
                          r.pos_mode, r.interleaved, r.eps, r.amplitude, r.dtype, r.wtype, stream);
  });
  return pack_results({&qo, &ko});
  END_HANDLE_TH_ERRORS
}

// dq, dk, freqs, positions, interleaved, q, k, q_weight, k_weight, eps, amplitude, q_grad, k_grad, workspace
PyObject* rotary_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!arity(n, 14)) return nullptr;
  const Tensor& dq = tensor("dq", a[0]);
  const Rotary r = rotary_of(dq, a[1], a[2], a[3], a[4], a[7], a[8], a[9], a[10]);
  const bool norm = r.qw != nullptr, both = r.Hk > 0;
  if (norm && (a[5] == Py_None || (both && a[6] == Py_None))) value_error("the gradients of a norm need q and k");
  if (!both && (a[6] != Py_None || a[12] != Py_None)) value_error("k and k_grad need dk");
  long long st[18] = {};
  const Sizes qs = {r.B, r.Hq, r.N, r.d}, ks = {r.B, r.Hk, r.N, r.d};
  const void* dqp = need_rows("dq", dq, qs, r.type, r.dev, st);
  const void* dkp = both ? need_rows("dk", tensor("dk", a[1]), ks, r.type, r.dev, st + 3) : nullptr;
  // Without a norm q and k only say how the new gradients are laid out.
  const Tensor* ql = a[5] != Py_None ? &tensor("q", a[5]) : nullptr;
  const Tensor* kl = both && a[6] != Py_None ? &tensor("k", a[6]) : nullptr;
  const void* qp = ql != nullptr ? need_rows("q", *ql, qs, r.type, r.dev, st + 6) : nullptr;
  const void* kp = kl != nullptr ? need_rows("k", *kl, ks, r.type, r.dev, st + 9) : nullptr;
  const Tensor qg = rows_output("q_grad", a[11], qs, r, ql, st + 12);
  Tensor kg, qwg, kwg;
  if (both) kg = rows_output("k_grad", a[12], ks, r, kl, st + 15);
  Space ws{};
  if (norm) {
    const auto opt = at::TensorOptions().dtype(r.weight).device(at::kCUDA, static_cast<c10::DeviceIndex>(r.dev));
    qwg = at::empty({r.d}, opt);
    if (both) kwg = at::empty({r.d}, opt);
    ws = workspace(a[13], fa2_rotary_bwd_workspace_size(r.B, r.Hq, r.Hk, r.N, r.d, 1), "fa2_rotary_bwd_workspace_size",
                   r.dev);
  }
  void *qgp = qg.data_ptr(), *kgp = both ? kg.data_ptr() : nullptr;
  void *qwp = norm ? qwg.data_ptr() : nullptr, *kwp = norm && both ? kwg.data_ptr() : nullptr;
  void* wp = norm ? ws.t.data_ptr() : nullptr;
  run("fa2_rotary_bwd", r.dev, [&](void* stream) {
    return fa2_rotary_bwd(dqp, dkp, norm ? qp : nullptr, norm ? kp : nullptr, r.freqs, r.positions, r.qw, r.kw, qgp, kgp,
                          qwp, kwp, st, r.B, r.Hq, r.Hk, r.N, r.d, r.r, r.pos_mode, r.interleaved, r.eps, r.amplitude,
                          r.dtype, r.wtype, wp, ws.bytes, stream);
  });
  return pack_results({&qg, &kg, &qwg, &kwg});
  END_HANDLE_TH_ERRORS
}

#define FA2_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FA2_METHOD(paged_decode), FA2_METHOD(cache_append), FA2_METHOD(cache_evict),
                           FA2_METHOD(key_weights), FA2_METHOD(rotary_forward), FA2_METHOD(rotary_backward),
                           FA2_METHOD(cache_resize), FA2_METHOD(prefix_decode), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&g_module); }
