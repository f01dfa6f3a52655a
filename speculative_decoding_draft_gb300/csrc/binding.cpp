// The binding of the operators around a ragged verification step: argument checks, output tensors and
// the call, as one extension function each.  A kernel of these takes from 3 us on; the same checks in
// Python took 13 us a call.
//
// Every function takes its arguments by position (serving.py gives them their names and defaults) and
// the addresses of the C ABI's entry points come from the loaded library (init), whichever build of it
// that is.  It returns the result's dict, or the entry point's error code as an int.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <optional>
#include <string>

#include "dspark.h"

namespace {

struct {
  decltype(&dspark_attn_norm_rope) norm_rope;
  decltype(&dspark_attn_append) append;
  decltype(&dspark_attn_cache_read) read;
  decltype(&dspark_attn_paged_workspace_bytes) workspace_bytes;
  decltype(&dspark_attn_paged) paged;
  decltype(&dspark_logits_penalize) penalize;
  decltype(&dspark_attn_prompt_workspace_bytes) prompt_workspace_bytes;
  decltype(&dspark_attn_prompt) prompt;
  decltype(&dspark_attn_append_byte) append_byte;
  decltype(&dspark_attn_cache_read_byte) read_byte;
  decltype(&dspark_attn_paged_byte_workspace_bytes) paged_byte_workspace_bytes;
  decltype(&dspark_attn_paged_byte) paged_byte;
} api;

struct Refused {};   // a Python error is set

[[noreturn]] void refuse(PyObject *kind, const std::string &what) {
  PyErr_SetString(kind, what.c_str());
  throw Refused();
}

std::string text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor &cuda_tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) refuse(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
  return THPVariable_Unpack(o);
}

void check(const at::Tensor &t, const char *name, at::ScalarType dtype, at::IntArrayRef shape, int dev) {
  if (t.scalar_type() != dtype)
    refuse(PyExc_TypeError, std::string(name) + " must have dtype " + c10::toString(dtype) + ", got " + c10::toString(t.scalar_type()));
  if (t.sizes() != shape) refuse(PyExc_ValueError, std::string(name) + " must have shape " + text(shape) + ", got " + text(t.sizes()));
  if (t.get_device() != dev)
    refuse(PyExc_ValueError, std::string(name) + " must be on cuda:" + std::to_string(dev) + ", got " + t.device().str());
}

// The address of a contiguous CUDA tensor of this type, shape and device.
template <class T = void>
T *like(PyObject *o, const char *name, at::ScalarType dtype, at::IntArrayRef shape, int dev) {
  const at::Tensor &t = cuda_tensor(o, name);
  check(t, name, dtype, shape, dev);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
  return (T *)t.data_ptr();
}

template <class T = void>
T *maybe(PyObject *o, const char *name, at::ScalarType dtype, at::IntArrayRef shape, int dev) {
  return o == Py_None ? nullptr : like<T>(o, name, dtype, shape, dev);
}

// A norm weight [dim] or None, which the kernels read 16 bytes at a time.
const void *weight(PyObject *o, const char *name, at::ScalarType dtype, int64_t dim, int dev) {
  const void *p = maybe(o, name, dtype, {dim}, dev);
  if ((uintptr_t)p % 16) refuse(PyExc_ValueError, std::string(name) + " must start on a 16-byte boundary");
  return p;
}

// A [rows, heads, dim] tensor whose last dimension is dense; rows and heads may be strided.
dspark_heads heads(PyObject *o, const char *name, at::ScalarType dtype, int64_t rows, int64_t n, int64_t dim, int dev) {
  const at::Tensor &t = cuda_tensor(o, name);
  check(t, name, dtype, {rows, n, dim}, dev);
  const int64_t unit = dtype == at::kFloat ? 4 : 8, sr = t.stride(0), sh = t.stride(1);
  if (t.stride(2) != 1 || (rows > 1 && sr % unit) || (n > 1 && sh % unit) || (uintptr_t)t.data_ptr() % 16)
    refuse(PyExc_ValueError, std::string(name) + " must have a dense last dimension and rows and heads on 16-byte boundaries");
  return {t.data_ptr(), rows > 1 ? sr : 0, n > 1 ? sh : 0};
}

int dtype_code(const at::Tensor &t, const char *name, std::initializer_list<at::ScalarType> allowed) {
  for (at::ScalarType a : allowed)
    if (t.scalar_type() == a) return a == at::kFloat ? DSPARK_F32 : (a == at::kBFloat16 ? DSPARK_BF16 : DSPARK_F16);
  std::string list;
  for (at::ScalarType a : allowed) list += (list.empty() ? "" : ", ") + std::string(c10::toString(a));
  refuse(PyExc_TypeError, std::string(name) + " must be one of " + list + ", got " + c10::toString(t.scalar_type()));
}

dspark_ragged ragged(PyObject *row_off, PyObject *kv_len, PyObject *table, int64_t rows, int dev) {
  const at::Tensor &t = cuda_tensor(table, "page_table");
  if (t.dim() != 2) refuse(PyExc_ValueError, "page_table must be [B, max_pages] int32");
  const int64_t B = t.size(0), width = t.size(1);
  return {like<int32_t>(row_off, "row_off", at::kInt, {B + 1}, dev), like<int32_t>(kv_len, "kv_len", at::kInt, {B}, dev),
          like<int32_t>(table, "page_table", at::kInt, {B, width}, dev), B, rows, width};
}

void *address(PyObject *o) {
  void *p = o == Py_None ? nullptr : PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Refused();
  return p;
}

// The stream of a call.  A given one is the current one for as long as this lives: what the call allocates, the fill
// of its status word and its kernels follow one another on it, and memory that the caller drops at once is not used
// again before they are done.  What it returns counts as used by the caller's current stream too.
class Stream {
 public:
  Stream(PyObject *given, int dev) : dev_((c10::DeviceIndex)dev) {
    if (given == Py_None) return;
    const cudaStream_t s = (cudaStream_t)address(given);
    before_ = c10::cuda::getCurrentCUDAStream(dev_);
    here_.reset_stream(s && s != cudaStreamLegacy ? c10::cuda::getStreamFromExternal(s, dev_)
                                                  : c10::cuda::getDefaultCUDAStream(dev_));
  }
  int device() const { return dev_; }
  void *raw() const { return (void *)c10::cuda::getCurrentCUDAStream(dev_).stream(); }
  // A Python object of a tensor that the call has made.
  PyObject *hand_out(at::Tensor t) const {
    if (before_ && before_->stream() != raw()) t.record_stream(before_->unwrap());
    PyObject *o = THPVariable_Wrap(std::move(t));
    if (!o) throw Refused();
    return o;
  }

 private:
  c10::DeviceIndex dev_;
  std::optional<c10::cuda::CUDAStream> before_;
  c10::cuda::OptionalCUDAStreamGuard here_;
};

// out[key], checked, or a new tensor.
struct Result {
  PyObject *object = nullptr;
  void *data = nullptr;
  Result() = default;
  Result(const Result &) = delete;
  ~Result() { Py_XDECREF(object); }
  void make(PyObject *out, const char *key, at::ScalarType dtype, at::IntArrayRef shape, const Stream &on) {
    const int dev = on.device();
    PyObject *given = out == Py_None ? nullptr : PyDict_GetItemString(out, key);
    if (given && given != Py_None) {
      data = like(given, (std::string("out['") + key + "']").c_str(), dtype, shape, dev);
      Py_INCREF(given);
      object = given;
    } else {
      at::Tensor t = at::empty(shape, at::TensorOptions(dtype).device(at::kCUDA, (c10::DeviceIndex)dev));
      data = t.data_ptr();
      object = on.hand_out(std::move(t));
    }
  }
  // The given workspace where it is fit for `need` bytes, or a new one; returns its bytes.
  int64_t workspace(PyObject *given, int64_t need, const Stream &on) {
    if (!need) return 0;
    if (given != Py_None) {
      const at::Tensor &w = cuda_tensor(given, "workspace");
      const bool fit = w.is_contiguous() && w.get_device() == on.device() && (uintptr_t)w.data_ptr() % 256 == 0;
      if (fit && (int64_t)w.nbytes() >= need) {
        data = w.data_ptr();
        Py_INCREF(given);
        object = given;
        return (int64_t)w.nbytes();
      }
    }
    make(Py_None, "workspace", at::kByte, {need}, on);
    return need;
  }
  void status(PyObject *given, const Stream &on) {
    const int dev = on.device();
    if (given != Py_None) {
      data = like(given, "status", at::kInt, {1}, dev);
      Py_INCREF(given);
      object = given;
    } else {
      at::Tensor t = at::zeros({1}, at::TensorOptions(at::kInt).device(at::kCUDA, (c10::DeviceIndex)dev));
      data = t.data_ptr();
      object = on.hand_out(std::move(t));
    }
  }
};

PyObject *answer(std::initializer_list<std::pair<const char *, const Result *>> parts) {
  PyObject *d = PyDict_New();
  if (!d) throw Refused();
  for (const auto &p : parts)
    if (PyDict_SetItemString(d, p.first, p.second->object ? p.second->object : Py_None)) {
      Py_DECREF(d);
      throw Refused();
    }
  return d;
}

int64_t whole(PyObject *o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
double real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return v;
}
void out_is_dict(PyObject *out) {
  if (out != Py_None && !PyDict_Check(out)) refuse(PyExc_TypeError, "out must be a dict");
}

// No C++ exception leaves a function of the module.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  try {
    if (n != N) refuse(PyExc_TypeError, "expected " + std::to_string(N) + " arguments, got " + std::to_string(n));
    return F(args);
  } catch (const Refused &) {
  } catch (const std::exception &e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

const dspark_rope *rope_for(PyObject *rope, int64_t d) {
  const auto *r = (const dspark_rope *)address(rope);
  if (r && r->rotary_dim > d)
    refuse(PyExc_ValueError, "rope turns " + std::to_string(r->rotary_dim) + " dimensions of heads with " + std::to_string(d));
  return r;
}

// q, k, positions, rope, q_weight, k_weight, eps, out, status, stream
PyObject *norm_rope(PyObject *const *v) {
  const at::Tensor &q = cuda_tensor(v[0], "q");
  const int code = dtype_code(q, "q", {at::kFloat, at::kBFloat16, at::kHalf});
  if (q.dim() != 3) refuse(PyExc_ValueError, "q must be [rows, heads, D]");
  const int64_t rows = q.size(0), hq = q.size(1), d = q.size(2);
  const int dev = q.get_device();
  const Stream on(v[9], dev);
  const at::ScalarType dt = q.scalar_type();
  out_is_dict(v[7]);
  if (d < 16 || d > 256 || d % 16) refuse(PyExc_ValueError, "head dimension must be a multiple of 16 to 256, got " + std::to_string(d));
  const dspark_heads qh = heads(v[0], "q", dt, rows, hq, d, dev);
  dspark_heads kh = {};
  Result qo, ko, st;
  int64_t hkv = 0;
  if (v[1] != Py_None) {
    const at::Tensor &k = cuda_tensor(v[1], "k");
    hkv = k.dim() == 3 ? k.size(1) : -1;
    kh = heads(v[1], "k", dt, rows, hkv, d, dev);
    ko.make(v[7], "k", dt, {rows, hkv, d}, on);
  }
  qo.make(v[7], "q", dt, {rows, hq, d}, on);
  const dspark_rope *rope = rope_for(v[3], d);
  const int32_t *pos = nullptr;
  if (rope || v[2] != Py_None) pos = like<int32_t>(v[2], "positions", at::kInt, {rows}, dev);
  const void *wq = weight(v[4], "q_weight", dt, d, dev), *wk = weight(v[5], "k_weight", dt, d, dev);
  st.status(v[8], on);
  if (rows) {
    const c10::cuda::CUDAGuard here((c10::DeviceIndex)dev);
    const int e = api.norm_rope(&qh, v[1] == Py_None ? nullptr : &kh, rows, (int32_t)hq, (int32_t)hkv, (int32_t)d, code, pos,
                                rope, wq, wk, (float)real(v[6]), qo.data, ko.data, (int32_t *)st.data, on.raw());
    if (e) return PyLong_FromLong(e);
  }
  return answer({{"q", &qo}, {"k", &ko}, {"status", &st}});
}

// cache, device, k, v, row_off, kv_len, page_table, positions, rope, k_weight, q, q_weight, eps, out, status, stream
template <class Cache, class Call>
PyObject *append_to(PyObject *const *v, Call call) {
  const auto *cache = (const Cache *)address(v[0]);
  const int dev = (int)whole(v[1]);
  const Stream on(v[15], dev);
  const at::Tensor &k = cuda_tensor(v[2], "k");
  const int code = dtype_code(k, "k", {at::kFloat, at::kBFloat16, at::kHalf});
  const at::ScalarType dt = k.scalar_type();
  const int64_t rows = k.dim() ? k.size(0) : -1, d = cache->head_dim, hkv = cache->kv_heads;
  out_is_dict(v[13]);
  const dspark_heads kh = heads(v[2], "k", dt, rows, hkv, d, dev), vh = heads(v[3], "v", dt, rows, hkv, d, dev);
  const dspark_ragged where = ragged(v[4], v[5], v[6], rows, dev);
  dspark_heads qh = {};
  Result qo, st;
  int64_t hq = 0;
  if (v[10] != Py_None) {
    const at::Tensor &q = cuda_tensor(v[10], "q");
    hq = q.dim() == 3 ? q.size(1) : -1;
    qh = heads(v[10], "q", dt, rows, hq, d, dev);
    qo.make(v[13], "q", dt, {rows, hq, d}, on);
  }
  const dspark_rope *rope = rope_for(v[8], d);
  const int32_t *pos = maybe<int32_t>(v[7], "positions", at::kInt, {rows}, dev);
  const void *wk = weight(v[9], "k_weight", dt, d, dev), *wq = weight(v[11], "q_weight", dt, d, dev);
  st.status(v[14], on);
  if (rows) {
    const c10::cuda::CUDAGuard here((c10::DeviceIndex)dev);
    const int e = call(&kh, &vh, qo.data ? &qh : nullptr, (int32_t)hq, code, cache, &where, pos, rope, wq, wk,
                             (float)real(v[12]), qo.data, (int32_t *)st.data, on.raw());
    if (e) return PyLong_FromLong(e);
  }
  return answer({{"q", &qo}, {"status", &st}});
}

PyObject *append(PyObject *const *v) { return append_to<dspark_cache>(v, api.append); }
PyObject *append_byte(PyObject *const *v) { return append_to<dspark_byte_cache>(v, api.append_byte); }

// cache, device, row_off, kv_len, page_table, rows, out, status, stream
PyObject *read(PyObject *const *v) {
  const auto *cache = (const dspark_cache *)address(v[0]);
  const int dev = (int)whole(v[1]);
  const Stream on(v[8], dev);
  const int64_t rows = whole(v[5]), d = cache->head_dim, h = cache->kv_heads;
  if (rows < 0) refuse(PyExc_ValueError, "rows must not be negative");
  out_is_dict(v[6]);
  const dspark_ragged where = ragged(v[2], v[3], v[4], rows, dev);
  Result k, ks, vo, vs, st;
  k.make(v[6], "k", at::kFloat8_e4m3fn, {rows, h, d}, on);
  ks.make(v[6], "k_scale", at::kFloat8_e4m3fn, {rows, h, d / 16}, on);
  vo.make(v[6], "v", at::kFloat8_e4m3fn, {rows, h, d}, on);
  vs.make(v[6], "v_scale", at::kFloat8_e4m3fn, {rows, h, d / 16}, on);
  st.status(v[7], on);
  if (rows) {
    const c10::cuda::CUDAGuard here((c10::DeviceIndex)dev);
    const int e = api.read(cache, &where, k.data, ks.data, vo.data, vs.data, (int32_t *)st.data, on.raw());
    if (e) return PyLong_FromLong(e);
  }
  return answer({{"k", &k}, {"k_scale", &ks}, {"v", &vo}, {"v_scale", &vs}, {"status", &st}});
}

// cache, device, row_off, kv_len, page_table, rows, dtype (a dspark_dtype), out, status, stream
PyObject *read_byte(PyObject *const *v) {
  const auto *cache = (const dspark_byte_cache *)address(v[0]);
  const int dev = (int)whole(v[1]), code = (int)whole(v[6]);
  const Stream on(v[9], dev);
  const int64_t rows = whole(v[5]), d = cache->head_dim, h = cache->kv_heads;
  if (rows < 0) refuse(PyExc_ValueError, "rows must not be negative");
  out_is_dict(v[7]);
  const dspark_ragged where = ragged(v[2], v[3], v[4], rows, dev);
  const at::ScalarType dt = code == DSPARK_F32 ? at::kFloat : (code == DSPARK_BF16 ? at::kBFloat16 : at::kHalf);
  Result k, vo, st;
  k.make(v[7], "k", dt, {rows, h, d}, on);
  vo.make(v[7], "v", dt, {rows, h, d}, on);
  st.status(v[8], on);
  if (rows) {
    const c10::cuda::CUDAGuard here((c10::DeviceIndex)dev);
    const int e = api.read_byte(cache, &where, code, k.data, vo.data, (int32_t *)st.data, on.raw());
    if (e) return PyLong_FromLong(e);
  }
  return answer({{"k", &k}, {"v", &vo}, {"status", &st}});
}

// q, cache, device, row_off, kv_len, page_table, scale, causal, window, max_rows, want_lse, out, workspace, status, stream
template <class Cache, class Bytes, class Call>
PyObject *paged_over(PyObject *const *v, Bytes bytes, Call call) {
  const at::Tensor &q = cuda_tensor(v[0], "q");
  const auto *cache = (const Cache *)address(v[1]);
  const int dev = (int)whole(v[2]), code = dtype_code(q, "q", {at::kBFloat16, at::kHalf});
  const Stream on(v[14], dev);
  if (q.dim() != 3) refuse(PyExc_ValueError, "q must be [rows, heads, D]");
  const at::ScalarType dt = q.scalar_type();
  const int64_t rows = q.size(0), hq = q.size(1), d = cache->head_dim, window = whole(v[8]);
  const int64_t max_rows = v[9] == Py_None ? (rows ? rows : 1) : whole(v[9]);
  out_is_dict(v[11]);
  if (hq % cache->kv_heads)
    refuse(PyExc_ValueError, std::to_string(hq) + " query heads are no multiple of " + std::to_string(cache->kv_heads) + " key/value heads");
  if (max_rows < 1 || window < 0) refuse(PyExc_ValueError, "max_rows must be positive and window not negative");
  const dspark_heads qh = heads(v[0], "q", dt, rows, hq, d, dev);
  const dspark_ragged where = ragged(v[3], v[4], v[5], rows, dev);
  Result o, lse, ws, st;
  o.make(v[11], "out", dt, {rows, hq, d}, on);
  if (PyObject_IsTrue(v[10])) lse.make(v[11], "lse", at::kFloat, {rows, hq}, on);
  st.status(v[13], on);
  if (rows) {
    const c10::cuda::CUDAGuard here((c10::DeviceIndex)dev);
    const int64_t need = (int64_t)bytes((int32_t)hq, cache, &where, max_rows);
    const int64_t have = ws.workspace(v[12], need, on);
    const double scale = v[6] == Py_None ? 1.0 / std::sqrt((double)d) : real(v[6]);
    const int e = call(&qh, (int32_t)hq, code, cache, &where, max_rows, (float)scale, PyObject_IsTrue(v[7]), window, o.data,
                            (float *)lse.data, ws.data, (size_t)have, (int32_t *)st.data, on.raw());
    if (e) return PyLong_FromLong(e);
  }
  return answer({{"out", &o}, {"lse", &lse}, {"status", &st}, {"workspace", &ws}});
}

PyObject *paged(PyObject *const *v) { return paged_over<dspark_cache>(v, api.workspace_bytes, api.paged); }
PyObject *paged_byte(PyObject *const *v) {
  return paged_over<dspark_byte_cache>(v, api.paged_byte_workspace_bytes, api.paged_byte);
}

// q, k, v, row_off, kv_off, scale, causal, window, want_lse, out, workspace, status, stream
PyObject *prompt(PyObject *const *v) {
  const at::Tensor &q = cuda_tensor(v[0], "q"), &k = cuda_tensor(v[1], "k"), &off = cuda_tensor(v[3], "row_off");
  const int dev = q.get_device(), code = dtype_code(q, "q", {at::kBFloat16, at::kHalf});
  const Stream on(v[12], dev);
  if (q.dim() != 3 || k.dim() != 3) refuse(PyExc_ValueError, "q and k must be [rows, heads, D]");
  const at::ScalarType dt = q.scalar_type();
  const int64_t rows = q.size(0), hq = q.size(1), d = q.size(2), kv_rows = k.size(0), hkv = k.size(1), window = whole(v[7]);
  out_is_dict(v[9]);
  if (d != 64 && d != 128) refuse(PyExc_ValueError, "heads must have 64 or 128 dimensions, got " + std::to_string(d));
  if (!hkv || !hq || hq % hkv)
    refuse(PyExc_ValueError, std::to_string(hq) + " query heads are no multiple of " + std::to_string(hkv) + " key/value heads");
  if (window < 0) refuse(PyExc_ValueError, "window must not be negative");
  if (off.dim() != 1 || !off.size(0)) refuse(PyExc_ValueError, "row_off must be [B + 1] int32");
  const int64_t B = off.size(0) - 1;
  const dspark_heads qh = heads(v[0], "q", dt, rows, hq, d, dev), kh = heads(v[1], "k", dt, kv_rows, hkv, d, dev),
                     vh = heads(v[2], "v", dt, kv_rows, hkv, d, dev);
  for (const dspark_heads *t : {&kh, &vh}) {
    const std::string name = t == &kh ? "k" : "v";
    const int64_t sr = t->row_stride, sh = t->head_stride;
    if ((kv_rows > 1 && !sr) || (hkv > 1 && !sh)) refuse(PyExc_ValueError, name + " must not be broadcast along rows or heads");
    if (kv_rows > 1 && hkv > 1 && (hkv - 1) * sh + d > sr && sh % sr)
      refuse(PyExc_ValueError, name + " must have its heads inside its rows, or its rows inside its heads with the heads' stride "
                                      "a multiple of the rows'");
  }
  const int32_t *row_off = like<int32_t>(v[3], "row_off", at::kInt, {B + 1}, dev);
  const int32_t *kv_off = v[4] == Py_None ? row_off : like<int32_t>(v[4], "kv_off", at::kInt, {B + 1}, dev);
  if (v[4] == Py_None && kv_rows != rows)
    refuse(PyExc_ValueError, "k has " + std::to_string(kv_rows) + " rows and q " + std::to_string(rows) + ": give kv_off");
  Result o, lse, ws, st;
  o.make(v[9], "out", dt, {rows, hq, d}, on);
  if (PyObject_IsTrue(v[8])) lse.make(v[9], "lse", at::kFloat, {rows, hq}, on);
  st.status(v[11], on);
  if (rows && B) {
    const c10::cuda::CUDAGuard here((c10::DeviceIndex)dev);
    const int64_t have = ws.workspace(
        v[10], (int64_t)api.prompt_workspace_bytes(rows, kv_rows, B, (int32_t)hq, (int32_t)hkv, (int32_t)d), on);
    const double scale = v[5] == Py_None ? 1.0 / std::sqrt((double)d) : real(v[5]);
    const int e = api.prompt(&qh, &kh, &vh, rows, kv_rows, B, (int32_t)hq, (int32_t)hkv, (int32_t)d, code, row_off, kv_off,
                             (float)scale, PyObject_IsTrue(v[6]), window, o.data, (float *)lse.data, ws.data, (size_t)have,
                             (int32_t *)st.data, on.raw());
    if (e) return PyLong_FromLong(e);
  }
  return answer({{"out", &o}, {"lse", &lse}, {"status", &st}, {"workspace", &ws}});
}

// logits, row_off, hist, hist_len, prompt_len, repetition, presence, frequency, draft_tok, bias_tok, bias_val, mask, out, status, stream
PyObject *penalize(PyObject *const *v) {
  const at::Tensor &z = cuda_tensor(v[0], "logits");
  const int code = dtype_code(z, "logits", {at::kFloat, at::kBFloat16});
  if (z.dim() != 2) refuse(PyExc_ValueError, "logits must be [rows, V]");
  const int64_t rows = z.size(0), V = z.size(1);
  const int dev = z.get_device();
  const Stream on(v[14], dev);
  out_is_dict(v[12]);
  const void *in = like(v[0], "logits", z.scalar_type(), {rows, V}, dev);
  const at::Tensor &hist = cuda_tensor(v[2], "hist");
  if (hist.dim() != 2) refuse(PyExc_ValueError, "hist must be [B, cap] int32");
  if ((v[9] == Py_None) != (v[10] == Py_None)) refuse(PyExc_ValueError, "bias_tok and bias_val go together");
  auto width = [](PyObject *o, const char *name) -> int64_t {
    if (o == Py_None) return 0;
    const at::Tensor &t = cuda_tensor(o, name);
    if (t.dim() != 2) refuse(PyExc_ValueError, std::string(name) + " must have two dimensions");
    return t.size(1);
  };
  dspark_penalties p = {};
  const int64_t B = hist.size(0);
  p.hist_cap = hist.size(1), p.draft_cap = width(v[8], "draft_tok"), p.bias_cap = width(v[9], "bias_tok");
  const int32_t *off = like<int32_t>(v[1], "row_off", at::kInt, {B + 1}, dev);
  p.hist = like<int32_t>(v[2], "hist", at::kInt, {B, p.hist_cap}, dev);
  p.hist_len = like<int32_t>(v[3], "hist_len", at::kInt, {B}, dev);
  p.prompt_len = like<int32_t>(v[4], "prompt_len", at::kInt, {B}, dev);
  p.repetition = like<float>(v[5], "repetition", at::kFloat, {B}, dev);
  p.presence = like<float>(v[6], "presence", at::kFloat, {B}, dev);
  p.frequency = like<float>(v[7], "frequency", at::kFloat, {B}, dev);
  p.draft_tok = maybe<int32_t>(v[8], "draft_tok", at::kInt, {B, p.draft_cap}, dev);
  p.bias_tok = maybe<int32_t>(v[9], "bias_tok", at::kInt, {B, p.bias_cap}, dev);
  p.bias_val = maybe<float>(v[10], "bias_val", at::kFloat, {B, p.bias_cap}, dev);
  p.mask = maybe(v[11], "mask", at::kInt, {rows, (V + 31) / 32}, dev);
  Result o, st;
  o.make(v[12], "logits", z.scalar_type(), {rows, V}, on);
  st.status(v[13], on);
  if (rows) {
    const c10::cuda::CUDAGuard here((c10::DeviceIndex)dev);
    const int e = api.penalize(in, code, rows, V, B, off, &p, o.data, (int32_t *)st.data, on.raw());
    if (e) return PyLong_FromLong(e);
  }
  return answer({{"logits", &o}, {"status", &st}});
}

// the addresses of the entry points, in the order of `api`
PyObject *init(PyObject *const *v) {
  void **slots = (void **)&api;
  for (size_t i = 0; i < sizeof(api) / sizeof(void *); ++i) slots[i] = PyLong_AsVoidPtr(v[i]);
  if (PyErr_Occurred()) throw Refused();
  Py_RETURN_NONE;
}

#define ENTRY(f, n) {#f, (PyCFunction)(void (*)(void))entry<f, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(init, 12),   ENTRY(norm_rope, 10), ENTRY(append, 16),
                         ENTRY(read, 9),   ENTRY(paged, 15),     ENTRY(penalize, 15),
                         ENTRY(prompt, 13), ENTRY(append_byte, 16), ENTRY(read_byte, 10),
                         ENTRY(paged_byte, 15), {}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
