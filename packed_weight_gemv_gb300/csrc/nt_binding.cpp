// nt_binding.cpp -- native marshalling for the calls that are made many times per token
// (nt_qk_norm_rope_append, nt_tree_*, nt_logits_adjust, nt_token_counts, nt_page*, nt_beam_select): reads torch tensors' types,
// shapes and strides, refuses what the C ABI cannot see, and calls libnt.so. Their Python forms
// are in nt.py. Through ctypes a call took 15 to 27 us on the host, most of a small call's time.
// Among what is refused are tensors of the host or of another GPU than the current one: their addresses would
// go to the kernel.
//
// The module links to no library of its own: init() gets the addresses of the loaded libnt.so's
// functions and the exception class.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "nt.h"

namespace {

PyObject* g_error = nullptr;  // NtError(status, call, detail)
decltype(&nt_last_error_string) p_last_error = nullptr;
decltype(&nt_qk_norm_rope_append) p_append = nullptr;
decltype(&nt_tree_layout) p_layout = nullptr;
decltype(&nt_tree_attention) p_attention = nullptr;
decltype(&nt_token_counts) p_counts = nullptr;
decltype(&nt_logits_adjust) p_adjust = nullptr;
decltype(&nt_tree_accept) p_accept = nullptr;
decltype(&nt_tree_commit) p_commit = nullptr;
decltype(&nt_page_fork) p_fork = nullptr;
decltype(&nt_page_extend) p_extend = nullptr;
decltype(&nt_page_copy) p_copy = nullptr;
decltype(&nt_page_compact) p_compact = nullptr;
decltype(&nt_paged_attention) p_paged = nullptr;
decltype(&nt_beam_select) p_beam = nullptr;

struct Refusal {
  int status;
  std::string what;
};
struct PythonError {};

using Shape = std::initializer_list<int64_t>;
constexpr auto kF32 = at::kFloat, kF64 = at::kDouble, kBf16 = at::kBFloat16, kI32 = at::kInt;

[[noreturn]] void refuse(const std::string& what) { throw Refusal{NT_ERR_INVALID_ARG, what}; }

std::string shape_text(Shape s) {
  std::string t = "[";
  for (int64_t n : s) t += (t.size() > 1 ? ", " : "") + std::to_string(n);
  return t + "]";
}

// The tensors of the call at hand; where they are is looked at once types and shapes are in order.
struct Given {
  const char* name;
  bool cuda;
  c10::DeviceIndex index;
};
struct Call {
  Given given[24];
  int n = 0;
  void add(const char* name, c10::Device device) {
    if (n == (int)(sizeof(given) / sizeof(given[0]))) refuse("too many tensors");
    given[n++] = Given{name, device.is_cuda(), device.index()};
  }
  void check() const {
    for (int i = 0; i < n; ++i)
      if (!given[i].cuda) refuse(std::string(given[i].name) + " must be a CUDA tensor");
    const c10::DeviceIndex current = c10::cuda::current_device();
    for (int i = 0; i < n; ++i)
      if (given[i].index != current)
        refuse(std::string(given[i].name) + " is on cuda:" + std::to_string(given[i].index) + ", not on the current device, cuda:" +
               std::to_string(current));
  }
};
thread_local Call* t_call = nullptr;  // of guarded() below

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
void* address(const at::Tensor& t, const char* name) {
  t_call->add(name, t.device());
  return t.data_ptr();
}

// Address of a contiguous tensor of this type (and shape, if one is given); None gives NULL.
template <typename T = void>
T* flat(PyObject* o, const char* name, at::ScalarType dtype, const Shape* shape = nullptr) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != dtype || !t.is_contiguous() || (shape && !t.sizes().equals(*shape)))
    refuse(std::string(name) + " must be a contiguous " + c10::toString(dtype) + " tensor" +
           (shape ? " of shape " + shape_text(*shape) : ""));
  return static_cast<T*>(address(t, name));
}
template <typename T = void>
T* flat(PyObject* o, const char* name, at::ScalarType dtype, const Shape& shape) {
  return flat<T>(o, name, dtype, &shape);
}

// Address of a [B, H, D] tensor whose heads are contiguous, and the distance between its tokens.
const void* rows(PyObject* o, const char* name, at::ScalarType dtype, Shape shape, int64_t* stride) {
  const at::Tensor& t = tensor(o, name);
  const int64_t *n = shape.begin();
  if (t.scalar_type() != dtype || !t.sizes().equals(shape) || t.stride(2) != 1 || (n[1] > 1 && t.stride(1) != n[2]))
    refuse(std::string(name) + " must be " + c10::toString(dtype) + " " + shape_text(shape) + " with contiguous heads");
  *stride = n[0] > 1 ? t.stride(0) : n[1] * n[2];
  return address(t, name);
}

// Address and row stride of a [n] tensor for all rows or a [B, n] tensor (stride 0: one row for all).
template <typename T>
T* shared(PyObject* o, const char* name, at::ScalarType dtype, int64_t B, int64_t n, int64_t* stride) {
  *stride = 0;
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  const int64_t d = t.dim();
  if (t.scalar_type() != dtype || d < 1 || d > 2 || t.size(d - 1) != n || (n > 1 && t.stride(d - 1) != 1) ||
      (d == 2 && t.size(0) != 1 && t.size(0) != B))
    refuse(std::string(name) + " must be " + c10::toString(dtype) + " " + shape_text({n}) + " or " + shape_text({B, n}) +
           " with contiguous rows");
  if (d == 2 && t.size(0) > 1) *stride = t.stride(0);
  return static_cast<T*>(address(t, name));
}

int integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  if (v < INT32_MIN || v > INT32_MAX) refuse("an integer argument leaves the int range");
  return (int)v;
}
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return (float)v;
}
int activation(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == kF32) return NT_F32;
  if (t.scalar_type() == kBf16) return NT_BF16;
  refuse(std::string(name) + " must be fp32 or bf16");
}
// None: torch's current stream; an object with cuda_stream, or the stream's address. The last argument to be read.
void* stream_of(PyObject* o) {
  t_call->check();
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  PyObject* a = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
  if (!a) throw PythonError{};
  void* s = PyLong_AsVoidPtr(a);
  Py_DECREF(a);
  if (PyErr_Occurred()) throw PythonError{};
  return s;
}
void* workspace(PyObject* o, size_t* bytes) {
  *bytes = 0;
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, "ws");
  if (!t.is_contiguous()) refuse("ws must be contiguous");
  *bytes = t.nbytes();
  return address(t, "ws");
}
// One number on the device, or None. (A tensor without elements has no address: it would pass for None.)
template <typename T>
T* single(PyObject* o, const char* name) {
  T* p = flat<T>(o, name, kI32);
  if (o != Py_None && tensor(o, name).numel() < 1) refuse(std::string(name) + " must have an element");
  return p;
}
uint32_t* counter(PyObject* o) { return single<uint32_t>(o, "n_bad"); }

template <typename F>
nt_status released(F&& f) {
  nt_status s;
  Py_BEGIN_ALLOW_THREADS s = f();
  Py_END_ALLOW_THREADS return s;
}

// Runs a call; a refusal, here or in the library, becomes an NtError.
template <typename F>
PyObject* guarded(const char* name, Py_ssize_t got, Py_ssize_t want, F&& f) {
  if (!g_error) {
    PyErr_SetString(PyExc_RuntimeError, "init() first");
    return nullptr;
  }
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%s: %zd arguments, not %zd", name, want, got);
    return nullptr;
  }
  int status = NT_OK;
  std::string what;
  Call call;
  t_call = &call;
  try {
    status = f();
    if (status != NT_OK) what = p_last_error();
  } catch (const Refusal& r) {
    status = r.status;
    what = r.what;
  } catch (const PythonError&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  if (status == NT_OK) Py_RETURN_NONE;
  if (PyObject* e = PyObject_CallFunction(g_error, "iss", status, name, what.c_str())) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

// (q, k, v, q_gamma, k_gamma, eps, inv_freq, layout, amplitude, q_out, k_cache, v_cache, pos, pos0,
//  rows, row0, n_bad, stream)
PyObject* append(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded("nt_qk_norm_rope_append", n, 18, [&]() -> nt_status {
    const at::Tensor &q = tensor(x[0], "q"), &k = tensor(x[1], "k"), &kc = tensor(x[10], "k_cache");
    if (q.dim() != 3 || k.dim() != 3 || kc.dim() != 3) refuse("q, k and the caches must have three dimensions");
    const int dtype = activation(q, "q");
    const auto type = q.scalar_type();
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = k.size(1), ts = kc.size(1);
    int64_t qs, ks, vs, rd = 0;
    const void *qp = rows(x[0], "q", type, {B, Hq, D}, &qs), *kp = rows(x[1], "k", type, {B, Hkv, D}, &ks),
               *vp = rows(x[2], "v", type, {B, Hkv, D}, &vs);
    const float *qg = flat<float>(x[3], "q_gamma", kF32, {D}), *kg = flat<float>(x[4], "k_gamma", kF32, {D});
    const double* f = flat<double>(x[6], "inv_freq", kF64);
    if (f) rd = 2 * tensor(x[6], "inv_freq").numel();
    void* out = flat(x[9], "q_out", type, {B, Hq, D});
    auto* kcp = flat<uint16_t>(x[10], "k_cache", kBf16, {Hkv, ts, D});
    auto* vcp = flat<uint16_t>(x[11], "v_cache", kBf16, {Hkv, ts, D});
    const auto *pos = flat<int32_t>(x[12], "pos", kI32, {B}), *rw = flat<int32_t>(x[14], "rows", kI32, {B});
    const float eps = number(x[5]), amp = number(x[8]);
    const int layout = integer(x[7]), pos0 = integer(x[13]), row0 = integer(x[15]);
    uint32_t* bad = counter(x[16]);
    void* st = stream_of(x[17]);
    if (B > INT32_MAX || ts > INT32_MAX || rd > INT32_MAX) refuse("a size leaves the int range");
    return released([&] {
      return p_append(qp, kp, vp, dtype, qs, ks, vs, qg, kg, eps, (int)B, (int)Hq, (int)Hkv, (int)D, f, (int)rd, layout, amp,
                      pos, pos0, rw, row0, out, kcp, vcp, (int)ts, bad, st);
    });
  });
}

// (parent, mask, pos, pos0, n_bad, stream)
PyObject* layout(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded("nt_tree_layout", n, 6, [&]() -> nt_status {
    const at::Tensor &p = tensor(x[0], "parent"), &m = tensor(x[1], "mask");
    const int64_t B = p.numel();
    if (m.dim() != 2 || m.size(0) != B) refuse("mask must be [B, words]");
    const auto* pp = flat<int32_t>(x[0], "parent", kI32);
    auto* mp = flat<uint32_t>(x[1], "mask", kI32);
    auto* pos = flat<int32_t>(x[2], "pos", kI32, {B});
    const int pos0 = integer(x[3]), words = (int)std::min<int64_t>(m.size(1), INT32_MAX);
    uint32_t* bad = counter(x[4]);
    void* st = stream_of(x[5]);
    return released([&] { return p_layout(pp, (int)std::min<int64_t>(B, INT32_MAX), pos0, mp, words, pos, bad, st); });
  });
}

// (q, k_cache, v_cache, prefix, tree_row0, mask, out, ws, stream)
PyObject* attention(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded("nt_tree_attention", n, 9, [&]() -> nt_status {
    const at::Tensor &q = tensor(x[0], "q"), &kc = tensor(x[1], "k_cache"), &m = tensor(x[5], "mask");
    if (q.dim() != 3 || kc.dim() != 3 || m.dim() != 2 || m.size(0) != q.size(0))
      refuse("q [B, Hq, D], caches [Hkv, t_stride, D] and mask [B, words] are needed");
    const int dtype = activation(q, "q");
    const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2), Hkv = kc.size(0), ts = kc.size(1);
    if (B > INT32_MAX || Hq > INT32_MAX || Hkv > INT32_MAX || ts > INT32_MAX || m.size(1) > INT32_MAX)
      refuse("a size leaves the int range");
    const void* qp = flat(x[0], "q", q.scalar_type());
    const auto *kp = flat<uint16_t>(x[1], "k_cache", kBf16, {Hkv, ts, D}), *vp = flat<uint16_t>(x[2], "v_cache", kBf16, {Hkv, ts, D});
    const int prefix = integer(x[3]), row0 = integer(x[4]);
    const auto* mp = flat<uint32_t>(x[5], "mask", kI32);
    void* out = flat(x[6], "out", q.scalar_type(), {B, Hq, D});
    size_t bytes;
    void *ws = workspace(x[7], &bytes), *st = stream_of(x[8]);
    return released([&] {
      return p_attention(qp, dtype, kp, vp, (int)B, (int)Hq, (int)Hkv, (int)D, prefix, row0, (int)ts, mp, (int)m.size(1), out, ws,
                         bytes, st);
    });
  });
}

// (tokens, index, n, counts, n_bad, stream)
PyObject* counts(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded("nt_token_counts", n, 6, [&]() -> nt_status {
    const at::Tensor &t = tensor(x[0], "tokens"), &c = tensor(x[3], "counts");
    const int64_t m = t.numel(), V = c.numel();
    if (m > INT32_MAX || V > INT32_MAX) refuse("a size leaves the int range");
    const auto *tp = flat<int32_t>(x[0], "tokens", kI32), *ip = flat<int32_t>(x[1], "index", kI32);
    if (ip && tensor(x[1], "index").numel() != m) refuse("index must have as many entries as tokens");
    const auto* np = single<const int32_t>(x[2], "n");
    auto* cp = flat<int32_t>(x[3], "counts", kI32);
    uint32_t* bad = counter(x[4]);
    void* st = stream_of(x[5]);
    return released([&] { return p_counts(tp, ip, (int)m, np, (int)V, cp, bad, st); });
  });
}

// (logits, counts, tree_mask, tokens, repetition, frequency, presence, bias, allowed, out, argmax, ws, stream)
PyObject* adjust(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded("nt_logits_adjust", n, 13, [&]() -> nt_status {
    const at::Tensor& l = tensor(x[0], "logits");
    if (l.dim() != 2) refuse("logits must be [B, V]");
    const int64_t B = l.size(0), V = l.size(1);
    if (B > INT32_MAX || V > INT32_MAX) refuse("a size leaves the int range");
    const auto* lp = flat<float>(x[0], "logits", kF32);
    int64_t cs, bs, as;
    const auto* cp = shared<int32_t>(x[1], "counts", kI32, B, V, &cs);
    int words = 0;
    if (x[2] != Py_None) {
      const at::Tensor& m = tensor(x[2], "tree_mask");
      if (m.dim() != 2 || m.size(0) != B) refuse("tree_mask must be [B, words]");
      words = (int)std::min<int64_t>(m.size(1), INT32_MAX);
    }
    const auto* mp = flat<uint32_t>(x[2], "tree_mask", kI32);
    const auto* tp = flat<int32_t>(x[3], "tokens", kI32, {B});
    const float rep = number(x[4]), freq = number(x[5]), pres = number(x[6]);
    const auto* bp = shared<float>(x[7], "bias", kF32, B, V, &bs);
    const auto* ap = shared<uint32_t>(x[8], "allowed", kI32, B, (V + 31) / 32, &as);
    auto* out = flat<float>(x[9], "out", kF32, {B, V});
    auto* am = flat<int32_t>(x[10], "argmax", kI32, {B});
    size_t bytes;
    void *ws = workspace(x[11], &bytes), *st = stream_of(x[12]);
    return released([&] {
      return p_adjust(lp, (int)B, (int)V, cp, cs, mp, words, tp, rep, freq, pres, bp, bs, ap, as, out, am, ws, bytes, st);
    });
  });
}

// (parent, token, argmax, emit, path, n_emit, stream)
PyObject* accept(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded("nt_tree_accept", n, 7, [&]() -> nt_status {
    const int64_t B = tensor(x[0], "parent").numel();
    const auto *p = flat<int32_t>(x[0], "parent", kI32, {B}), *t = flat<int32_t>(x[1], "token", kI32, {B}),
               *a = flat<int32_t>(x[2], "argmax", kI32, {B});
    auto *e = flat<int32_t>(x[3], "emit", kI32, {B}), *w = flat<int32_t>(x[4], "path", kI32, {B}),
         *m = single<int32_t>(x[5], "n_emit");
    void* st = stream_of(x[6]);
    return released([&] { return p_accept(p, t, a, (int)std::min<int64_t>(B, INT32_MAX), e, w, m, st); });
  });
}

// (k_caches, v_caches: addresses of arrays of n_layers pointers, n_layers, Hkv, D, t_stride, path, n_emit, src_row0, dst_row0, stream, the caches' CUDA device or -1)
PyObject* commit(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded("nt_tree_commit", n, 12, [&]() -> nt_status {
    auto* kp = static_cast<uint16_t* const*>(PyLong_AsVoidPtr(x[0]));
    auto* vp = static_cast<uint16_t* const*>(PyLong_AsVoidPtr(x[1]));
    if (PyErr_Occurred()) throw PythonError{};
    const int L = integer(x[2]), Hkv = integer(x[3]), D = integer(x[4]), ts = integer(x[5]);
    const int64_t B = tensor(x[6], "path").numel();
    const auto *p = flat<int32_t>(x[6], "path", kI32), *m = single<int32_t>(x[7], "n_emit");
    const int src = integer(x[8]), dst = integer(x[9]), at = integer(x[11]);
    t_call->add("the caches", at < 0 ? c10::Device(c10::kCPU) : c10::Device(c10::kCUDA, (c10::DeviceIndex)at));
    void* st = stream_of(x[10]);
    return released([&] { return p_commit(kp, vp, L, Hkv, D, ts, p, m, (int)std::min<int64_t>(B, INT32_MAX), src, dst, st); });
  });
}

int64_t fit(int64_t n) {
  if (n > INT32_MAX) refuse("a size leaves the int range");
  return n;
}
// A table [S][width] of pages.
const at::Tensor& pages(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.dim() != 2) refuse(std::string(name) + " must be [S, width]");
  fit(t.size(0));
  fit(t.size(1));
  return t;
}

// (table, length, parent, refs, page, table_out, length_out, n_bad, stream)
PyObject* fork(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded("nt_page_fork", n, 9, [&]() -> nt_status {
    const int64_t S = pages(x[0], "table").size(0), W = tensor(x[0], "table").size(1), So = fit(tensor(x[2], "parent").numel()),
                  P = fit(tensor(x[3], "refs").numel());
    const auto *t = flat<int32_t>(x[0], "table", kI32), *l = flat<int32_t>(x[1], "length", kI32, {S}), *p = flat<int32_t>(x[2], "parent", kI32, {So});
    auto *r = flat<int32_t>(x[3], "refs", kI32, {P}), *to = flat<int32_t>(x[5], "table_out", kI32, {So, W}),
         *lo = flat<int32_t>(x[6], "length_out", kI32, {So});
    const int page = integer(x[4]);
    uint32_t* bad = counter(x[7]);
    void* st = stream_of(x[8]);
    return released([&] { return p_fork(t, l, (int)S, (int)W, p, (int)So, page, r, (int)P, to, lo, bad, st); });
  });
}

// (table, length, refs, q_start, page, rows, pos, pairs, n_bad, stream)
PyObject* extend(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded("nt_page_extend", n, 10, [&]() -> nt_status {
    const int64_t S = pages(x[0], "table").size(0), W = tensor(x[0], "table").size(1), P = fit(tensor(x[2], "refs").numel()),
                  T = fit(tensor(x[5], "rows").numel());
    auto *t = flat<int32_t>(x[0], "table", kI32), *l = flat<int32_t>(x[1], "length", kI32, {S}), *r = flat<int32_t>(x[2], "refs", kI32, {P}),
         *q = flat<int32_t>(x[3], "q_start", kI32, {S + 1}), *rw = flat<int32_t>(x[5], "rows", kI32, {T}), *ps = flat<int32_t>(x[6], "pos", kI32, {T}),
         *pr = flat<int32_t>(x[7], "pairs", kI32, {S, 2});
    const int page = integer(x[4]);
    uint32_t* bad = counter(x[8]);
    void* st = stream_of(x[9]);
    return released([&] { return p_extend(t, l, (int)S, (int)W, q, (int)T, page, r, (int)P, rw, ps, pr, bad, st); });
  });
}

// (k_caches, v_caches: addresses of arrays of n_layers pointers, n_layers, Hkv, D, t_stride, page, pairs, stream, the caches' CUDA device or -1)
PyObject* copy(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded("nt_page_copy", n, 10, [&]() -> nt_status {
    auto* kp = static_cast<uint16_t* const*>(PyLong_AsVoidPtr(x[0]));
    auto* vp = static_cast<uint16_t* const*>(PyLong_AsVoidPtr(x[1]));
    if (PyErr_Occurred()) throw PythonError{};
    const int L = integer(x[2]), Hkv = integer(x[3]), D = integer(x[4]), ts = integer(x[5]), page = integer(x[6]), at = integer(x[9]);
    const int64_t m = pages(x[7], "pairs").size(0);
    const auto* p = flat<int32_t>(x[7], "pairs", kI32, {m, 2});
    t_call->add("the caches", at < 0 ? c10::Device(c10::kCPU) : c10::Device(c10::kCUDA, (c10::DeviceIndex)at));
    void* st = stream_of(x[8]);
    if (m == 0) return NT_OK;  // of a pool of one page
    return released([&] { return p_copy(kp, vp, L, Hkv, D, ts, page, p, (int)m, st); });
  });
}

// (refs, table, length, page, pairs, n_used, n_bad, ws, stream)
PyObject* compact(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded("nt_page_compact", n, 9, [&]() -> nt_status {
    const int64_t P = fit(tensor(x[0], "refs").numel()), S = pages(x[1], "table").size(0), W = tensor(x[1], "table").size(1),
                  m = pages(x[4], "pairs").size(0);
    auto *r = flat<int32_t>(x[0], "refs", kI32, {P}), *t = flat<int32_t>(x[1], "table", kI32), *l = flat<int32_t>(x[2], "length", kI32, {S}),
         *pr = flat<int32_t>(x[4], "pairs", kI32, {m, 2});
    const int page = integer(x[3]);
    auto* used = single<int32_t>(x[5], "n_used");
    uint32_t* bad = counter(x[6]);
    size_t bytes;
    void *ws = workspace(x[7], &bytes), *st = stream_of(x[8]);
    return released([&] { return p_compact(r, (int)P, t, l, (int)S, (int)W, page, pr, (int)m, used, bad, ws, bytes, st); });
  });
}

// (q, k_pool, v_pool, page, table, q_start, length, out, ws, max_new, window, cap, slopes, n_bad, stream)
PyObject* paged(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded("nt_paged_attention", n, 15, [&]() -> nt_status {
    const at::Tensor &q = tensor(x[0], "q"), &kc = tensor(x[1], "k_pool");
    if (q.dim() != 3 || kc.dim() != 3) refuse("q [T, Hq, D] and pools [Hkv, t_stride, D] are needed");
    const int dtype = activation(q, "q");
    const int64_t T = fit(q.size(0)), Hq = fit(q.size(1)), D = fit(q.size(2)), Hkv = fit(kc.size(0)), ts = fit(kc.size(1));
    const int64_t S = pages(x[4], "table").size(0), W = tensor(x[4], "table").size(1);
    int64_t qs;
    const void* qp = rows(x[0], "q", q.scalar_type(), {T, Hq, D}, &qs);
    const auto *kp = flat<uint16_t>(x[1], "k_pool", kBf16, {Hkv, ts, D}), *vp = flat<uint16_t>(x[2], "v_pool", kBf16, {Hkv, ts, D});
    const auto *t = flat<int32_t>(x[4], "table", kI32), *qst = flat<int32_t>(x[5], "q_start", kI32, {S + 1}),
               *l = flat<int32_t>(x[6], "length", kI32, {S});
    void* out = flat(x[7], "out", q.scalar_type(), {T, Hq, D});
    size_t bytes;
    void* ws = workspace(x[8], &bytes);
    const int page = integer(x[3]), most = integer(x[9]), window = integer(x[10]);
    const float cap = number(x[11]);
    const auto* sl = flat<float>(x[12], "slopes", kF32, {Hq});
    uint32_t* bad = counter(x[13]);
    void* st = stream_of(x[14]);
    return released([&] {
      return p_paged(qp, dtype, qs, kp, vp, (int)T, (int)S, (int)Hq, (int)Hkv, (int)D, page, (int)ts, t, (int)W, qst, l, most, window, cap,
                     sl, out, bad, ws, bytes, st);
    });
  });
}

// (logits, scores, beams, parent, token, score, done, done_out, eos, lengths, alpha, ws, stream)
PyObject* beam(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded("nt_beam_select", n, 13, [&]() -> nt_status {
    const at::Tensor& lg = tensor(x[0], "logits");
    if (lg.dim() != 2) refuse("logits must be [N, V]");
    const int64_t N = fit(lg.size(0)), V = fit(lg.size(1)), M = fit(tensor(x[3], "parent").numel());
    const int W = integer(x[2]);
    if (W < 1 || N % W != 0 || N < W || M % (N / W) != 0) refuse("need rows of logits a multiple of beams, and as many results for each group");
    const auto *lp = flat<float>(x[0], "logits", kF32), *sp = flat<float>(x[1], "scores", kF32, {N});
    auto *p = flat<int32_t>(x[3], "parent", kI32), *t = flat<int32_t>(x[4], "token", kI32);
    auto* sc = flat<float>(x[5], "score", kF32);
    if (tensor(x[4], "token").numel() != M || tensor(x[5], "score").numel() != M) refuse("parent, token and score must be alike");
    const auto* d = flat<int32_t>(x[6], "done", kI32, {N});
    auto* dn = flat<int32_t>(x[7], "done_out", kI32);
    if (dn && tensor(x[7], "done_out").numel() != M) refuse("done_out must be like parent");
    const int eos = integer(x[8]);
    const auto* l = flat<int32_t>(x[9], "lengths", kI32, {N});
    const double alpha = PyFloat_AsDouble(x[10]);
    if (alpha == -1.0 && PyErr_Occurred()) throw PythonError{};
    size_t bytes;
    void *ws = workspace(x[11], &bytes), *st = stream_of(x[12]);
    return released([&] {
      return p_beam(lp, sp, (int)N, W, (int)V, (int)(M / (N / W)), d, eos, l, alpha, p, t, sc, dn, ws, bytes, st);
    });
  });
}

// (NtError, last_error, append, layout, attention, counts, adjust, accept, commit, fork, extend, copy, compact, paged, beam): addresses of
// the library's functions
PyObject* init(PyObject*, PyObject* const* x, Py_ssize_t n) {
  constexpr int kArgs = 15;
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "init: %d arguments", kArgs);
    return nullptr;
  }
  void* p[kArgs] = {};
  for (int i = 1; i < kArgs; ++i) p[i] = PyLong_AsVoidPtr(x[i]);
  if (PyErr_Occurred()) return nullptr;
  Py_INCREF(x[0]);
  Py_XDECREF(g_error);
  g_error = x[0];
  int i = 0;
  auto next = [&](auto& f) { f = reinterpret_cast<std::decay_t<decltype(f)>>(p[++i]); };
  next(p_last_error);
  next(p_append);
  next(p_layout);
  next(p_attention);
  next(p_counts);
  next(p_adjust);
  next(p_accept);
  next(p_commit);
  next(p_fork);
  next(p_extend);
  next(p_copy);
  next(p_compact);
  next(p_paged);
  next(p_beam);
  Py_RETURN_NONE;
}

#define NT_METHOD(name) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr }
PyMethodDef g_methods[] = {NT_METHOD(init),   NT_METHOD(append), NT_METHOD(layout), NT_METHOD(attention), NT_METHOD(counts),
                           NT_METHOD(adjust), NT_METHOD(accept), NT_METHOD(commit), NT_METHOD(fork),   NT_METHOD(extend),
                           NT_METHOD(copy),   NT_METHOD(compact), NT_METHOD(paged), NT_METHOD(beam), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ntbind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ntbind(void) { return PyModule_Create(&g_module); }
