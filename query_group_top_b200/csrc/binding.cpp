// The compiled half of the Python binding of the serving step over a paged cache:
// the checks of qk_rope, paged_append, paged_attention and sparse_attention_paged,
// their outputs and workspaces, and the call into the C ABI (pivot.h).
//
// These calls take 3 to 5 us on the device in a decode step, so a step that is
// not captured is bound by the host.  Here a call takes the host 4 to 6 us (the
// attention 9), of which the launch is 3; the same checks in Python, with the C
// functions called through ctypes, took 12 to 14 (19).
//
// The C functions are those of the library that Python loaded (bind), so there is
// one copy of it, its status words and its traces.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <stdexcept>
#include <string>

#include "pivot.h"

namespace {

struct Lib {
  decltype(&pivot_last_error) last_error;
  decltype(&pivot_qk_rope) qk_rope;
  decltype(&pivot_paged_append) paged_append;
  decltype(&pivot_paged_attention_workspace_size) attention_workspace;
  decltype(&pivot_paged_attention) paged_attention;
  decltype(&pivot_sparse_attention_paged) sparse_paged;
} lib;
PyObject* pivot_error;   // the exception

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};

[[noreturn]] __attribute__((format(printf, 1, 2))) void refuse(const char* fmt, ...) {
  char text[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  throw Refused(text);
}

void check(int rc) {
  if (rc != 0) refuse("pivot error %d: %s", rc, lib.last_error());
}

// Releases the interpreter's lock while a call launches (a full queue blocks).
struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};

std::string name_of(at::ScalarType t) { return c10::toString(t); }

std::string shape_of(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

// ------------------------------------------------------------------ arguments
using Arg = const at::Tensor*;   // null: None

Arg optional(const char* name, PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
  return &THPVariable_Unpack(o);
}
const at::Tensor& required(const char* name, PyObject* o) {
  Arg t = optional(name, o);
  if (!t) refuse("%s must be a tensor", name);
  return *t;
}
double number(const char* name, PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse("%s must be a number", name);
  }
  return x;
}
long long whole(const char* name, PyObject* o) {
  PyObject* n = PyNumber_Long(o);
  const long long x = n ? PyLong_AsLongLong(n) : -1;
  Py_XDECREF(n);
  if (x == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse("%s must be a whole number in range", name);
  }
  return x;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// New tokens' rows x: [T, heads, d], or [B, g, heads, d].
struct Tokens {
  bool batched;
  int64_t n0, n1;   // T and 1, or B and g
  int64_t heads;
  int d, dev;
  int64_t count() const { return n0 * n1; }
};

Tokens tokens(const char* name, const at::Tensor& x) {
  if (!x.is_cuda()) refuse("%s must be a CUDA tensor", name);
  const auto s = x.sizes();
  if (s.size() != 3 && s.size() != 4) refuse("%s must be [T, heads, d] or [B, g, heads, d]", name);
  const bool batched = s.size() == 4;
  const int64_t d = s.back();
  if (d != 64 && d != 128) refuse("head_dim must be 64 or 128 (got %lld)", static_cast<long long>(d));
  Tokens t{batched, s[0], batched ? s[1] : 1, s[s.size() - 2], static_cast<int>(d), x.get_device()};
  if (t.heads < 1 || t.heads > INT_MAX || t.n0 > INT_MAX || t.n1 > INT_MAX || t.count() > INT_MAX)
    refuse("%s has no heads, or more tokens than fit", name);
  return t;
}

int dtype_of(const char* names, at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return PIVOT_BF16;
    case at::kHalf: return PIVOT_FP16;
    case at::kFloat: return PIVOT_FP32;
    default: refuse("%s must be bfloat16, float16 or float32 (got %s)", names, name_of(t).c_str());
  }
}

// x's rows for the C call: tokens and channels as `like`, any number of heads; a
// strided view (a slice of a fused projection) as it is.
pivot_heads_t heads(const char* name, const at::Tensor& x, Arg weight, const Tokens& like, at::ScalarType dtype) {
  const auto s = x.sizes();
  const size_t nd = like.batched ? 4 : 3;
  if (s.size() != nd || s[0] != like.n0 || (like.batched && s[1] != like.n1) || s.back() != like.d)
    refuse("%s must have the call's tokens and heads of %d channels (got %s)", name, like.d, shape_of(s).c_str());
  if (x.scalar_type() != dtype || !x.is_cuda() || x.get_device() != like.dev)
    refuse("%s must be %s on cuda:%d, as the call's other tensors (is %s on %s)", name, name_of(dtype).c_str(), like.dev,
           name_of(x.scalar_type()).c_str(), x.device().str().c_str());
  const int64_t H = s[nd - 2];
  if (H < 1 || H > INT_MAX) refuse("%s has no heads", name);
  int64_t ts = H * like.d, hs = like.d;
  if (!x.is_contiguous()) {
    const auto st = x.strides();
    if (st.back() != 1) refuse("%s's channels must be adjacent", name);
    ts = st[nd - 3];
    if (like.batched) {
      if (like.n1 == 1)
        ts = st[0];
      else if (like.n0 > 1 && st[0] != like.n1 * ts)
        refuse("%s's tokens must be evenly spaced (strides %s)", name, shape_of(st).c_str());
    }
    if (like.count() <= 1) ts = 0;
    hs = H > 1 ? st[nd - 2] : 0;
    const int64_t step = 16 / static_cast<int64_t>(x.element_size());
    if (ts % step || hs % step) refuse("%s's rows must start on 16-byte boundaries", name);
  }
  if (!aligned16(x.const_data_ptr())) refuse("%s's rows must start on 16-byte boundaries", name);
  pivot_heads_t h{x.const_data_ptr(), nullptr, ts, hs, static_cast<int>(H)};
  if (weight) {
    h.weight = weight->const_data_ptr();
    if (weight->scalar_type() != dtype || weight->dim() != 1 || weight->size(0) != like.d || !weight->is_cuda() ||
        weight->get_device() != like.dev || !aligned16(h.weight) || !weight->is_contiguous())
      refuse("%s_weight must be a contiguous, 16-byte aligned %s tensor of %d channels on cuda:%d", name,
             name_of(dtype).c_str(), like.d, like.dev);
  }
  return h;
}

pivot_rope_t rotation(Arg freqs, PyObject* layout, PyObject* amplitude, PyObject* eps, const Tokens& t) {
  pivot_rope_t r{nullptr, 1.0, number("eps", eps), 0, PIVOT_ROPE_HALF};
  if (!PyUnicode_Check(layout)) refuse("layout must be \"half\" or \"interleaved\"");
  if (PyUnicode_CompareWithASCIIString(layout, "interleaved") == 0)
    r.layout = PIVOT_ROPE_INTERLEAVED;
  else if (PyUnicode_CompareWithASCIIString(layout, "half") != 0)
    refuse("layout must be \"half\" or \"interleaved\"");
  const double amp = number("amplitude", amplitude);
  if (!(r.eps >= 0.0) || !std::isfinite(r.eps) || !std::isfinite(amp))
    refuse("eps must be >= 0, and eps and amplitude finite");
  if (!freqs) return r;
  if (freqs->scalar_type() != at::kDouble || freqs->dim() != 1 || !freqs->is_cuda() || freqs->get_device() != t.dev ||
      !freqs->is_contiguous())
    refuse("freqs must be a contiguous float64 vector of rot_dim / 2 frequencies on cuda:%d", t.dev);
  const int64_t rot = 2 * freqs->numel();
  if (rot < 16 || rot > t.d || rot % 16)
    refuse("rot_dim must be a multiple of 16 in [16, d] (got %lld)", static_cast<long long>(rot));
  r.freqs = static_cast<const double*>(freqs->const_data_ptr());
  r.amplitude = amp;
  r.rot_dim = static_cast<int>(rot);
  return r;
}

const int32_t* int32(const char* name, const at::Tensor& t, int dev, at::IntArrayRef shape) {
  if (t.scalar_type() != at::kInt || t.sizes() != shape || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
    refuse("%s must be a contiguous int32 tensor of shape %s on cuda:%d", name, shape_of(shape).c_str(), dev);
  return static_cast<const int32_t*>(t.const_data_ptr());
}

// The caller's output, checked, or a new contiguous tensor.  `ref`: a new
// reference to what Python gets back.
struct Output {
  void* data = nullptr;
  PyObject* ref = nullptr;
  at::Tensor t;
  Output() = default;
  Output(const Output&) = delete;
  Output& operator=(const Output&) = delete;
  ~Output() { Py_XDECREF(ref); }

  void make(const char* name, PyObject* out, at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor& like) {
    if (out == Py_None) {
      t = at::empty(shape, like.options().dtype(dtype));
      ref = THPVariable_Wrap(t);
      if (!ref) throw python_error();
    } else {
      t = required(name, out);
      if (t.sizes() != shape || t.scalar_type() != dtype || !t.is_contiguous() || t.device() != like.device())
        refuse("%s must be a contiguous %s tensor of shape %s on %s", name, name_of(dtype).c_str(), shape_of(shape).c_str(),
               like.device().str().c_str());
      Py_INCREF(out);
      ref = out;
    }
    data = t.data_ptr();
  }
  PyObject* release() {
    PyObject* r = ref ? ref : Py_NewRef(Py_None);
    ref = nullptr;
    return r;
  }
};

struct Pages {
  int n, size, heads;
};

Pages pages(const at::Tensor& k, Arg v, const Tokens& t) {
  const auto s = k.sizes();
  if (k.scalar_type() != at::kBFloat16 || s.size() != 4 || s[3] != t.d || !k.is_cuda() || k.get_device() != t.dev ||
      !k.is_contiguous())
    refuse("kpages must be contiguous bfloat16 [num_pages, page_size, heads, %d] on cuda:%d", t.d, t.dev);
  if (v && (v->scalar_type() != at::kBFloat16 || v->sizes() != s || !v->is_cuda() || v->get_device() != t.dev ||
            !v->is_contiguous()))
    refuse("vpages must be contiguous bfloat16 %s on cuda:%d, as kpages", shape_of(s).c_str(), t.dev);
  if (s[1] < 1 || (s[1] & (s[1] - 1))) refuse("page_size must be a power of two (got %lld)", static_cast<long long>(s[1]));
  if (s[0] < 1 || s[2] < 1) refuse("the cache has no pages or no heads");
  if (s[0] > INT_MAX || s[1] > INT_MAX || s[2] > INT_MAX) refuse("the cache has too many pages or heads");
  return Pages{static_cast<int>(s[0]), static_cast<int>(s[1]), static_cast<int>(s[2])};
}

// A call's new tokens by sequence.
struct Sequences {
  int T, B, g, max_pages;
  const int32_t *cu, *seqlens, *table;
};

Sequences sequences(const Tokens& t, const char* cu_name, Arg cu, const at::Tensor& seqlens, const at::Tensor& table) {
  if (table.dim() != 2 || table.size(1) < 1 || table.size(0) > INT_MAX - 1 || table.size(1) > INT_MAX)
    refuse("block_table must be an int32 tensor [B, max_pages]");
  const int64_t B = table.size(0);
  Sequences s{static_cast<int>(t.count()), static_cast<int>(B), 0, static_cast<int>(table.size(1)), nullptr, nullptr, nullptr};
  if (!cu) {
    if (!t.batched || t.n0 != B)
      refuse("without %s, the new tokens are [B, g, heads, d] with block_table's B = %lld", cu_name, static_cast<long long>(B));
    s.g = static_cast<int>(t.n1);
  } else {
    if (t.batched) refuse("with %s, the new tokens are [T, heads, d]", cu_name);
    s.cu = int32(cu_name, *cu, t.dev, {B + 1});
  }
  s.seqlens = int32("seqlens", seqlens, t.dev, {B});
  s.table = int32("block_table", table, t.dev, table.sizes());
  return s;
}

// ------------------------------------------------------------------ the calls
PyObject* qk_rope(PyObject* const* a) {
  PyObject *const q_ = a[0], *const k_ = a[1];
  Arg q = optional("q", q_), k = optional("k", k_), freqs = optional("freqs", a[3]);
  Arg wq = optional("q_weight", a[6]), wk = optional("k_weight", a[7]);
  if (!q && !k) refuse("qk_rope needs q or k");
  const at::Tensor& x = q ? *q : *k;
  const Tokens t = tokens(q ? "q" : "k", x);
  const at::ScalarType type = x.scalar_type();
  const int dtype = dtype_of("q and k", type);
  if ((!q && wq) || (!k && wk)) refuse("a norm weight without its heads");
  pivot_heads_t hq{}, hk{};
  if (q) hq = heads("q", *q, wq, t, type);
  if (k) hk = heads("k", *k, wk, t, type);
  const pivot_rope_t rope = rotation(freqs, a[4], a[5], a[8], t);
  const int32_t* pos = nullptr;
  if (freqs) {
    Arg p = optional("positions", a[2]);
    if (!p || p->numel() != t.count()) refuse("positions must hold one int32 position a token");
    pos = int32("positions", *p, t.dev, p->sizes());
  }
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(t.dev));
  Output oq, ok;
  if (q) oq.make("out_q", a[9], q->sizes(), at::kBFloat16, *q);
  if (k) ok.make("out_k", a[10], k->sizes(), at::kBFloat16, *k);
  if (t.count()) {
    const cudaStream_t st = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(t.dev)).stream();
    int rc;
    {
      NoGil free;
      rc = lib.qk_rope(q ? &hq : nullptr, k ? &hk : nullptr, dtype, pos, &rope, static_cast<int>(t.count()), t.d, oq.data,
                       ok.data, st);
    }
    check(rc);
  }
  PyObject* pair = PyTuple_New(2);
  if (!pair) throw python_error();
  PyTuple_SET_ITEM(pair, 0, oq.release());
  PyTuple_SET_ITEM(pair, 1, ok.release());
  return pair;
}

PyObject* paged_append(PyObject* const* a) {
  const at::Tensor& k = required("k", a[0]);
  Arg v = optional("v", a[1]);
  const at::Tensor& kpages = required("kpages", a[2]);
  Arg vpages = optional("vpages", a[3]);
  const at::Tensor &table = required("block_table", a[4]), &seqlens = required("seqlens", a[5]);
  Arg cu = optional("cu_new", a[6]), freqs = optional("freqs", a[7]), wk = optional("k_weight", a[10]);
  Arg q = optional("q", a[11]), wq = optional("q_weight", a[12]);
  const Tokens t = tokens("k", k);
  const at::ScalarType type = k.scalar_type();
  const int dtype = dtype_of("k, v and q", type);
  if (!v != !vpages) refuse("v and vpages go together");
  if (!q && (a[14] != Py_None || wq)) refuse("out_q and q_weight need q");
  pivot_heads_t hv{}, hq{};
  const pivot_heads_t hk = heads("k", k, wk, t, type);
  if (v) hv = heads("v", *v, nullptr, t, type);
  if (q) hq = heads("q", *q, wq, t, type);
  const Pages pg = pages(kpages, vpages, t);
  if (pg.heads != hk.heads || (v && hv.heads != hk.heads)) refuse("k and v must have the cache's %d heads", pg.heads);
  const pivot_rope_t rope = rotation(freqs, a[8], a[9], a[13], t);
  const Sequences s = sequences(t, "cu_new", cu, seqlens, table);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(t.dev));
  Output oq;
  if (q) oq.make("out_q", a[14], q->sizes(), at::kBFloat16, *q);
  const bool fresh = q && a[14] == Py_None;   // tokens that are left out have zeros in it, not what the memory held
  if (fresh && !s.B) oq.t.zero_();
  if (s.T && s.B) {
    const cudaStream_t st = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(t.dev)).stream();
    void *const kp = kpages.data_ptr(), *const vp = vpages ? vpages->data_ptr() : nullptr;
    int rc;
    {
      NoGil free;
      rc = lib.paged_append(&hk, v ? &hv : nullptr, q ? &hq : nullptr, fresh ? dtype | PIVOT_CLEAR_LEFT_OUT : dtype, &rope, s.table, s.seqlens, s.cu, s.T, s.B, t.d,
                            s.g, pg.n, pg.size, s.max_pages, kp, vp, oq.data, st);
    }
    check(rc);
  }
  return oq.release();
}

// The queries of an attention call.
const at::Tensor& queries(PyObject* o) {
  const at::Tensor& q = required("q", o);
  if (!q.is_cuda()) refuse("q must be a CUDA tensor");
  if (q.scalar_type() != at::kBFloat16 || !q.is_contiguous()) refuse("q must be a contiguous bfloat16 tensor");
  return q;
}

PyObject* paged_attention(PyObject* const* a) {
  const at::Tensor &q = queries(a[0]), &kpages = required("kpages", a[1]), &vpages = required("vpages", a[2]);
  const at::Tensor &table = required("block_table", a[3]), &seqlens = required("seqlens", a[4]);
  const long long max_seqlen = whole("max_seqlen", a[5]);
  Arg cu = optional("cu_q", a[6]), lse = optional("out_lse", a[10]);
  const Tokens t = tokens("q", q);
  const Pages pg = pages(kpages, &vpages, t);
  if (t.heads % pg.heads)
    refuse("q's heads must be a multiple of the cache's %d (got %lld)", pg.heads, static_cast<long long>(t.heads));
  Sequences s = sequences(t, "cu_q", cu, seqlens, table);
  if (max_seqlen < 1 || max_seqlen >= (1ll << 30)) refuse("max_seqlen must be in [1, 2^30) (got %lld)", max_seqlen);
  if (cu && a[11] != Py_None) {
    const long long most = whole("max_q", a[11]);
    if (most < 1 || most > INT_MAX) refuse("max_q must be >= 1");
    s.g = static_cast<int>(most);
  }
  const int self = PyObject_IsTrue(a[8]);
  if (self < 0) throw python_error();
  const pivot_attend_t opt{a[7] == Py_None ? 1.0 / std::sqrt(static_cast<double>(t.d)) : number("scale", a[7]), self};
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(t.dev));
  Output out, ol;
  out.make("out", a[9], q.sizes(), at::kBFloat16, q);
  if (lse) ol.make("out_lse", a[10], q.sizes().slice(0, q.dim() - 1), at::kFloat, q);
  if (s.T && s.B) {
    const int Hq = static_cast<int>(t.heads), most = static_cast<int>(max_seqlen);
    const size_t bytes = lib.attention_workspace(s.T, s.B, Hq, pg.heads, t.d, most);
    at::Tensor ws;
    if (bytes) ws = at::empty({static_cast<int64_t>(bytes)}, q.options().dtype(at::kByte));
    const cudaStream_t st = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(t.dev)).stream();
    void* const pws = bytes ? ws.data_ptr() : nullptr;
    const void *const pq = q.const_data_ptr(), *const kp = kpages.const_data_ptr(), *const vp = vpages.const_data_ptr();
    int rc;
    {
      NoGil free;
      rc = lib.paged_attention(pq, kp, vp, s.table, s.seqlens, s.cu, &opt, s.T, s.B, Hq, pg.heads, t.d, s.g, pg.n, pg.size,
                               s.max_pages, most, out.data, static_cast<float*>(ol.data), pws, bytes, st);
    }
    check(rc);
  }
  return out.release();
}

PyObject* sparse_attention_paged(PyObject* const* a) {
  const at::Tensor &q = queries(a[0]), &kpages = required("kpages", a[1]), &vpages = required("vpages", a[2]);
  const at::Tensor &table = required("block_table", a[3]), &seqlens = required("seqlens", a[4]), &idx = required("idx", a[5]);
  const Tokens t = tokens("q", q);
  const Pages pg = pages(kpages, &vpages, t);
  if (pg.heads != t.heads) refuse("q must have the cache's %d heads (got %lld)", pg.heads, static_cast<long long>(t.heads));
  const Sequences s = sequences(t, "cu_q", nullptr, seqlens, table);
  if (idx.dim() != 4 || idx.size(3) > INT_MAX) refuse("idx must be an int32 tensor [B, g, H, top_k]");
  const int top_k = static_cast<int>(idx.size(3));
  const int32_t* rows = int32("idx", idx, t.dev, {t.n0, t.n1, t.heads, idx.size(3)});
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(t.dev));
  Output out;
  out.make("out", a[6], q.sizes(), at::kFloat, q);
  if (s.T && top_k) {
    const cudaStream_t st = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(t.dev)).stream();
    const void *const pq = q.const_data_ptr(), *const kp = kpages.const_data_ptr(), *const vp = vpages.const_data_ptr();
    int rc;
    {
      NoGil free;
      rc = lib.sparse_paged(pq, kp, vp, s.table, s.seqlens, rows, s.B, pg.heads, t.d, s.g, pg.n, pg.size, s.max_pages, top_k,
                            static_cast<float*>(out.data), st);
    }
    check(rc);
  } else {
    out.t.zero_();
  }
  return out.release();
}

// ------------------------------------------------------------------ the module
template <PyObject* (*Call)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "takes %d arguments (got %zd)", N, n);
    return nullptr;
  }
  try {
    return Call(args);
  } catch (const Refused& e) {
    PyErr_SetString(pivot_error ? pivot_error : PyExc_RuntimeError, e.what());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// bind(exception, addresses of the C functions in Lib's order)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind takes an exception and six addresses");
    return nullptr;
  }
  void* f[6];
  for (int i = 0; i < 6; ++i) {
    f[i] = PyLong_AsVoidPtr(args[i + 1]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  lib = Lib{reinterpret_cast<decltype(lib.last_error)>(f[0]),      reinterpret_cast<decltype(lib.qk_rope)>(f[1]),
            reinterpret_cast<decltype(lib.paged_append)>(f[2]),    reinterpret_cast<decltype(lib.attention_workspace)>(f[3]),
            reinterpret_cast<decltype(lib.paged_attention)>(f[4]), reinterpret_cast<decltype(lib.sparse_paged)>(f[5])};
  Py_INCREF(args[0]);
  Py_XSETREF(pivot_error, args[0]);
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {
    {"bind", FAST(bind), METH_FASTCALL, nullptr},
    {"qk_rope", FAST((entry<qk_rope, 11>)), METH_FASTCALL, nullptr},
    {"paged_append", FAST((entry<paged_append, 15>)), METH_FASTCALL, nullptr},
    {"paged_attention", FAST((entry<paged_attention, 12>)), METH_FASTCALL, nullptr},
    {"sparse_attention_paged", FAST((entry<sparse_attention_paged, 7>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_step", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__step() {
  PyObject* m = PyModule_Create(&module);
  // the torch whose C++ classes this calls: another version may lay them out otherwise
  if (m && PyModule_AddStringConstant(m, "built_for", PIVOT_TORCH) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
