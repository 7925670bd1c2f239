// Python entry points of the attention side: checks of tensors and the C
// ABI's calls (include/pi_attn.h), for attention.py.
//
// A decode step's calls take 3 to 10 microseconds on the GPU.  The same checks
// in Python, with the arguments' way through ctypes, took as long again, so the
// GPU waited for the host; here they take a few tenths of a microsecond beside the launch.
// Every function returns the call's pi_status; a tensor that the C ABI could not
// read raises TypeError or ValueError, and nothing is launched.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPStream.h>
#include <algorithm>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pi.h"

namespace {

// libpi's functions, from the library that the package has loaded (use_library).
struct Library {
  decltype(&::pi_qk_rope) qk_rope;
  decltype(&::pi_kv_append) kv_append;
  decltype(&::pi_kv_read) kv_read;
  decltype(&::pi_attend) attend;
  decltype(&::pi_kv_evict) kv_evict;
} lib;

struct BadArgument {};     // the Python error is set

void fail(PyObject* type, const char* format, const char* name, long long n = 0) {
  PyErr_Format(type, format, name, n);
  throw BadArgument();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

void on_device(const at::Tensor& t, const char* name, int dev) {
  if (!t.is_cuda()) fail(PyExc_ValueError, "%s must live in GPU memory", name);
  if (t.get_device() != dev) fail(PyExc_ValueError, "%s must be on the same device as the rest", name);
}

// Token rows [n_tok][heads][d] of type dt on device dev.
struct Rows {
  void* p;
  int64_t ts, hs;
  int n_tok, heads;
};
Rows rows(PyObject* o, const char* name, int64_t heads, int64_t d, at::ScalarType dt, int dev) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != dt)
    fail(PyExc_TypeError, dt == at::kHalf ? "%s must be torch.float16" : "%s must be torch.float32", name);
  on_device(t, name, dev);
  if (t.dim() != 3 || t.size(2) != d) fail(PyExc_ValueError, "%s must be [n_tok, heads, %lld]", name, d);
  if (heads >= 0 && t.size(1) != heads) fail(PyExc_ValueError, "%s must have %lld heads", name, heads);
  if (t.stride(2) != 1) fail(PyExc_ValueError, "%s: the elements of a head must be contiguous", name);
  if (t.size(0) > 0x7fffffff || t.size(1) > 0x7fffffff) fail(PyExc_ValueError, "%s is too large", name);
  return Rows{t.data_ptr(), t.stride(0), t.stride(1), (int)t.size(0), (int)t.size(1)};
}

void same_tokens(const Rows& a, const Rows& b, const char* names) {
  if (a.n_tok != b.n_tok) fail(PyExc_ValueError, "%s must have the same tokens", names);
}

int32_t* int32s(PyObject* o, const char* name, int64_t n, int dev) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    fail(PyExc_ValueError, "%s must be contiguous int32 [%lld]", name, n);
  on_device(t, name, dev);
  return static_cast<int32_t*>(t.data_ptr());
}

int64_t integer(PyObject* o, const char* name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw BadArgument();
  if (v < -0x80000000ll || v > 0x7fffffffll) fail(PyExc_ValueError, "%s is out of range", name);
  return v;
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw BadArgument();
  return v;
}

template <typename D>
const D* descriptor(PyObject* o) {
  const void* p = PyLong_AsVoidPtr(o);
  if (!p) fail(PyExc_ValueError, "%s is missing", "the descriptor");
  return static_cast<const D*>(p);
}

const pi_kv_cache* cache_of(PyObject* o) {
  const auto* c = descriptor<pi_kv_cache>(o);
  if (c->n_seqs < 1) fail(PyExc_ValueError, "%s must have sequences", "the cache");      // (rows are divided by them)
  return c;
}

// None: the device's current stream; else a handle.
void* stream_of(PyObject* o, int dev) {
  if (o == Py_None) return c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream();
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw BadArgument();
  return p;
}

// The call itself, with device dev current.  Other Python threads run while it
// is queued (a full queue makes it wait).
template <typename F>
int64_t queue(int dev, F f) {
  const c10::DeviceGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
  pi_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = f();
  Py_END_ALLOW_THREADS;
  return st;
}

at::ScalarType scalar_of(int dtype) { return dtype == PI_F32 ? at::kFloat : at::kHalf; }

void arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) fail(PyExc_TypeError, "%s: wrong number of arguments", "the binding");
}

// lens, q_start and the bound on a sequence's rows.
struct Bounds {
  const int32_t *lens, *q_start;
  int max_q;
};
// `most`: what the bound is at most where it is left out beside q_start.
Bounds bounds(const pi_kv_cache* c, PyObject* lens, PyObject* q_start, PyObject* max_q, int n_tok, int dev, int64_t most) {
  Bounds b;
  b.lens = int32s(lens, "lens", c->n_seqs, dev);
  b.q_start = nullptr;
  if (q_start == Py_None) {
    const int64_t m = max_q == Py_None ? n_tok / c->n_seqs : integer(max_q, "the bound on a sequence's rows");
    if (n_tok != m * c->n_seqs)
      fail(PyExc_ValueError, "%s there must be the same number of rows for every sequence", "without q_start");
    b.max_q = (int)m;
  } else {
    b.q_start = int32s(q_start, "q_start", (int64_t)c->n_seqs + 1, dev);
    b.max_q = max_q == Py_None ? (int)std::min<int64_t>(n_tok, most) : (int)integer(max_q, "the bound on a sequence's rows");
  }
  return b;
}

// (rope, dev, q, k, pos, q_out, k_out, stream)
int64_t qk_rope(PyObject* const* a, Py_ssize_t n) {
  arguments(n, 8);
  const pi_rope* r = descriptor<pi_rope>(a[0]);
  const int dev = (int)integer(a[1], "dev");
  const at::ScalarType dt = tensor(a[2], "q").scalar_type();
  if (dt != at::kHalf && dt != at::kFloat) fail(PyExc_TypeError, "%s must be float16 or float32", "q");
  const Rows q = rows(a[2], "q", -1, r->head_dim, dt, dev), k = rows(a[3], "k", -1, r->head_dim, dt, dev);
  const Rows qo = rows(a[5], "q_out", q.heads, r->head_dim, dt, dev);
  const Rows ko = rows(a[6], "k_out", k.heads, r->head_dim, dt, dev);
  same_tokens(q, k, "q and k"), same_tokens(q, qo, "q and q_out"), same_tokens(q, ko, "k and k_out");
  const int32_t* pos = int32s(a[4], "pos", q.n_tok, dev);
  if (q.n_tok == 0) return PI_OK;
  void* s = stream_of(a[7], dev);
  return queue(dev, [&] {
    return lib.qk_rope(r, q.p, q.ts, q.hs, q.heads, k.p, k.ts, k.hs, k.heads, pos, q.n_tok,
                       dt == at::kHalf ? PI_F16 : PI_F32, qo.p, qo.ts, qo.hs, ko.p, ko.ts, ko.hs, s);
  });
}

// (cache, dev, k, v, lens, q_start, max_new, stream)
template <bool READ>
int64_t kv_rows(PyObject* const* a, Py_ssize_t n) {
  arguments(n, 8);
  const pi_kv_cache* c = cache_of(a[0]);
  const int dev = (int)integer(a[1], "dev");
  const at::ScalarType dt = scalar_of(c->dtype);
  const Rows k = rows(a[2], READ ? "k_out" : "k", c->n_kv_heads, c->head_dim, dt, dev);
  const Rows v = rows(a[3], READ ? "v_out" : "v", c->n_kv_heads, c->head_dim, dt, dev);
  same_tokens(k, v, READ ? "k_out and v_out" : "k and v");
  // (a sequence's new rows are among those that its table row holds)
  const Bounds b = bounds(c, a[4], a[5], a[6], k.n_tok, dev, (int64_t)c->max_blocks * PI_KV_BLOCK);
  if (k.n_tok == 0) return PI_OK;
  void* s = stream_of(a[7], dev);
  return queue(dev, [&] {
    return READ ? lib.kv_read(c, b.lens, b.q_start, b.max_q, k.p, k.ts, k.hs, v.p, v.ts, v.hs, k.n_tok, s)
                : lib.kv_append(c, k.p, k.ts, k.hs, v.p, v.ts, v.hs, k.n_tok, b.lens, b.q_start, b.max_q, s);
  });
}

// (cache, dev, q, lens, out, q_start, max_q, max_len, scale, add_score, ws, stream)
int64_t attend(PyObject* const* a, Py_ssize_t n) {
  arguments(n, 12);
  const pi_kv_cache* c = cache_of(a[0]);
  const int dev = (int)integer(a[1], "dev");
  const at::ScalarType dt = scalar_of(c->dtype);
  const Rows q = rows(a[2], "q", -1, c->head_dim, dt, dev), out = rows(a[4], "out", q.heads, c->head_dim, dt, dev);
  same_tokens(q, out, "q and out");
  const Bounds b = bounds(c, a[3], a[5], a[6], q.n_tok, dev, q.n_tok);
  const int max_len = (int)integer(a[7], "max_len"), add_score = PyObject_IsTrue(a[9]);
  const float scale = (float)real(a[8]);
  const at::Tensor& ws = tensor(a[10], "ws");
  if (ws.scalar_type() != at::kByte || !ws.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous uint8", "ws");
  on_device(ws, "ws", dev);
  if (add_score && !c->score) fail(PyExc_ValueError, "%s needs a cache with a score", "add_score");
  if (q.n_tok == 0) return PI_OK;
  void* s = stream_of(a[11], dev);
  return queue(dev, [&] {
    return lib.attend(c, q.p, q.ts, q.hs, q.heads, q.n_tok, b.lens, b.q_start, b.max_q, max_len, scale, add_score,
                      out.p, out.ts, out.hs, ws.data_ptr(), (size_t)ws.numel(), s);
  });
}

// A contiguous [n_seqs][heads][blocks] tensor like `like`.
void* same(PyObject* o, const char* name, const at::Tensor& like, at::ScalarType dt, int dev) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != dt)
    fail(PyExc_TypeError, dt == at::kInt ? "%s must be torch.int32" : "%s must be torch.float32", name);
  on_device(t, name, dev);
  if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name);
  if (t.sizes() != like.sizes()) fail(PyExc_ValueError, "%s must have the shape of table", name);
  return t.data_ptr();
}

// (table, score, lens, keep, recent, lens_out, table_out, score_out, stream)
int64_t kv_evict(PyObject* const* a, Py_ssize_t n) {
  arguments(n, 9);
  const at::Tensor& table = tensor(a[0], "table");
  if (!table.is_cuda()) fail(PyExc_ValueError, "%s must live in GPU memory", "table");
  if (table.dim() != 3 || table.numel() > 0x7fffffffffff)
    fail(PyExc_ValueError, "%s must be [n_seqs, n_kv_heads, max_blocks]", "table");
  const int dev = table.get_device();
  auto* t = static_cast<int32_t*>(same(a[0], "table", table, at::kInt, dev));
  auto* s = static_cast<float*>(same(a[1], "score", table, at::kFloat, dev));
  auto* to = static_cast<int32_t*>(same(a[6], "table_out", table, at::kInt, dev));
  auto* so = static_cast<float*>(same(a[7], "score_out", table, at::kFloat, dev));
  for (int i = 0; i < 3; ++i)
    if (table.size(i) > 0x7fffffff) fail(PyExc_ValueError, "%s is too large", "table");
  const int32_t* lens = int32s(a[2], "lens", table.size(0), dev);
  int32_t* lens_out = int32s(a[5], "lens_out", table.size(0), dev);
  const int keep = (int)integer(a[3], "keep"), recent = (int)integer(a[4], "recent");
  void* st = stream_of(a[8], dev);
  return queue(dev, [&] {
    return lib.kv_evict(t, s, lens, (int)table.size(0), (int)table.size(1), (int)table.size(2), keep, recent, to, so,
                        lens_out, st);
  });
}

// (handle of the loaded libpi)
int64_t use_library(PyObject* const* a, Py_ssize_t n) {
  arguments(n, 1);
  void* h = PyLong_AsVoidPtr(a[0]);
  if (!h) fail(PyExc_ValueError, "%s is missing", "the library's handle");
  auto find = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(dlsym(h, name));
    if (!f) fail(PyExc_ImportError, "libpi.so lacks %s", name);
  };
  find(lib.qk_rope, "pi_qk_rope");
  find(lib.kv_append, "pi_kv_append");
  find(lib.kv_read, "pi_kv_read");
  find(lib.attend, "pi_attend");
  find(lib.kv_evict, "pi_kv_evict");
  return 0;
}

// No C++ exception reaches the interpreter.
template <int64_t (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    return PyLong_FromLongLong(F(args, n));
  } catch (const BadArgument&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <int64_t (*F)(PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F>));
}

PyMethodDef methods[] = {{"use_library", fast<use_library>(), METH_FASTCALL, nullptr},
                         {"qk_rope", fast<qk_rope>(), METH_FASTCALL, nullptr},
                         {"kv_append", fast<kv_rows<false>>(), METH_FASTCALL, nullptr},
                         {"kv_read", fast<kv_rows<true>>(), METH_FASTCALL, nullptr},
                         {"attend", fast<attend>(), METH_FASTCALL, nullptr},
                         {"kv_evict", fast<kv_evict>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn", "Entry points of the attention side (see attention.py).", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn(void) { return PyModule_Create(&module); }
