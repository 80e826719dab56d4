// The binding's calls that take a few microseconds on the GPU: argument checks
// and marshalling, as _serving.py's, compiled (from Python a tensor's checks
// cost half a microsecond each: the rotation of one token with its append took
// 8.5 us a call that way, its kernel 3). Each function takes the arguments of
// the package's function of its name, checked against one device, and the
// stream as a number; errors are the package's MdsError.
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <cmath>
#include <cstring>
#include <stdexcept>
#include <string>

#include "../../include/mds.h"

namespace {

PyObject* g_error = nullptr;  // MdsError

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
void need(bool ok, const char* message) {
  if (!ok) throw Refused(message);
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
int device(const at::Tensor& t) { return t.is_cuda() ? (int)t.get_device() : -1; }

int64_t whole(PyObject* o, const char* name, int64_t lo = INT32_MIN, int64_t hi = INT32_MAX) {
  int overflow = 0;
  const int64_t x = PyIndex_Check(o) ? PyLong_AsLongLongAndOverflow(o, &overflow) : -1;
  if (!PyIndex_Check(o) || overflow || x < lo || x > hi || (x == -1 && PyErr_Occurred())) {
    PyErr_Clear();
    throw Refused(std::string(name) + ": an argument is no integer or out of range");
  }
  return x;
}
double real(PyObject* o, const char* name) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused(std::string(name) + " must be a number");
  }
  return x;
}
bool truth(PyObject* o, const char* name) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) {
    PyErr_Clear();
    throw Refused(std::string(name) + " must be true or false");
  }
  return x != 0;
}
void* stream_of(PyObject* o) { return (void*)(uintptr_t)whole(o, "stream", INT64_MIN, INT64_MAX); }

// The pointer of a contiguous tensor of n elements on the device
void* vec(PyObject* o, at::ScalarType type, int64_t n, int dev, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type || t.numel() != n || device(t) != dev || !t.is_contiguous())
    throw Refused(std::string(name) + " must be a contiguous " + toString(type) + " tensor of " + std::to_string(n) +
                  " elements on cuda:" + std::to_string(dev));
  return t.data_ptr();
}
void* opt(PyObject* o, at::ScalarType type, int64_t n, int dev, const char* name) {
  return o == Py_None ? nullptr : vec(o, type, n, dev, name);
}
uint32_t* status_of(PyObject* o, int dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, "status");
  need(t.numel() == 1 && t.element_size() == 4 && device(t) == dev, "status: one 4-byte word on the device");
  return (uint32_t*)t.data_ptr();
}

// bf16 [T, H, D] with a unit last stride
struct Heads {
  void* p;
  int64_t ts, hs;
};
Heads heads(PyObject* o, int64_t T, int64_t H, int64_t D, int dev, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 3 || t.size(0) != T || t.size(1) != H || t.size(2) != D ||
      device(t) != dev || (t.stride(2) != 1 && t.numel()))
    throw Refused(std::string(name) + " must be bf16 [" + std::to_string(T) + ", " + std::to_string(H) + ", " +
                  std::to_string(D) + "] with a unit last stride on cuda:" + std::to_string(dev));
  return {t.data_ptr(), t.stride(0), t.stride(1)};
}

struct Pages {
  void *k, *v;
  int code;
  int64_t n, size, heads, dim, ks[3], vs[3];
};
Pages pages(PyObject* ko, PyObject* vo, int dev) {
  const at::Tensor &k = tensor(ko, "k_pages"), &v = tensor(vo, "v_pages");
  need(k.dim() == 4 && v.sizes() == k.sizes() && v.scalar_type() == k.scalar_type(),
       "k_pages and v_pages must be [n_pages, page_size, Hkv, D] of one shape and dtype");
  need(device(k) == dev && device(v) == dev, "the pages must be on the tensors' device");
  need(k.stride(3) == 1 && v.stride(3) == 1, "pages must have a unit last stride");
  const bool e4m3 = k.scalar_type() == at::kFloat8_e4m3fn;
  need(e4m3 || k.scalar_type() == at::kBFloat16, "unsupported cache dtype");
  Pages p{k.data_ptr(), v.data_ptr(), e4m3 ? MDS_E4M3 : MDS_BF16, k.size(0), k.size(1), k.size(2), k.size(3), {}, {}};
  for (int i = 0; i < 3; ++i) {
    p.ks[i] = k.stride(i);
    p.vs[i] = v.stride(i);
  }
  need(p.n <= INT32_MAX && p.size <= INT32_MAX && p.heads <= INT32_MAX && p.dim <= INT32_MAX, "the cache is too large");
  return p;
}

// Dimensions of a tensor that go over as int
int small(int64_t n, const char* name) {
  if (n > INT32_MAX) throw Refused(std::string(name) + " is too large");
  return (int)n;
}

// The library's call, which may wait for room in the stream's queue: other
// threads of the interpreter run meanwhile. It touches no Python object.
template <typename F>
PyObject* enqueue(const char* what, F call) {
  struct Others {
    PyThreadState* state = PyEval_SaveThread();
    ~Others() { PyEval_RestoreThread(state); }
  };
  const int rc = [&] {
    Others run;
    return call();
  }();
  if (rc) {
    PyErr_Format(g_error, "%s: %s (%d): %s", what, mds_status_string(rc), rc, mds_last_error());
    return nullptr;
  }
  Py_RETURN_NONE;
}
template <typename F>
PyObject* guarded(const char* what, Py_ssize_t got, Py_ssize_t want, F f) {
  try {
    need(got == want, "wrong number of arguments");
    return f();
  } catch (const Refused& e) {
    PyErr_SetString(g_error, e.what());
  } catch (const std::exception& e) {
    PyErr_Format(g_error, "%s: %s", what, e.what());
  } catch (...) {
    PyErr_Format(g_error, "%s: an unknown error", what);
  }
  return nullptr;
}

// Queries and keys of the two rotations, and what turns them
struct Rotation {
  int dev, T, Hq, Hk, D, R;
  Heads q, k, out;
  const int64_t* positions;
  const double* freq;
  void *q_weight, *k_weight;
  float eps;
  double scale;
  int interleaved;
};
Rotation rotation(PyObject* q, PyObject* k, PyObject* positions, PyObject* freq, PyObject* q_out, PyObject* q_weight,
                  PyObject* k_weight, PyObject* eps, PyObject* interleaved, PyObject* scale) {
  const at::Tensor &qt = tensor(q, "q"), &kt = tensor(k, "k");
  Rotation r;
  r.dev = device(qt);
  need(r.dev >= 0, "tensors must be on the GPU");
  need(qt.dim() == 3 && kt.dim() == 3, "q and k must be [T, heads, D]");
  r.T = small(qt.size(0), "T");
  r.Hq = small(qt.size(1), "Hq");
  r.D = small(qt.size(2), "D");
  r.Hk = small(kt.size(1), "Hkv");
  const int64_t half = freq == Py_None ? 0 : tensor(freq, "inv_freq").numel();
  r.R = small(2 * half, "inv_freq");
  r.q = heads(q, r.T, r.Hq, r.D, r.dev, "q");
  r.k = heads(k, r.T, r.Hk, r.D, r.dev, "k");
  r.out = heads(q_out, r.T, r.Hq, r.D, r.dev, "q_out");
  r.positions = (const int64_t*)vec(positions, at::kLong, r.T, r.dev, "positions");
  r.freq = (const double*)opt(freq, at::kDouble, half, r.dev, "inv_freq");
  r.q_weight = opt(q_weight, at::kBFloat16, r.D, r.dev, "q_weight");
  r.k_weight = opt(k_weight, at::kBFloat16, r.D, r.dev, "k_weight");
  r.eps = (float)real(eps, "eps");
  r.scale = real(scale, "rope_scale");
  r.interleaved = truth(interleaved, "interleaved");
  return r;
}

PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("qk_norm_rope", n, 12, [&] {
    const Rotation r = rotation(a[0], a[1], a[2], a[3], a[4], a[6], a[7], a[8], a[9], a[10]);
    const Heads ko = heads(a[5], r.T, r.Hk, r.D, r.dev, "k_out");
    void* stream = stream_of(a[11]);
    return enqueue("qk_norm_rope", [&] {
      return mds_qk_norm_rope(r.T, r.Hq, r.Hk, r.D, r.R, r.q.p, r.q.ts, r.q.hs, r.k.p, r.k.ts, r.k.hs, r.positions,
                              r.freq, r.q_weight, r.k_weight, r.eps, r.scale, r.interleaved, r.out.p, r.out.ts, r.out.hs,
                              ko.p, ko.ts, ko.hs, stream);
    });
  });
}

PyObject* qk_norm_rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("qk_norm_rope_append", n, 18, [&] {
    const Rotation r = rotation(a[0], a[1], a[3], a[4], a[5], a[9], a[10], a[11], a[12], a[13]);
    const Pages p = pages(a[6], a[7], r.dev);
    need(p.heads == r.Hk && p.dim == r.D, "the pages must be [n_pages, page_size, Hkv, D] of the keys' heads");
    const Heads v = heads(a[2], r.T, r.Hk, r.D, r.dev, "v");
    auto* slots = (const int64_t*)vec(a[8], at::kLong, r.T, r.dev, "slot_map");
    auto* ks = (const float*)opt(a[14], at::kFloat, r.Hk, r.dev, "k_scale");
    auto* vs = (const float*)opt(a[15], at::kFloat, r.Hk, r.dev, "v_scale");
    uint32_t* status = status_of(a[16], r.dev);
    void* stream = stream_of(a[17]);
    return enqueue("qk_norm_rope_append", [&] {
      return mds_qk_norm_rope_append(
          r.T, r.Hq, r.Hk, r.D, r.R, r.q.p, r.q.ts, r.q.hs, r.k.p, r.k.ts, r.k.hs, v.p, v.ts, v.hs, r.positions, r.freq,
          r.q_weight, r.k_weight, r.eps, r.scale, r.interleaved, r.out.p, r.out.ts, r.out.hs, p.k, p.v, p.code,
          (int)p.size, (int)p.n, p.ks[0], p.ks[1], p.ks[2], p.vs[0], p.vs[1], p.vs[2], slots, ks, vs, status, stream);
    });
  });
}

PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("paged_attention", n, 19, [&] {
    const at::Tensor &q = tensor(a[0], "q"), &table = tensor(a[3], "block_table"), &ws = tensor(a[17], "workspace");
    const int dev = device(q);
    need(dev >= 0, "tensors must be on the GPU");
    const Pages p = pages(a[1], a[2], dev);
    need(q.dim() == 3, "q must be bf16 [T, Hq, D]");
    const int T = small(q.size(0), "T"), Hq = small(q.size(1), "Hq");
    const Heads qh = heads(a[0], T, Hq, p.dim, dev, "q"), oh = heads(a[6], T, Hq, p.dim, dev, "out");
    const int B = small(tensor(a[5], "seq_lens").numel(), "B");
    need(table.dim() == 2, "block_table must be [n_slots, max_pages]");
    const int N = small(table.size(0), "n_slots"), MP = small(table.size(1), "max_pages");
    need(ws.scalar_type() == at::kByte && device(ws) == dev && ws.is_contiguous(),
         "workspace must be a contiguous uint8 tensor on the tensors' device");
    void* work = ws.data_ptr();
    const size_t work_bytes = (size_t)ws.numel();
    const float scale = a[9] == Py_None ? (float)(1.0 / std::sqrt((double)p.dim)) : (float)real(a[9], "scale");
    auto* tables = (const int32_t*)vec(a[3], at::kInt, (int64_t)N * MP, dev, "block_table");
    auto* map = (const int32_t*)opt(a[13], at::kInt, B, dev, "idx_map");
    auto* start = (const int32_t*)vec(a[4], at::kInt, (int64_t)B + 1, dev, "query_start");
    auto* lens = (const int32_t*)vec(a[5], at::kInt, B, dev, "seq_lens");
    const int max_q = (int)whole(a[7], "max_q_len");
    const int64_t max_seq = whole(a[8], "max_seq_len", INT64_MIN, INT64_MAX);
    const int causal = truth(a[10], "causal"), window = (int)whole(a[11], "window"), sinks = (int)whole(a[12], "sinks");
    auto* ks = (const float*)opt(a[14], at::kFloat, p.heads, dev, "k_scale");
    auto* vs = (const float*)opt(a[15], at::kFloat, p.heads, dev, "v_scale");
    float* lse = (float*)opt(a[16], at::kFloat, (int64_t)T * Hq, dev, "lse");
    void* stream = stream_of(a[18]);
    return enqueue("paged_attention", [&] {
      return mds_paged_attention_sinks(T, B, Hq, (int)p.heads, (int)p.dim, qh.p, qh.ts, qh.hs, p.k, p.v, p.code,
                                       (int)p.size, (int)p.n, p.ks[0], p.ks[1], p.ks[2], p.vs[0], p.vs[1], p.vs[2],
                                       tables, N, MP, map, start, lens, max_q, max_seq, scale, causal, window, sinks, ks,
                                       vs, oh.p, oh.ts, oh.hs, lse, work, work_bytes, stream);
    });
  });
}

PyObject* lm_head_mxfp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("lm_head_mxfp4", n, 6, [&] {
    const at::Tensor &x = tensor(a[0], "hidden"), &o = tensor(a[3], "out");
    const int dev = device(x);
    need(dev >= 0, "tensors must be on the GPU");
    const int K = (int)whole(a[4], "K");
    need(x.scalar_type() == at::kBFloat16 && x.dim() == 2 && x.stride(1) == 1 && K >= 1 && x.size(0) % K == 0,
         "hidden must be bf16 [B*K, H] with unit column stride");
    const int H = small(x.size(1), "H"), B = small(x.size(0) / K, "B");
    need(o.dim() == 3 && o.size(0) == B && o.size(1) >= K && o.stride(2) == 1 && device(o) == dev,
         "out must be [B, >=K, V] with unit column stride");
    const int V = small(o.size(2), "V");
    auto tiles = [&](PyObject* p, int64_t columns, const char* message) {
      const at::Tensor& t = tensor(p, "lm_head and scales");
      need(t.scalar_type() == at::kByte && t.dim() == 2 && t.size(0) == ((int64_t)V + 15) / 16 && t.size(1) == columns &&
               t.is_contiguous() && device(t) == dev,
           message);
      return t.data_ptr();
    };
    void* w = tiles(a[1], 8 * (int64_t)H, "the tiled codes must be contiguous uint8 [ceil(V/16), 8 H]");
    void* s = tiles(a[2], 256 * (((int64_t)H + 511) / 512),
                    "the tiled scales must be contiguous uint8 [ceil(V/16), 256 ceil(H/512)]");
    need(o.scalar_type() == at::kFloat || o.scalar_type() == at::kBFloat16, "unsupported dtype: out must be float32 or bf16");
    const int type = o.scalar_type() == at::kFloat ? MDS_F32 : MDS_BF16;
    void *xp = x.data_ptr(), *op = o.data_ptr(), *stream = stream_of(a[5]);
    const int64_t xs = x.stride(0), bs = o.stride(0), rs = o.stride(1);
    return enqueue("lm_head_mxfp4",
                   [&] { return mds_lm_head_mxfp4(B, K, V, H, xp, xs, w, s, op, type, bs, rs, stream); });
  });
}

// set_error(MdsError): the class of the errors raised here
PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XSETREF(g_error, type);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, (PyCFunction)(void (*)())F, METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {method<qk_norm_rope>("qk_norm_rope"),
                           method<qk_norm_rope_append>("qk_norm_rope_append"),
                           method<paged_attention>("paged_attention"),
                           method<lm_head_mxfp4>("lm_head_mxfp4"),
                           {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

// Whether the library and torch that are loaded are those whose declarations this was compiled with
bool fits() {
  if (mds_abi_version() != MDS_ABI_VERSION) {
    PyErr_Format(PyExc_ImportError, "built for version %d of the library's interface, which is %d", MDS_ABI_VERSION,
                 mds_abi_version());
    return false;
  }
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* version = torch ? PyObject_GetAttrString(torch, "__version__") : nullptr;
  const char* v = version ? PyUnicode_AsUTF8(version) : nullptr;
  const size_t n = sizeof(TORCH_VERSION) - 1;
  // (2.10.0, and 2.10.0+rocm7.0, but not 2.10.01)
  const bool same = v && strncmp(v, TORCH_VERSION, n) == 0 && !(v[n] >= '0' && v[n] <= '9');
  if (v && !same) PyErr_Format(PyExc_ImportError, "built with torch %s, not %s", TORCH_VERSION, v);
  Py_XDECREF(version);
  Py_XDECREF(torch);
  return same;
}

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  if (!fits()) return nullptr;
  PyObject* m = PyModule_Create(&g_module);
  if (!m) return nullptr;
  Py_INCREF(PyExc_RuntimeError);
  g_error = PyExc_RuntimeError;  // until set_error
  return m;
}
