// The short way from Python to the rotary, decode and serving entry points.
//
// A decode step is 4 to 15 us of GPU work, and the checks, allocations and
// argument conversions of the binding's Python functions cost 16 to 30 us
// around it. These functions do the same for the ordinary case (tensors of
// the right types and shapes on the current device, the current stream) in a
// few. In every other case, and when the library refuses the call before it
// launches anything, they return None and the Python function does it all
// itself: what is wrong is found and told there, and nothing depends on this
// module but time. A call that may have launched is never made again: its
// error is raised here.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <ATen/ops/zeros_like.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <utility>

#include "../../include/swa_attn.h"

namespace {

struct Lib {
  decltype(&swa_rope_tables) tables;
  decltype(&swa_rope_apply) apply;
  decltype(&swa_kv4_plan) plan;
  decltype(&swa_kv4_append) append;
  decltype(&swa_kv4_read) read;
  decltype(&swa_kv4_attn) attn;
};
Lib libs[2];   // bf16, fp32; filled by bind()
struct More {
  decltype(&swa_rms_norm) norm;
  decltype(&swa_rms_norm_workspace_size) norm_ws;
  decltype(&swa_rms_norm_bwd) norm_bwd;
  decltype(&swa_w4_linear) linear;
  decltype(&swa_kv4_tree) tree;
  decltype(&swa_kv4_tree_attn) tree_attn;
  decltype(&swa_kv4_move) move;
};
More more[2];  // likewise, by bind_more()

struct Refused {};   // not the ordinary case; nothing is launched

PyObject* error_type = nullptr;   // SwaError(status, what); set by raises()

// Lets other Python threads run for its life.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// The library call of a function below: its status, and whether it may have
// launched.
struct Call {
  bool launched = false;
  swa_status status = SWA_OK;
  // Runs f, which allocates outputs and makes the call, both of which may wait
  // for the device; nothing of Python is used in it. INVALID_ARG, UNSUPPORTED
  // and WORKSPACE are decided before a launch. Any other status may come after
  // it: SWA_ERR_CUDA also tells of errors that older calls left behind.
  template <typename F>
  void operator()(F f) {
    swa_status s;
    {
      Unlocked unlocked;
      s = f();
    }
    if (s == SWA_ERR_INVALID_ARG || s == SWA_ERR_UNSUPPORTED || s == SWA_ERR_WORKSPACE) throw Refused{};
    launched = true;
    status = s;
  }
};

int device_now() { return static_cast<int>(c10::cuda::current_device()); }
void* stream_now(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw Refused{};
  return THPVariable_Unpack(o);
}
// Address of a tensor after its checks; None passes as NULL.
void* at_(PyObject* o, at::ScalarType type, int dev, at::IntArrayRef shape) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o);
  if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev || t.sizes() != shape || !t.is_contiguous())
    throw Refused{};
  return t.data_ptr();
}
int small(int64_t x) {
  if (x < 0 || x > INT32_MAX) throw Refused{};
  return static_cast<int>(x);
}
int int_of(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (PyErr_Occurred() || x < INT32_MIN || x > INT32_MAX) throw Refused{};
  return static_cast<int>(x);
}
double double_of(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) throw Refused{};
  return x;
}
bool truth_of(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw Refused{};
  return x != 0;
}
int kind_of(at::ScalarType t) {
  const int kind = t == at::kBFloat16 ? 0 : (t == at::kFloat ? 1 : -1);
  if (kind < 0 || libs[kind].attn == nullptr) throw Refused{};   // another type, or its library is not loaded yet
  return kind;
}
// Rotary tables: false where there are none.
bool rope_of(PyObject* cos, PyObject* sin, PyObject* interleaved, int dev, swa_rope& r) {
  if (cos == Py_None) return false;
  const at::Tensor& c = tensor(cos);
  if (c.dim() != 2) throw Refused{};
  r.cos = static_cast<const float*>(at_(cos, at::kFloat, dev, c.sizes()));
  r.sin = static_cast<const float*>(at_(sin, at::kFloat, dev, c.sizes()));
  if (r.sin == nullptr) throw Refused{};
  r.rows = small(c.size(0));
  r.rot = small(2 * c.size(1));
  r.interleaved = truth_of(interleaved);
  return true;
}
struct Ws {
  void* at;
  size_t bytes;
};
Ws ws_of(PyObject* o, int dev) {
  if (o == Py_None) return {nullptr, 0};
  const at::Tensor& t = tensor(o);
  return {at_(o, at::kByte, dev, {t.numel()}), static_cast<size_t>(t.numel())};
}
struct CacheDims {
  swa_kv4_cache c;
  int Hkv, d;
};
CacheDims cache_of(PyObject* o, int dev) {
  const at::Tensor& t = tensor(o);
  if (t.dim() != 4 || (t.size(3) != 18 * 64 && t.size(3) != 18 * 128)) throw Refused{};
  CacheDims x{};
  x.c.data = at_(o, at::kByte, dev, t.sizes());
  x.c.n_pages = small(t.size(0));
  x.Hkv = small(t.size(1));
  x.c.page = small(16 * t.size(2));
  x.d = small(t.size(3) / 18);
  return x;
}
at::TensorOptions on(int dev, at::ScalarType type) {
  return at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)));
}
PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  PyObject* x = a.defined() ? THPVariable_Wrap(a) : Py_NewRef(Py_None);
  PyObject* y = b.defined() ? THPVariable_Wrap(b) : Py_NewRef(Py_None);
  PyObject* t = PyTuple_Pack(2, x, y);
  Py_DECREF(x);
  Py_DECREF(y);
  return t;
}

// Runs f, whose library call is `what`; anything out of the ordinary before
// the launch is None.
template <typename F>
PyObject* guarded(const char* what, F f) {
  Call call;
  PyObject* r = nullptr;
  try {
    r = f(call);
  } catch (...) {
    r = nullptr;
  }
  if (!call.launched) {
    if (r != nullptr) return r;
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  if (call.status != SWA_OK) {
    Py_XDECREF(r);
    PyErr_Clear();
    PyObject* e = error_type != nullptr ? PyObject_CallFunction(error_type, "is", static_cast<int>(call.status), what) : nullptr;
    if (e != nullptr) PyErr_SetObject(error_type, e);
    Py_XDECREF(e);
    r = nullptr;
  }
  if (r == nullptr && !PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s: failed after its launch", what);
  return r;
}

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) Py_RETURN_NONE;
  return guarded("bind", [&](Call&) -> PyObject* {
    void* f[6];
    for (int i = 0; i < 6; ++i) f[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (PyErr_Occurred()) throw Refused{};
    libs[int_of(a[0]) & 1] = Lib{reinterpret_cast<decltype(&swa_rope_tables)>(f[0]), reinterpret_cast<decltype(&swa_rope_apply)>(f[1]),
                                 reinterpret_cast<decltype(&swa_kv4_plan)>(f[2]), reinterpret_cast<decltype(&swa_kv4_append)>(f[3]),
                                 reinterpret_cast<decltype(&swa_kv4_read)>(f[4]), reinterpret_cast<decltype(&swa_kv4_attn)>(f[5])};
    Py_RETURN_TRUE;
  });
}

PyObject* bind_more(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) Py_RETURN_NONE;
  return guarded("bind_more", [&](Call&) -> PyObject* {
    void* f[7];
    for (int i = 0; i < 7; ++i) f[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (PyErr_Occurred()) throw Refused{};
    more[int_of(a[0]) & 1] =
        More{reinterpret_cast<decltype(&swa_rms_norm)>(f[0]),     reinterpret_cast<decltype(&swa_rms_norm_workspace_size)>(f[1]),
             reinterpret_cast<decltype(&swa_rms_norm_bwd)>(f[2]), reinterpret_cast<decltype(&swa_w4_linear)>(f[3]),
             reinterpret_cast<decltype(&swa_kv4_tree)>(f[4]),     reinterpret_cast<decltype(&swa_kv4_tree_attn)>(f[5]),
             reinterpret_cast<decltype(&swa_kv4_move)>(f[6])};
    Py_RETURN_TRUE;
  });
}
// As kind_of, for the functions of More.
int kind_more(at::ScalarType t) {
  const int kind = t == at::kBFloat16 ? 0 : (t == at::kFloat ? 1 : -1);
  if (kind < 0 || more[kind].move == nullptr) throw Refused{};
  return kind;
}
PyObject* dict_of(std::initializer_list<std::pair<const char*, const at::Tensor*>> items) {
  PyObject* dict = PyDict_New();
  for (const auto& i : items) {
    PyObject* v = i.second != nullptr && i.second->defined() ? THPVariable_Wrap(*i.second) : Py_NewRef(Py_None);
    PyDict_SetItemString(dict, i.first, v);
    Py_DECREF(v);
  }
  return dict;
}

PyObject* raises(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 1 || !PyType_Check(a[0])) Py_RETURN_NONE;
  Py_INCREF(a[0]);
  Py_XDECREF(error_type);
  error_type = a[0];
  Py_RETURN_TRUE;
}

// rope_tables(rows, rot, scaling, base, factor, orig_len, slow, fast, amplitude, first)
PyObject* rope_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 10 || libs[0].tables == nullptr) Py_RETURN_NONE;
  return guarded("swa_rope_tables", [&](Call& call) -> PyObject* {
    const int dev = device_now(), rows = int_of(a[0]), first = int_of(a[9]);
    swa_rope_freq f{int_of(a[1]), int_of(a[2]), double_of(a[3]), double_of(a[4]), double_of(a[5]),
                    double_of(a[6]), double_of(a[7]), double_of(a[8])};
    if (rows < 1 || f.rot < 2) throw Refused{};
    at::Tensor cos, sin;
    call([&] {
      cos = at::empty({rows, f.rot / 2}, on(dev, at::kFloat));
      sin = at::empty_like(cos);
      return libs[0].tables(&f, first, rows, cos.data_ptr<float>(), sin.data_ptr<float>(), stream_now(dev));
    });
    return pair(cos, sin);
  });
}

// rope_apply(q, k, cos, sin, pos, interleaved, inverse, q_out, k_out, workspace)
PyObject* rope_apply(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 10) Py_RETURN_NONE;
  return guarded("swa_rope_apply", [&](Call& call) -> PyObject* {
    const bool has_q = a[0] != Py_None, has_k = a[1] != Py_None;
    const at::Tensor& x = tensor(has_q ? a[0] : a[1]);
    if (x.dim() != 4) throw Refused{};
    const int dev = device_now();
    const auto type = x.scalar_type();
    const int kind = kind_of(type);
    const int64_t B = x.size(0), T = x.size(1), d = x.size(3);
    int64_t Hq = x.size(2), Hkv = Hq;
    if (has_q) {
      Hkv = 1;
      if (has_k) {
        if (tensor(a[1]).dim() != 4) throw Refused{};
        Hkv = tensor(a[1]).size(2);
      }
    }
    const void* q = at_(a[0], type, dev, {B, T, Hq, d});
    const void* k = at_(a[1], type, dev, {B, T, Hkv, d});
    const int32_t* pos = static_cast<const int32_t*>(at_(a[4], at::kInt, dev, {B, T}));
    swa_rope r{};
    if (!rope_of(a[2], a[3], a[5], dev, r)) throw Refused{};
    void* qo = at_(a[7], type, dev, {B, T, Hq, d});
    void* ko = at_(a[8], type, dev, {B, T, Hkv, d});
    const Ws ws = ws_of(a[9], dev);
    // Outputs allocated here hold nothing yet: the call is told so, or, beside
    // one of the caller's, they begin as zeros where a row may be left out.
    const bool fresh = qo == nullptr && ko == nullptr, zeros = !fresh && pos != nullptr;
    if ((qo == nullptr && a[7] != Py_None) || (ko == nullptr && a[8] != Py_None)) throw Refused{};
    const int mode = (truth_of(a[6]) ? 1 : 0) | (fresh ? SWA_ROPE_NEW_OUTPUTS : 0);
    const swa_params p{small(B), small(T), small(Hq), small(Hkv), small(d), -1, 1, 0.f, 0.f, 0.f, 0};
    const at::Tensor none;
    const at::Tensor &qi = has_q ? tensor(a[0]) : none, &ki = has_k ? tensor(a[1]) : none;
    at::Tensor qt = has_q && qo != nullptr ? tensor(a[7]) : none, kt = has_k && ko != nullptr ? tensor(a[8]) : none;
    call([&] {
      if (has_q && qo == nullptr) {
        qt = zeros ? at::zeros_like(qi) : at::empty_like(qi);
        qo = qt.data_ptr();
      }
      if (has_k && ko == nullptr) {
        kt = zeros ? at::zeros_like(ki) : at::empty_like(ki);
        ko = kt.data_ptr();
      }
      return libs[kind].apply(&p, &r, pos, q, k, qo, ko, mode, ws.at, ws.bytes, stream_now(dev));
    });
    return pair(qt, kt);
  });
}

// kv4_plan(lens, new_lens, table, free_pages, free_head, page, n_pages, n_tokens, workspace)
PyObject* kv4_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 9 || libs[0].plan == nullptr) Py_RETURN_NONE;
  return guarded("swa_kv4_plan", [&](Call& call) -> PyObject* {
    const int dev = device_now();
    const at::Tensor &lens = tensor(a[0]), &table = tensor(a[2]), &free = tensor(a[3]);
    if (lens.dim() != 1 || table.dim() != 2) throw Refused{};
    const int64_t B = lens.size(0), N = int_of(a[7]);
    if (N < 0 || B < 1) throw Refused{};
    const auto* l = static_cast<const int32_t*>(at_(a[0], at::kInt, dev, {B}));
    const auto* nl = static_cast<const int32_t*>(at_(a[1], at::kInt, dev, {B}));
    auto* tb = static_cast<int32_t*>(at_(a[2], at::kInt, dev, {B, table.size(1)}));
    const auto* fr = static_cast<const int32_t*>(at_(a[3], at::kInt, dev, {free.numel()}));
    const auto* hd = static_cast<const int32_t*>(at_(a[4], at::kInt, dev, {1}));
    const Ws ws = ws_of(a[8], dev);
    const int page = int_of(a[5]), n_pages = int_of(a[6]), b = small(B), width = small(table.size(1)), n_free = small(free.numel());
    at::Tensor slot, pos, row, cu, lens_out, head;
    call([&] {
      const auto i32 = on(dev, at::kInt);
      slot = at::empty({N}, on(dev, at::kLong));
      pos = at::empty({N}, i32);
      row = at::empty({N}, i32);
      cu = at::empty({B + 1}, i32);
      lens_out = at::empty({B}, i32);
      head = at::empty({1}, i32);
      return libs[0].plan(n_pages, page, b, width, l, nl, tb, fr, n_free, hd, static_cast<int>(N), slot.data_ptr<int64_t>(),
                          pos.data_ptr<int32_t>(), row.data_ptr<int32_t>(), cu.data_ptr<int32_t>(), lens_out.data_ptr<int32_t>(),
                          head.data_ptr<int32_t>(), ws.at, ws.bytes, stream_now(dev));
    });
    PyObject* dict = PyDict_New();
    const struct { const char* name; const at::Tensor& t; } out[] = {
        {"slot", slot}, {"pos", pos}, {"row", row}, {"cu", cu}, {"lens", lens_out}, {"free_head", head}};
    for (const auto& o : out) {
      PyObject* v = THPVariable_Wrap(o.t);
      PyDict_SetItemString(dict, o.name, v);
      Py_DECREF(v);
    }
    return dict;
  });
}

// kv4_append(cache, k, v, slot, pos, cos, sin, interleaved, gk, eps, ve, tok, ve_gate, ve_scale, workspace)
PyObject* kv4_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 15) Py_RETURN_NONE;
  return guarded("swa_kv4_append", [&](Call& call) -> PyObject* {
    const int dev = device_now();
    const CacheDims c = cache_of(a[0], dev);
    const at::Tensor& k = tensor(a[1]);
    if (k.dim() != 4) throw Refused{};
    const auto type = k.scalar_type();
    const int kind = kind_of(type);
    const int64_t B = k.size(0), T = k.size(1);
    const at::DimVector rows{B, T, c.Hkv, c.d};
    const void *ka = at_(a[1], type, dev, rows), *va = at_(a[2], type, dev, rows);
    const auto* slot = static_cast<const int64_t*>(at_(a[3], at::kLong, dev, {B, T}));
    const auto* pos = static_cast<const int32_t*>(at_(a[4], at::kInt, dev, {B, T}));
    swa_rope r{};
    const bool rope = rope_of(a[5], a[6], a[7], dev, r);
    const auto* gk = static_cast<const float*>(at_(a[8], at::kFloat, dev, {c.d}));
    const void* ve = nullptr;
    const int32_t* tok = nullptr;
    const float* gate = nullptr;
    int vocab = 0;
    if (a[10] != Py_None) {
      if (tensor(a[10]).dim() != 2) throw Refused{};
      vocab = small(tensor(a[10]).size(0));
      ve = at_(a[10], type, dev, {vocab, static_cast<int64_t>(c.Hkv) * c.d});
      tok = static_cast<const int32_t*>(at_(a[11], at::kInt, dev, {B, T}));
      gate = static_cast<const float*>(at_(a[12], at::kFloat, dev, {B, T, c.Hkv}));
    }
    const Ws ws = ws_of(a[14], dev);
    const swa_params p{small(B), small(T), c.Hkv, c.Hkv, c.d, -1, 1, 0.f, static_cast<float>(double_of(a[9])),
                       static_cast<float>(double_of(a[13])), vocab};
    call([&] {
      return libs[kind].append(&p, nullptr, &c.c, rope ? &r : nullptr, ka, va, gk, ve, tok, gate, pos, slot, ws.at, ws.bytes,
                               stream_now(dev));
    });
    Py_RETURN_TRUE;
  });
}

// kv4_read(cache, slot, fp32, workspace)
PyObject* kv4_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) Py_RETURN_NONE;
  return guarded("swa_kv4_read", [&](Call& call) -> PyObject* {
    const int dev = device_now();
    const CacheDims c = cache_of(a[0], dev);
    const at::Tensor& s = tensor(a[1]);
    if (s.dim() != 2) throw Refused{};
    const int kind = kind_of(truth_of(a[2]) ? at::kFloat : at::kBFloat16);
    const auto* slot = static_cast<const int64_t*>(at_(a[1], at::kLong, dev, s.sizes()));
    const Ws ws = ws_of(a[3], dev);
    const swa_params p{small(s.size(0)), small(s.size(1)), c.Hkv, c.Hkv, c.d, -1, 1, 0.f, 0.f, 0.f, 0};
    at::Tensor k, v;
    call([&] {
      k = at::empty({p.B, p.T, c.Hkv, c.d}, on(dev, kind ? at::kFloat : at::kBFloat16));
      v = at::empty_like(k);
      return libs[kind].read(&p, &c.c, slot, k.data_ptr(), v.data_ptr(), ws.at, ws.bytes, stream_now(dev));
    });
    return pair(k, v);
  });
}

// kv4_attention(cache, q, table, lens, cos, sin, interleaved, gq, window, softmax_scale, eps, workspace)
PyObject* kv4_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 12) Py_RETURN_NONE;
  return guarded("swa_kv4_attn", [&](Call& call) -> PyObject* {
    const int dev = device_now();
    const CacheDims c = cache_of(a[0], dev);
    const at::Tensor &q = tensor(a[1]), &table = tensor(a[2]);
    if (q.dim() != 3 || table.dim() != 2 || a[11] == Py_None) throw Refused{};
    const auto type = q.scalar_type();
    const int kind = kind_of(type);
    const int64_t B = q.size(0), Hq = q.size(1), width = table.size(1);
    const void* qa = at_(a[1], type, dev, {B, Hq, c.d});
    const auto* ta = static_cast<const int32_t*>(at_(a[2], at::kInt, dev, {B, width}));
    const auto* la = static_cast<const int32_t*>(at_(a[3], at::kInt, dev, {B}));
    swa_rope r{};
    const bool rope = rope_of(a[4], a[5], a[6], dev, r);
    const auto* gq = static_cast<const float*>(at_(a[7], at::kFloat, dev, {c.d}));
    const Ws ws = ws_of(a[11], dev);
    const swa_params p{small(B), 1, small(Hq), c.Hkv, c.d, int_of(a[8]), 1, static_cast<float>(double_of(a[9])),
                       static_cast<float>(double_of(a[10])), 0.f, 0};
    const int max_pages = small(width);
    at::Tensor o, lse;
    call([&] {
      o = at::empty_like(q);
      lse = at::empty({B, Hq}, on(dev, at::kFloat));
      return libs[kind].attn(&p, nullptr, &c.c, rope ? &r : nullptr, qa, gq, ta, max_pages, la, o.data_ptr(), lse.data_ptr<float>(),
                             ws.at, ws.bytes, stream_now(dev));
    });
    return pair(o, lse);
  });
}

// rms_norm(x, gain, add, eps, fp8, inplace)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) Py_RETURN_NONE;
  return guarded("swa_rms_norm", [&](Call& call) -> PyObject* {
    const int dev = device_now();
    const at::Tensor& x = tensor(a[0]);
    if (x.dim() < 1 || x.numel() == 0) throw Refused{};
    const auto type = x.scalar_type();
    const int kind = kind_more(type);
    const int64_t C = x.size(-1), rows = x.numel() / C;
    void* xa = at_(a[0], type, dev, x.sizes());
    const auto* g = static_cast<const float*>(at_(a[1], at::kFloat, dev, {C}));
    const void* add = at_(a[2], type, dev, x.sizes());
    const float eps = static_cast<float>(double_of(a[3]));
    const bool fp8 = truth_of(a[4]), over = truth_of(a[5]);
    const int width = small(C);
    at::Tensor h = x, y, rstd, scale;
    call([&] {
      if (add != nullptr && !over) h = at::empty_like(x);
      y = at::empty(x.sizes(), on(dev, fp8 ? at::kFloat8_e4m3fn : type));
      rstd = at::empty(x.sizes().slice(0, x.dim() - 1), on(dev, at::kFloat));
      if (fp8) scale = at::empty_like(rstd);
      return more[kind].norm(rows, width, eps, xa, add, g, add != nullptr ? h.data_ptr() : nullptr, fp8 ? nullptr : y.data_ptr(),
                             fp8 ? y.data_ptr() : nullptr, fp8 ? scale.data_ptr<float>() : nullptr, rstd.data_ptr<float>(), stream_now(dev));
    });
    PyObject* r = dict_of({{"y", &y}, {"scale", &scale}, {"rstd", &rstd}, {"h", &h}});
    if (add == nullptr || over) PyDict_SetItemString(r, "h", a[0]);
    return r;
  });
}

// rms_norm_backward(h, rstd, dy, gain, dh, workspace)
PyObject* rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) Py_RETURN_NONE;
  return guarded("swa_rms_norm_bwd", [&](Call& call) -> PyObject* {
    const int dev = device_now();
    const at::Tensor& h = tensor(a[0]);
    if (h.dim() < 1 || h.numel() == 0) throw Refused{};
    const auto type = h.scalar_type();
    const int kind = kind_more(type);
    const int64_t C = h.size(-1), rows = h.numel() / C;
    const void* ha = at_(a[0], type, dev, h.sizes());
    const auto* rs = static_cast<const float*>(at_(a[1], at::kFloat, dev, h.sizes().slice(0, h.dim() - 1)));
    const void* dy = at_(a[2], type, dev, h.sizes());
    const auto* g = static_cast<const float*>(at_(a[3], at::kFloat, dev, {C}));
    const void* dh = at_(a[4], type, dev, h.sizes());
    const Ws ws = ws_of(a[5], dev);
    const int width = small(C);
    if (rs == nullptr || dy == nullptr) throw Refused{};
    at::Tensor dx, dg, part;
    call([&] {
      dx = at::empty_like(h);
      dg = at::empty({C}, on(dev, at::kFloat));
      void* at = ws.at;
      size_t bytes = ws.bytes;
      if (at == nullptr) {
        bytes = more[kind].norm_ws(rows, width);
        part = at::empty({static_cast<int64_t>(bytes)}, on(dev, at::kByte));
        at = part.data_ptr();
      }
      return more[kind].norm_bwd(rows, width, ha, rs, g, dy, dh, dx.data_ptr(), dg.data_ptr<float>(), at, bytes, stream_now(dev));
    });
    return dict_of({{"dx", &dx}, {"dgain", &dg}});
  });
}

// w4_linear(x, w4, out_features (None: all), scale, add, dtype (0: x's, or bf16 with a scale; 1: bf16; 2: fp32), out, workspace)
PyObject* w4_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) Py_RETURN_NONE;
  return guarded("swa_w4_linear", [&](Call& call) -> PyObject* {
    const int dev = device_now();
    const at::Tensor &x = tensor(a[0]), &w = tensor(a[1]);
    if (x.dim() < 1 || x.numel() == 0 || w.dim() != 3) throw Refused{};
    const bool x8 = a[3] != Py_None;
    const int want = int_of(a[5]);
    const auto type = want == 0 ? (x8 ? at::kBFloat16 : x.scalar_type()) : (want == 1 ? at::kBFloat16 : at::kFloat);
    const int kind = kind_more(type);
    const int64_t K = x.size(-1), M = x.numel() / K, N = a[2] == Py_None ? 16 * w.size(0) : int_of(a[2]);
    if (N < 1) throw Refused{};
    const void* xa = at_(a[0], x8 ? at::kFloat8_e4m3fn : type, dev, x.sizes());
    const void* wa = at_(a[1], at::kByte, dev, {(N + 15) / 16, (K + 63) / 64, 544});
    const auto* sa = static_cast<const float*>(at_(a[3], at::kFloat, dev, x.sizes().slice(0, x.dim() - 1)));
    at::DimVector shape(x.sizes().begin(), x.sizes().end());
    shape.back() = N;
    const void* add = at_(a[4], type, dev, shape);
    void* to = at_(a[6], type, dev, shape);
    const Ws ws = ws_of(a[7], dev);
    const int m = small(M), nn = small(N), k = small(K);
    if (to == nullptr && a[6] != Py_None) throw Refused{};
    at::Tensor y;
    if (to != nullptr) y = tensor(a[6]);
    call([&] {
      if (to == nullptr) {
        y = at::empty(shape, on(dev, type));
        to = y.data_ptr();
      }
      return more[kind].linear(m, nn, k, xa, sa, wa, add, to, ws.at, ws.bytes, stream_now(dev));
    });
    return a[6] != Py_None ? Py_NewRef(a[6]) : THPVariable_Wrap(y);
  });
}

// kv4_tree(parent, cu, lens, max_new, workspace)
PyObject* kv4_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5 || more[0].tree == nullptr) Py_RETURN_NONE;
  return guarded("swa_kv4_tree", [&](Call& call) -> PyObject* {
    const int dev = device_now();
    const at::Tensor &parent = tensor(a[0]), &cu = tensor(a[1]);
    if (parent.dim() != 1 || cu.dim() != 1 || cu.numel() < 1 || parent.numel() < 1) throw Refused{};
    const int64_t N = parent.size(0), B = cu.size(0) - 1;
    const auto* pa = static_cast<const int32_t*>(at_(a[0], at::kInt, dev, {N}));
    const auto* ca = static_cast<const int32_t*>(at_(a[1], at::kInt, dev, {B + 1}));
    const auto* la = static_cast<const int32_t*>(at_(a[2], at::kInt, dev, {B}));
    const int most = int_of(a[3]), b = small(B), rows = small(N);
    const Ws ws = ws_of(a[4], dev);
    at::Tensor pos, seen;
    call([&] {
      pos = at::empty({N}, on(dev, at::kInt));
      seen = at::empty({N}, on(dev, at::kLong));
      return more[0].tree(b, rows, most, pa, ca, la, pos.data_ptr<int32_t>(), seen.data_ptr<int64_t>(), ws.at, ws.bytes, stream_now(dev));
    });
    return pair(pos, seen);
  });
}

// kv4_tree_attention(cache, q, table, lens, cu, pos, seen, max_new, cos, sin, interleaved, gq, window, softmax_scale, eps, workspace)
PyObject* kv4_tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 16) Py_RETURN_NONE;
  return guarded("swa_kv4_tree_attn", [&](Call& call) -> PyObject* {
    const int dev = device_now();
    const CacheDims c = cache_of(a[0], dev);
    const at::Tensor &q = tensor(a[1]), &table = tensor(a[2]);
    if (q.dim() != 3 || q.numel() == 0 || table.dim() != 2 || a[15] == Py_None) throw Refused{};
    const auto type = q.scalar_type();
    const int kind = kind_more(type);
    const int64_t N = q.size(0), Hq = q.size(1), B = table.size(0), width = table.size(1);
    const void* qa = at_(a[1], type, dev, {N, Hq, c.d});
    const auto* ta = static_cast<const int32_t*>(at_(a[2], at::kInt, dev, {B, width}));
    const auto* la = static_cast<const int32_t*>(at_(a[3], at::kInt, dev, {B}));
    const auto* ca = static_cast<const int32_t*>(at_(a[4], at::kInt, dev, {B + 1}));
    const auto* pa = static_cast<const int32_t*>(at_(a[5], at::kInt, dev, {N}));
    const auto* sa = static_cast<const int64_t*>(at_(a[6], at::kLong, dev, {N}));
    const int most = int_of(a[7]);
    swa_rope r{};
    const bool rope = rope_of(a[8], a[9], a[10], dev, r);
    const auto* gq = static_cast<const float*>(at_(a[11], at::kFloat, dev, {c.d}));
    const Ws ws = ws_of(a[15], dev);
    const swa_params p{small(B), 1, small(Hq), c.Hkv, c.d, int_of(a[12]), 1, static_cast<float>(double_of(a[13])),
                       static_cast<float>(double_of(a[14])), 0.f, 0};
    const int max_pages = small(width), rows = small(N);
    at::Tensor o, lse;
    call([&] {
      o = at::empty_like(q);
      lse = at::empty({N, Hq}, on(dev, at::kFloat));
      return more[kind].tree_attn(&p, nullptr, &c.c, rope ? &r : nullptr, rows, most, qa, gq, ta, max_pages, la, ca, pa, sa, o.data_ptr(),
                                  lse.data_ptr<float>(), ws.at, ws.bytes, stream_now(dev));
    });
    return pair(o, lse);
  });
}

// kv4_move(cache, src, dst, workspace)
PyObject* kv4_move(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4 || more[0].move == nullptr) Py_RETURN_NONE;
  return guarded("swa_kv4_move", [&](Call& call) -> PyObject* {
    const int dev = device_now();
    const CacheDims c = cache_of(a[0], dev);
    const at::Tensor& s = tensor(a[1]);
    if (s.dim() != 2) throw Refused{};
    const auto* sa = static_cast<const int64_t*>(at_(a[1], at::kLong, dev, s.sizes()));
    const auto* da = static_cast<const int64_t*>(at_(a[2], at::kLong, dev, s.sizes()));
    const Ws ws = ws_of(a[3], dev);
    const swa_params p{small(s.size(0)), small(s.size(1)), c.Hkv, c.Hkv, c.d, -1, 1, 0.f, 0.f, 0.f, 0};
    call([&] { return more[0].move(&p, &c.c, sa, da, ws.at, ws.bytes, stream_now(dev)); });
    Py_RETURN_TRUE;
  });
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),       FAST(raises),      FAST(rope_tables), FAST(rope_apply),    FAST(kv4_plan),
                         FAST(kv4_append), FAST(kv4_read),    FAST(kv4_attention), FAST(bind_more), FAST(rms_norm), FAST(rms_norm_backward), FAST(w4_linear),
                         FAST(kv4_tree),   FAST(kv4_tree_attention), FAST(kv4_move), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast() { return PyModule_Create(&module); }
