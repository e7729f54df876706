// bind.cpp -- CPython binding of the ragged appends, the windowed and tree attentions
// and the calls on 8-bit caches (include/vh.h) on torch tensors.
//
// These calls are small: a decode step's append or attention runs for a few
// microseconds, and reading a dozen tensors' shapes, strides and types from
// Python costs more than that.  So arguments are checked and taken apart here,
// against torch's C++ interface, and passed to the C functions as they are.
// Nothing is computed, copied or kept between calls.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>

#include "../../include/vh.h"

namespace {

struct Raised {};  // a Python exception is set

template <typename... A>
[[noreturn]] void raise(PyObject* type, const char* text, A... a) {
  PyErr_Format(type, text, a...);
  throw Raised{};
}

// Positional and keyword arguments of one function, by position.
struct Signature {
  const char* function;
  int required;
  const char* names[32];  // (string literals; an initializer_list's own array would not outlive the constructor)
  PyObject* interned[32];
  int n = 0;
  Signature(const char* f, std::initializer_list<const char*> ns, int req) : function(f), required(req) {
    for (const char* s : ns) {
      names[n] = s;
      interned[n++] = PyUnicode_InternFromString(s);
    }
  }
  const char* name(int i) const { return names[i]; }
  void parse(PyObject* const* args, Py_ssize_t nargs, PyObject* kw, PyObject** to) const {
    if (nargs > n) raise(PyExc_TypeError, "%s takes at most %d arguments", function, n);
    for (int i = 0; i < n; ++i) to[i] = i < nargs ? args[i] : nullptr;
    const Py_ssize_t nk = kw ? PyTuple_GET_SIZE(kw) : 0;
    for (Py_ssize_t k = 0; k < nk; ++k) {
      PyObject* key = PyTuple_GET_ITEM(kw, k);
      int i = 0;
      while (i < n && interned[i] != key) ++i;
      if (i == n)
        for (i = 0; i < n && PyUnicode_Compare(interned[i], key) != 0;) ++i;
      if (i == n) raise(PyExc_TypeError, "%s got an unexpected argument '%U'", function, key);
      if (to[i]) raise(PyExc_TypeError, "%s got two values for '%s'", function, name(i));
      to[i] = args[nargs + k];
    }
    for (int i = 0; i < required; ++i)
      if (!to[i]) raise(PyExc_TypeError, "%s needs the argument '%s'", function, name(i));
  }
};

bool given(PyObject* o) { return o && o != Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

long integer(PyObject* o, long dflt) {
  if (!o) return dflt;
  PyObject* i = PyNumber_Index(o);
  if (!i) throw Raised{};
  const long x = PyLong_AsLong(i);
  Py_DECREF(i);
  if (x == -1 && PyErr_Occurred()) throw Raised{};
  return x;
}

int integer32(PyObject* o, int dflt, const char* name) {
  const long x = integer(o, dflt);
  if (x < INT32_MIN || x > INT32_MAX) raise(PyExc_ValueError, "%s is out of range", name);
  return static_cast<int>(x);
}

float real(PyObject* o, float dflt) {
  if (!o) return dflt;
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised{};
  return static_cast<float>(x);
}

bool truth(PyObject* o) {
  if (!o) return false;
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw Raised{};
  return x != 0;
}

bool shape_is(const at::Tensor& t, std::initializer_list<int64_t> s) { return t.sizes().equals(at::IntArrayRef(s)); }

// The current device, which holds t: the launch goes there.
int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda() || t.get_device() != c10::cuda::current_device())
    raise(PyExc_ValueError, "%s must be a CUDA tensor on the current device", name);
  return static_cast<int>(t.get_device());
}

void* address(const at::Tensor& t, at::ScalarType type, int dev, const char* name, bool contiguous = true) {
  if (!t.is_cuda() || t.get_device() != dev)
    raise(PyExc_ValueError, "%s must be a CUDA tensor on the current device", name);
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
  if (contiguous && !t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
  return t.data_ptr();
}

void* address_or_null(PyObject* o, at::ScalarType type, int dev, const char* name) {
  return given(o) ? address(tensor(o, name), type, dev, name) : nullptr;
}

// A [NP, P, Hkv, D] view of the K and V caches with its page table.
struct Cache {
  at::ScalarType type;
  int P, Hkv, NP, per_row = 0;
  int64_t page, token, head;  // strides
  uint16_t *k = nullptr, *v = nullptr;
  const int32_t* table = nullptr;
  const char *k_name, *v_name;
  const at::Tensor &kt, &vt;
  Cache(PyObject* ko, PyObject* vo, int64_t D, bool eight = false, const char* kn = "k_cache", const char* vn = "v_cache")
      : k_name(kn), v_name(vn), kt(tensor(ko, kn)), vt(tensor(vo, vn)) {
    if (kt.dim() != 4 || vt.sizes() != kt.sizes() || vt.strides() != kt.strides())
      raise(PyExc_ValueError, "%s / %s must be [NP, P, Hkv, D] views with equal strides", kn, vn);
    if (kt.size(3) != D) raise(PyExc_ValueError, "shape mismatch: the head dims of the cache and of the queries differ");
    if (kt.stride(3) != 1) raise(PyExc_ValueError, "head_dim must be contiguous in the cache");
    if (kt.size(0) > INT32_MAX) raise(PyExc_ValueError, "too many pages");
    type = kt.scalar_type();
    if (eight ? type != at::kFloat8_e4m3fn : type != at::kBFloat16 && type != at::kHalf)
      raise(PyExc_TypeError, "%s must be %s, got %s", kn, eight ? "float8_e4m3fn" : "bfloat16 or float16", c10::toString(type));
    NP = static_cast<int>(kt.size(0));
    P = static_cast<int>(kt.size(1));
    Hkv = static_cast<int>(kt.size(2));
    // (torch gives a dimension of one element any stride)
    head = Hkv > 1 ? kt.stride(2) : D;
    token = P > 1 ? kt.stride(1) : Hkv * D;
    page = NP > 1 ? kt.stride(0) : static_cast<int64_t>(P) * Hkv * D;
  }
  void locate(PyObject* table_o, int B, int dev, const char* table_name = "page_table") {
    k = static_cast<uint16_t*>(address(kt, type, dev, k_name, false));
    v = static_cast<uint16_t*>(address(vt, type, dev, v_name, false));
    if (given(table_o)) {
      const at::Tensor& t = tensor(table_o, table_name);
      table = static_cast<const int32_t*>(address(t, at::kInt, dev, table_name));
      per_row = static_cast<int>(t.size(1));
    } else {
      if (B < 1 || NP % B) raise(PyExc_ValueError, "without a page table the cache must hold a whole number of pages per row");
      per_row = NP / B;
    }
  }
  unsigned flags() const { return type == at::kHalf ? VH_FLAG_FP16 : 0u; }
};

// The scales of an 8-bit cache: [NP, Hkv, P] views.
struct Scales {
  float *k = nullptr, *v = nullptr;
  int64_t page, head;  // strides
  const at::Tensor &kt, &vt;
  Scales(PyObject* ko, PyObject* vo, const Cache& c) : kt(tensor(ko, "k_scale")), vt(tensor(vo, "v_scale")) {
    if (!shape_is(kt, {c.NP, c.Hkv, c.P}) || vt.sizes() != kt.sizes() || vt.strides() != kt.strides() || (c.P > 1 && kt.stride(2) != 1))
      raise(PyExc_ValueError, "k_scale / v_scale must be [%d, %d, %d] views (pages, kv heads, slots) with equal strides and "
                              "contiguous slots", c.NP, c.Hkv, c.P);
    head = c.Hkv > 1 ? kt.stride(1) : (c.P + 3) / 4 * 4;
    page = c.NP > 1 ? kt.stride(0) : c.Hkv * head;
  }
  void locate(int dev) {
    k = static_cast<float*>(address(kt, at::kFloat, dev, "k_scale", false));
    v = static_cast<float*>(address(vt, at::kFloat, dev, "v_scale", false));
  }
};

// Rows of the batch; the arrays with one entry a row agree on it.
int rows_of(PyObject* lens, PyObject* active, PyObject* start, PyObject* table, const char* table_name = "page_table") {
  const at::Tensor& l = tensor(lens, "seq_lens");
  if (l.dim() != 1) raise(PyExc_ValueError, "seq_lens must be one-dimensional");
  const int64_t B = l.size(0);
  if (B > INT32_MAX - 1) raise(PyExc_ValueError, "too many rows");
  if (!shape_is(tensor(active, "active"), {B})) raise(PyExc_ValueError, "active must have shape (%lld,)", static_cast<long long>(B));
  if (given(start) && !shape_is(tensor(start, "token_start"), {B + 1}))
    raise(PyExc_ValueError, "token_start must have shape (%lld,)", static_cast<long long>(B + 1));
  if (given(table)) {
    const at::Tensor& t = tensor(table, table_name);
    if (t.dim() != 2 || t.size(0) != B || t.size(1) > INT32_MAX)
      raise(PyExc_ValueError, "%s must have shape (%lld, pages per row)", table_name, static_cast<long long>(B));
  }
  return static_cast<int>(B);
}

// Address and token stride of a [T, heads, D] tensor whose tokens may lie apart.
const uint16_t* tokens(const at::Tensor& t, at::ScalarType type, int dev, const char* name, int64_t* stride) {
  const int64_t heads = t.size(1), D = t.size(2);
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != D))
    raise(PyExc_ValueError, "the heads of one token of %s must be contiguous", name);
  *stride = t.size(0) > 1 ? t.stride(0) : heads * D;
  return static_cast<const uint16_t*>(address(t, type, dev, name, false));
}

void* stream_of(PyObject* o, int dev) {
  if (!given(o)) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  PyObject* s = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : PyNumber_Index(o);
  if (!s) throw Raised{};
  void* p = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  if (!p && PyErr_Occurred()) throw Raised{};
  return p;
}

PyObject* done(int status, const char* where, PyObject* result) {
  if (status == VH_OK) {
    Py_INCREF(result);
    return result;
  }
  PyObject* mod = PyImport_ImportModule("paged_len_decode_gb300");
  PyObject* cls = mod ? PyObject_GetAttrString(mod, "VHError") : nullptr;
  PyObject* e = cls ? PyObject_CallFunction(cls, "is", status, where) : nullptr;
  if (e) PyErr_SetObject(cls, e);
  Py_XDECREF(e);
  Py_XDECREF(cls);
  Py_XDECREF(mod);
  return nullptr;
}

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

int32_t* ints(void* p) { return static_cast<int32_t*>(p); }

// A call of a C function without Python's lock: a launch waits where the device's
// queue is full, and other threads go on meanwhile.  (The caller holds the
// arguments' tensors.  All that touches Python is done before.)
template <typename F>
int without_lock(F f) {
  PyThreadState* t = PyEval_SaveThread();
  const int status = f();
  PyEval_RestoreThread(t);
  return status;
}

// Both appends: EIGHT, into a cache of 8 bits, whose scales follow it in the argument list.
template <bool EIGHT>
PyObject* kv_append(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    enum { Q, K, V, CS, KC, VC, TABLE, LENS, ACTIVE, QROT, START, POS, AXIS, ERR, QW, KW, EPS, ILV, STREAM, COUNT };
    static const Signature sig = EIGHT ? Signature("vh_quant_kv_append",
                                                   {"q", "k_new", "v_new", "cos_sin", "k_cache", "v_cache", "k_scale", "v_scale",
                                                    "page_table", "seq_lens", "active", "q_rot", "token_start", "positions",
                                                    "pair_axis", "err_flag", "q_norm_w", "k_norm_w", "norm_eps", "interleaved",
                                                    "stream"},
                                                   QROT + 3)
                                       : Signature("vh_mrope_kv_append",
                                                   {"q", "k_new", "v_new", "cos_sin", "k_cache", "v_cache", "page_table",
                                                    "seq_lens", "active", "q_rot", "token_start", "positions", "pair_axis",
                                                    "err_flag", "q_norm_w", "k_norm_w", "norm_eps", "interleaved", "stream"},
                                                   QROT + 1);
    PyObject *given_args[COUNT + 2], **a = given_args, *scales[2] = {};
    sig.parse(args, nargs, kw, given_args);
    if (EIGHT) {
      scales[0] = given_args[TABLE];
      scales[1] = given_args[TABLE + 1];
      for (int i = TABLE; i < COUNT; ++i) a[i] = given_args[i + 2];
    }
    const at::Tensor &q = tensor(a[Q], "q"), &kn = tensor(a[K], "k_new"), &vn = tensor(a[V], "v_new"),
                     &cs = tensor(a[CS], "cos_sin"), &rot = tensor(a[QROT], "q_rot");
    if (q.dim() != 3) raise(PyExc_ValueError, "q must have shape [T, Hq, D]");
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
    Cache c(a[KC], a[VC], D, EIGHT);
    const at::ScalarType type = EIGHT ? q.scalar_type() : c.type;  // of q, k_new and v_new
    if (EIGHT && type != at::kBFloat16 && type != at::kHalf)
      raise(PyExc_TypeError, "q must be bfloat16 or float16, got %s", c10::toString(type));
    if (T > INT32_MAX || rot.sizes() != q.sizes() || !shape_is(kn, {T, c.Hkv, D}) || !shape_is(vn, {T, c.Hkv, D}))
      raise(PyExc_ValueError, "shape mismatch between q, k_new, v_new, q_rot and the cache");
    if (cs.dim() != 2 || cs.size(1) != D || cs.size(0) > INT32_MAX)
      raise(PyExc_ValueError, "cos_sin must have shape [max_pos, %lld]", static_cast<long long>(D));
    const int B = rows_of(a[LENS], a[ACTIVE], a[START], a[TABLE]);
    int axes = 1;
    if (given(a[POS])) {
      const at::Tensor& p = tensor(a[POS], "positions");
      if (p.dim() == 2 ? (p.size(1) != T || p.size(0) > 255) : !shape_is(p, {T}))
        raise(PyExc_ValueError, "positions must have shape (T,) or (axes, T), with T = %lld", static_cast<long long>(T));
      if (p.dim() == 2) axes = static_cast<int>(p.size(0));
    }
    uint8_t axis[512];
    if (given(a[AXIS])) {
      PyObject* s = PySequence_Fast(a[AXIS], "pair_axis must be a sequence of integers");
      if (!s) throw Raised{};
      const Py_ssize_t n = PySequence_Fast_GET_SIZE(s);
      bool ok = n == D / 2 && n <= 512;
      int top = 0;
      for (Py_ssize_t i = 0; ok && i < n; ++i) {
        const long x = PyLong_AsLong(PySequence_Fast_GET_ITEM(s, i));
        ok = x >= 0 && x < 4;
        axis[i] = static_cast<uint8_t>(x & 3);
        if (x > top) top = static_cast<int>(x);
      }
      Py_DECREF(s);
      if (PyErr_Occurred()) throw Raised{};
      if (!given(a[POS])) axes = top + 1;
      if (!ok || top >= axes)
        raise(PyExc_ValueError, "pair_axis must hold an axis of positions for each of the %lld pairs", static_cast<long long>(D / 2));
    }
    for (int i : {QW, KW}) {
      const char* name = i == QW ? "q_norm_w" : "k_norm_w";
      if (given(a[i]) && !shape_is(tensor(a[i], name), {D}))
        raise(PyExc_ValueError, "%s must have shape (%lld,)", name, static_cast<long long>(D));
    }
    const int dev = device_of(q, "q");
    c.locate(a[TABLE], B, dev);
    if (rot.scalar_type() != at::kFloat && rot.scalar_type() != type)
      raise(PyExc_TypeError, "q_rot must be float32 or %s type, got %s", EIGHT ? "q's" : "the cache's", c10::toString(rot.scalar_type()));
    int64_t qs, ks, vs;
    const uint16_t *qp = tokens(q, type, dev, "q", &qs), *kp = tokens(kn, type, dev, "k_new", &ks),
                   *vp = tokens(vn, type, dev, "v_new", &vs);
    const unsigned flags = (type == at::kHalf ? VH_FLAG_FP16 : 0u) | (truth(a[ILV]) ? VH_FLAG_ROPE_INTERLEAVED : 0u) |
                           (rot.scalar_type() == type ? VH_FLAG_Q16 : 0u);
    const float* angles = static_cast<const float*>(address(cs, at::kFloat, dev, "cos_sin"));
    const int32_t *pos = ints(address_or_null(a[POS], at::kInt, dev, "positions")),
                  *start = ints(address_or_null(a[START], at::kInt, dev, "token_start")),
                  *lens = ints(address(tensor(a[LENS], "seq_lens"), at::kInt, dev, "seq_lens")),
                  *active = ints(address(tensor(a[ACTIVE], "active"), at::kInt, dev, "active"));
    const float *qw = static_cast<const float*>(address_or_null(a[QW], at::kFloat, dev, "q_norm_w")),
                *kw_ = static_cast<const float*>(address_or_null(a[KW], at::kFloat, dev, "k_norm_w"));
    const float eps = real(a[EPS], 1e-6f);
    void *to = address(rot, rot.scalar_type(), dev, "q_rot"), *stream = stream_of(a[STREAM], dev);
    int32_t* err = ints(address_or_null(a[ERR], at::kInt, dev, "err_flag"));
    const uint8_t* pair_axis = given(a[AXIS]) ? axis : nullptr;
    const int max_pos = static_cast<int>(cs.size(0));
    if constexpr (EIGHT) {
      Scales s(scales[0], scales[1], c);
      s.locate(dev);
      const int st = without_lock([&] {
        return vh_quant_kv_append(qp, kp, vp, qs, ks, vs, angles, max_pos, pos, pair_axis, axes, qw, kw_, eps,
                                  reinterpret_cast<vh_e4m3*>(c.k), reinterpret_cast<vh_e4m3*>(c.v), c.page, c.token, c.head, s.k,
                                  s.v, s.page, s.head, c.NP, c.table, c.per_row, start, lens, active, to, err, flags,
                                  static_cast<int>(T), B, static_cast<int>(Hq), c.Hkv, static_cast<int>(D), c.P, stream);
      });
      return done(st, sig.function, a[QROT]);
    }
    const int st = without_lock([&] {
      return vh_mrope_kv_append(qp, kp, vp, qs, ks, vs, angles, max_pos, pos, pair_axis, axes, qw, kw_, eps, c.k, c.v, c.page,
                                c.token, c.head, c.NP, c.table, c.per_row, start, lens, active, to, err, flags,
                                static_cast<int>(T), B, static_cast<int>(Hq), c.Hkv, static_cast<int>(D), c.P, stream);
    });
    return done(st, sig.function, a[QROT]);
  });
}

PyObject* window_decode_attn(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    enum { Q, KC, VC, TABLE, LENS, ACTIVE, OUT, WS, WINDOW, SINKS, SCALE, CTAS, ERR, PDL, STREAM, COUNT };
    static const Signature sig("vh_window_decode_attn",
                               {"q_rot", "k_cache", "v_cache", "page_table", "seq_lens", "active", "out", "workspace",
                                "window", "sinks", "sm_scale", "num_ctas", "err_flag", "pdl", "stream"},
                               WS + 1);
    PyObject* a[COUNT];
    sig.parse(args, nargs, kw, a);
    const at::Tensor &q = tensor(a[Q], "q_rot"), &out = tensor(a[OUT], "out"), &ws = tensor(a[WS], "workspace");
    if (q.dim() != 3 || out.sizes() != q.sizes())
      raise(PyExc_ValueError, "shape mismatch: q_rot and out must both have shape [B, Hq, D]");
    const int64_t Hq = q.size(1), D = q.size(2);
    Cache c(a[KC], a[VC], D);
    const int B = rows_of(a[LENS], a[ACTIVE], nullptr, a[TABLE]);
    if (q.size(0) != B) raise(PyExc_ValueError, "shape mismatch: q_rot has %lld rows, seq_lens %d", static_cast<long long>(q.size(0)), B);
    const int dev = device_of(q, "q_rot");
    c.locate(a[TABLE], B, dev);
    const float* qp = static_cast<const float*>(address(q, at::kFloat, dev, "q_rot"));
    const int32_t *lens = ints(address(tensor(a[LENS], "seq_lens"), at::kInt, dev, "seq_lens")),
                  *active = ints(address(tensor(a[ACTIVE], "active"), at::kInt, dev, "active"));
    const int window = integer32(a[WINDOW], 0, "window"), sinks = integer32(a[SINKS], 0, "sinks"),
              ctas = integer32(a[CTAS], 0, "num_ctas");
    uint16_t* to = static_cast<uint16_t*>(address(out, c.type, dev, "out"));
    const float scale = real(a[SCALE], 0.f);
    void *work = address(ws, ws.scalar_type(), dev, "workspace"), *stream = stream_of(a[STREAM], dev);
    const size_t bytes = ws.nbytes();
    int32_t* err = ints(address_or_null(a[ERR], at::kInt, dev, "err_flag"));
    const unsigned flags = c.flags() | (truth(a[PDL]) ? VH_FLAG_PDL : 0u);
    const int st = without_lock([&] {
      return vh_window_decode_attn(qp, c.k, c.v, c.page, c.token, c.head, c.NP, c.table, c.per_row, lens, active, window, sinks,
                                   to, scale, ctas, work, bytes, err, flags, B, static_cast<int>(Hq), c.Hkv,
                                   static_cast<int>(D), c.P, stream);
    });
    return done(st, sig.function, a[OUT]);
  });
}

PyObject* quant_decode_attn(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    enum { Q, KC, VC, KS, VS, TABLE, LENS, ACTIVE, OUT, WS, WINDOW, SINKS, SCALE, CTAS, ERR, PDL, STREAM, COUNT };
    static const Signature sig("vh_quant_decode_attn",
                               {"q_rot", "k_cache", "v_cache", "k_scale", "v_scale", "page_table", "seq_lens", "active", "out",
                                "workspace", "window", "sinks", "sm_scale", "num_ctas", "err_flag", "pdl", "stream"},
                               WS + 1);
    PyObject* a[COUNT];
    sig.parse(args, nargs, kw, a);
    const at::Tensor &q = tensor(a[Q], "q_rot"), &out = tensor(a[OUT], "out"), &ws = tensor(a[WS], "workspace");
    if (q.dim() != 3 || out.sizes() != q.sizes())
      raise(PyExc_ValueError, "shape mismatch: q_rot and out must both have shape [B, Hq, D]");
    const int64_t Hq = q.size(1), D = q.size(2);
    Cache c(a[KC], a[VC], D, true);
    Scales s(a[KS], a[VS], c);
    const int B = rows_of(a[LENS], a[ACTIVE], nullptr, a[TABLE]);
    if (q.size(0) != B) raise(PyExc_ValueError, "shape mismatch: q_rot has %lld rows, seq_lens %d", static_cast<long long>(q.size(0)), B);
    if (out.scalar_type() != at::kBFloat16 && out.scalar_type() != at::kHalf)
      raise(PyExc_TypeError, "out must be bfloat16 or float16, got %s", c10::toString(out.scalar_type()));
    const int dev = device_of(q, "q_rot");
    c.locate(a[TABLE], B, dev);
    s.locate(dev);
    const float* qp = static_cast<const float*>(address(q, at::kFloat, dev, "q_rot"));
    const int32_t *lens = ints(address(tensor(a[LENS], "seq_lens"), at::kInt, dev, "seq_lens")),
                  *active = ints(address(tensor(a[ACTIVE], "active"), at::kInt, dev, "active"));
    const int window = integer32(a[WINDOW], 0, "window"), sinks = integer32(a[SINKS], 0, "sinks"),
              ctas = integer32(a[CTAS], 0, "num_ctas");
    uint16_t* to = static_cast<uint16_t*>(address(out, out.scalar_type(), dev, "out"));
    const float scale = real(a[SCALE], 0.f);
    void *work = address(ws, ws.scalar_type(), dev, "workspace"), *stream = stream_of(a[STREAM], dev);
    const size_t bytes = ws.nbytes();
    int32_t* err = ints(address_or_null(a[ERR], at::kInt, dev, "err_flag"));
    const unsigned flags = (out.scalar_type() == at::kHalf ? VH_FLAG_FP16 : 0u) | (truth(a[PDL]) ? VH_FLAG_PDL : 0u);
    const int st = without_lock([&] {
      return vh_quant_decode_attn(qp, reinterpret_cast<vh_e4m3*>(c.k), reinterpret_cast<vh_e4m3*>(c.v), c.page, c.token, c.head,
                                  s.k, s.v, s.page, s.head, c.NP, c.table, c.per_row, lens, active, window, sinks, to, scale,
                                  ctas, work, bytes, err, flags, B, static_cast<int>(Hq), c.Hkv, static_cast<int>(D), c.P, stream);
    });
    return done(st, sig.function, a[OUT]);
  });
}

PyObject* quant_kv_read(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    enum { KC, VC, KS, VS, TABLE, LENS, ACTIVE, KOUT, VOUT, OUT_TABLE, FIRST, SINKS, ERR, STREAM, COUNT };
    static const Signature sig("vh_quant_kv_read",
                               {"k_cache", "v_cache", "k_scale", "v_scale", "page_table", "seq_lens", "active", "k_out", "v_out",
                                "out_page_table", "first_slot", "sinks", "err_flag", "stream"},
                               OUT_TABLE + 1);
    PyObject* a[COUNT];
    sig.parse(args, nargs, kw, a);
    const at::Tensor& kt = tensor(a[KC], "k_cache");
    if (kt.dim() != 4) raise(PyExc_ValueError, "k_cache / v_cache must be [NP, P, Hkv, D] views with equal strides");
    const int64_t D = kt.size(3);
    Cache c(a[KC], a[VC], D, true), o(a[KOUT], a[VOUT], D, false, "k_out", "v_out");
    Scales s(a[KS], a[VS], c);
    if (o.Hkv != c.Hkv) raise(PyExc_ValueError, "shape mismatch: the kv heads of the two caches differ");
    const int B = rows_of(a[LENS], a[ACTIVE], nullptr, a[TABLE]);
    rows_of(a[LENS], a[ACTIVE], nullptr, a[OUT_TABLE], "out_page_table");
    if (given(a[FIRST]) && !shape_is(tensor(a[FIRST], "first_slot"), {B})) raise(PyExc_ValueError, "first_slot must have shape (%d,)", B);
    const int dev = device_of(kt, "k_cache");
    c.locate(a[TABLE], B, dev);
    o.locate(a[OUT_TABLE], B, dev, "out_page_table");
    s.locate(dev);
    const int32_t *lens = ints(address(tensor(a[LENS], "seq_lens"), at::kInt, dev, "seq_lens")),
                  *active = ints(address(tensor(a[ACTIVE], "active"), at::kInt, dev, "active")),
                  *first = ints(address_or_null(a[FIRST], at::kInt, dev, "first_slot"));
    const int sinks = integer32(a[SINKS], 0, "sinks");
    int32_t* err = ints(address_or_null(a[ERR], at::kInt, dev, "err_flag"));
    void* stream = stream_of(a[STREAM], dev);
    const int st = without_lock([&] {
      return vh_quant_kv_read(reinterpret_cast<vh_e4m3*>(c.k), reinterpret_cast<vh_e4m3*>(c.v), c.page, c.token, c.head, s.k, s.v,
                              s.page, s.head, c.NP, c.table, c.per_row, lens, active, first, sinks, o.k, o.v, o.page, o.token,
                              o.head, o.NP, o.table, o.per_row, err, o.flags(), B, c.Hkv, static_cast<int>(D), c.P, o.P, stream);
    });
    return done(st, sig.function, Py_None);
  });
}

// Both attentions of ragged batches: TREE, of drafted tokens, whose masks follow `active` in the argument list.
template <bool TREE>
PyObject* ragged_attn(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kw) {
  return guarded([&]() -> PyObject* {
    enum { Q, KC, VC, TABLE, START, LENS, ACTIVE, OUT, WS, WINDOW, SINKS, SCALE, SPLITS, ERR, STREAM, COUNT };
    static const Signature sig = TREE ? Signature("vh_tree_attn",
                                                  {"q", "k_cache", "v_cache", "page_table", "token_start", "seq_lens", "active",
                                                   "tree_mask", "out", "workspace", "window", "sinks", "sm_scale", "num_splits",
                                                   "err_flag", "stream"},
                                                  WS + 2)
                                      : Signature("vh_window_prompt_attn",
                                                  {"q", "k_cache", "v_cache", "page_table", "token_start", "seq_lens", "active",
                                                   "out", "workspace", "window", "sinks", "sm_scale", "num_splits", "err_flag",
                                                   "stream"},
                                                  WS + 1);
    PyObject *given_args[COUNT + 1], **a = given_args, *mask = nullptr;
    sig.parse(args, nargs, kw, given_args);
    if (TREE) {
      mask = given_args[OUT];
      for (int i = OUT; i < COUNT; ++i) a[i] = given_args[i + 1];
    }
    const at::Tensor &q = tensor(a[Q], "q"), &out = tensor(a[OUT], "out"), &ws = tensor(a[WS], "workspace");
    if (q.dim() != 3 || q.size(0) > INT32_MAX || out.sizes() != q.sizes())
      raise(PyExc_ValueError, "shape mismatch: q and out must both have shape [T, Hq, D]");
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
    Cache c(a[KC], a[VC], D);
    const int B = rows_of(a[LENS], a[ACTIVE], a[START], a[TABLE]);
    const int dev = device_of(q, "q");
    c.locate(a[TABLE], B, dev);
    const uint16_t* qp = static_cast<const uint16_t*>(address(q, c.type, dev, "q"));
    const int32_t *start = ints(address(tensor(a[START], "token_start"), at::kInt, dev, "token_start")),
                  *lens = ints(address(tensor(a[LENS], "seq_lens"), at::kInt, dev, "seq_lens")),
                  *active = ints(address(tensor(a[ACTIVE], "active"), at::kInt, dev, "active"));
    const int window = integer32(a[WINDOW], 0, "window"), sinks = integer32(a[SINKS], 0, "sinks"),
              splits = integer32(a[SPLITS], 0, "num_splits");
    uint16_t* to = static_cast<uint16_t*>(address(out, c.type, dev, "out"));
    const float scale = real(a[SCALE], 0.f);
    void *work = address(ws, ws.scalar_type(), dev, "workspace"), *stream = stream_of(a[STREAM], dev);
    const size_t bytes = ws.nbytes();
    int32_t* err = ints(address_or_null(a[ERR], at::kInt, dev, "err_flag"));
    if constexpr (TREE) {
      const at::Tensor& m = tensor(mask, "tree_mask");
      if (m.dim() != 2 || m.size(0) != T || m.size(1) < 1 || m.size(1) > VH_TREE_WORDS_MAX)
        raise(PyExc_ValueError, "tree_mask must have shape (%lld, words), with 1 to %d words", static_cast<long long>(T), VH_TREE_WORDS_MAX);
      const int64_t* bits = static_cast<const int64_t*>(address(m, at::kLong, dev, "tree_mask"));
      const int words = static_cast<int>(m.size(1));
      const int st = without_lock([&] {
        return vh_tree_attn(qp, c.k, c.v, c.page, c.token, c.head, c.NP, c.table, c.per_row, start, lens, active, bits, words,
                            window, sinks, to, scale, splits, work, bytes, err, c.flags(), static_cast<int>(T), B,
                            static_cast<int>(Hq), c.Hkv, static_cast<int>(D), c.P, stream);
      });
      return done(st, sig.function, a[OUT]);
    }
    const int st = without_lock([&] {
      return vh_window_prompt_attn(qp, c.k, c.v, c.page, c.token, c.head, c.NP, c.table, c.per_row, start, lens, active, window,
                                   sinks, to, scale, splits, work, bytes, err, c.flags(), static_cast<int>(T), B,
                                   static_cast<int>(Hq), c.Hkv, static_cast<int>(D), c.P, stream);
    });
    return done(st, sig.function, a[OUT]);
  });
}

#define VH_METHOD(name, f, doc) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL | METH_KEYWORDS, doc}

PyMethodDef g_methods[] = {
    VH_METHOD("vh_mrope_kv_append", kv_append<false>,
              "vh_mrope_kv_append(q, k_new, v_new, cos_sin, k_cache, v_cache, page_table, seq_lens, active, q_rot, "
              "token_start=None, positions=None, pair_axis=None, err_flag=None, q_norm_w=None, k_norm_w=None, "
              "norm_eps=1e-6, interleaved=False, stream=None)\n--\n\n"
              "RoPE with several axes of positions and KV append for T ragged tokens.\n"
              "q [T, Hq, D], k_new, v_new [T, Hkv, D]: the tokens may lie apart (slices of a\n"
              "packed projection).  token_start int32 [B + 1], or None: one token a row.\n"
              "positions int32 [T] or [axes, T], or None (the slot); pair_axis: the axis of\n"
              "each of the D/2 pairs (see mrope_pair_axis), or None (axis 0).  q_rot\n"
              "[T, Hq, D] is float32, or the cache's type (VH_FLAG_Q16).  Returns q_rot."),
    VH_METHOD("vh_window_decode_attn", window_decode_attn,
              "vh_window_decode_attn(q_rot, k_cache, v_cache, page_table, seq_lens, active, out, workspace, window=0, "
              "sinks=0, sm_scale=0.0, num_ctas=0, err_flag=None, pdl=False, stream=None)\n--\n\n"
              "Attention of one new token a row (q_rot float32 [B, Hq, D]) over the last\n"
              "`window` cached tokens (0: all) and the first `sinks`, in one launch.\n"
              "`workspace`: from alloc_workspace (zero-filled before its first use).  Returns out."),
    VH_METHOD("vh_window_prompt_attn", ragged_attn<false>,
              "vh_window_prompt_attn(q, k_cache, v_cache, page_table, token_start, seq_lens, active, out, workspace, "
              "window=0, sinks=0, sm_scale=0.0, num_splits=0, err_flag=None, stream=None)\n--\n\n"
              "Attention of T ragged new tokens (q [T, Hq, D] of the cache's type, already\n"
              "rotated) over the cache, which holds their keys and values: each sees the last\n"
              "`window` tokens up to itself (0: all) and the first `sinks`.  `workspace`:\n"
              "from alloc_prompt_workspace.  Returns out."),
    VH_METHOD("vh_tree_attn", ragged_attn<true>,
              "vh_tree_attn(q, k_cache, v_cache, page_table, token_start, seq_lens, active, tree_mask, out, workspace, "
              "window=0, sinks=0, sm_scale=0.0, num_splits=0, err_flag=None, stream=None)\n--\n\n"
              "vh_window_prompt_attn for drafted tokens that form a tree: a token sees the\n"
              "context and, of its row's drafted tokens, its ancestors and itself.  tree_mask\n"
              "int64 [T, words]: bit k % 64 of word k / 64 says that the row's k-th drafted\n"
              "token is an ancestor (see tree_masks).  A window counts back from the context's\n"
              "length plus the number of ancestors, and hides slots of the context only: where a\n"
              "tree has more levels than that, give tree_masks the window too.  Returns out."),
    VH_METHOD("vh_quant_kv_append", kv_append<true>,
              "vh_quant_kv_append(q, k_new, v_new, cos_sin, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, "
              "active, q_rot, token_start=None, positions=None, pair_axis=None, err_flag=None, q_norm_w=None, "
              "k_norm_w=None, norm_eps=1e-6, interleaved=False, stream=None)\n--\n\n"
              "vh_mrope_kv_append into a cache of 8 bits: k_cache, v_cache float8_e4m3fn\n"
              "[NP, P, Hkv, D] views, k_scale, v_scale float32 [NP, Hkv, P] views (see\n"
              "alloc_quant_cache).  q_rot is float32 or q's type.  Returns q_rot."),
    VH_METHOD("vh_quant_decode_attn", quant_decode_attn,
              "vh_quant_decode_attn(q_rot, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, active, out, "
              "workspace, window=0, sinks=0, sm_scale=0.0, num_ctas=0, err_flag=None, pdl=False, stream=None)\n--\n\n"
              "vh_window_decode_attn over a cache of 8 bits.  out is bfloat16 or float16.\n"
              "`workspace`: from alloc_workspace (zero-filled before its first use).  Returns out."),
    VH_METHOD("vh_quant_kv_read", quant_kv_read,
              "vh_quant_kv_read(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, active, k_out, v_out, "
              "out_page_table, first_slot=None, sinks=0, err_flag=None, stream=None)\n--\n\n"
              "Slots first_slot[b] (int32 [B], None: 0) to seq_lens[b] - 1 and those below\n"
              "`sinks` of a cache of 8 bits, read back into the same slots of a 16-bit cache\n"
              "k_out, v_out [NP2, P2, Hkv, D] with its own page table (None: contiguous)."),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_vh_bind", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__vh_bind(void) { return PyModule_Create(&g_module); }
