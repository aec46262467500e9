// The allocating calls of the operators around the recurrent layer, from tensors to the C
// ABI: what the Python wrappers of the other operators do (shapes, types and devices
// checked, outputs and workspaces allocated on the inputs' device, that device's current
// stream), compiled.  These calls' kernels often take 3 to 20 us, less than Python
// takes to check and allocate for them.  Host time of a call, in Python and here: a gated
// step 14.7 and 3.9 us, the recurrence's gradients 32.9 and 13.3, a norm 18.0 and 6.7, its
// gradients 25.9 and 9.9, rotary positions 18.2 and 5.2.
//
// The Python functions of the same names hold the documentation, the argument names and
// the defaults, and pass every argument by position.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/DeviceGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <optional>
#include <string>

#include "linattn.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

PyObject* g_error;  // LinAttnError(code, where)

// ---------------------------------------------------------------- refusals

struct Refused {
  PyObject* type;
  std::string what;
};

[[noreturn]] void value_error(const std::string& s) { throw Refused{PyExc_ValueError, s}; }
[[noreturn]] void type_error(const std::string& s) { throw Refused{PyExc_TypeError, s}; }
struct Raised {};  // a Python exception is set

std::string text(IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
  return s + (shape.size() == 1 ? ",)" : ")");
}
const char* text(ScalarType t) {
  switch (t) {
    case ScalarType::Float: return "torch.float32";
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Half: return "torch.float16";
    case ScalarType::Double: return "torch.float64";
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Long: return "torch.int64";
    default: return c10::toString(t);
  }
}

// ---------------------------------------------------------------- arguments

bool none(PyObject* o) { return o == Py_None; }

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + ": a tensor is needed");
  return THPVariable_Unpack(o);
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
long whole(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

// The interface's sizes and strides are integers of 32 bits.
int size(int64_t n) {
  if (n > INT_MAX) value_error("sizes above " + std::to_string(INT_MAX));
  return static_cast<int>(n);
}

la_dtype code_of(const Tensor& t) {
  if (t.scalar_type() == ScalarType::Float) return LA_F32;
  if (t.scalar_type() == ScalarType::BFloat16) return LA_BF16;
  type_error(std::string("unsupported dtype ") + text(t.scalar_type()) + ": use float32 or bfloat16");
}
int format_of(const Tensor& t) {
  if (t.scalar_type() == ScalarType::Char) return LA_CODE_I8;
  if (t.scalar_type() == ScalarType::Float8_e4m3fn) return LA_CODE_E4M3;
  type_error(std::string("unsupported code ") + text(t.scalar_type()) + ": use int8 or float8_e4m3fn");
}

void like(const Tensor& t, const char* name, IntArrayRef shape, ScalarType type, c10::Device dev) {
  const std::string n = name;
  if (t.sizes() != shape) value_error(n + ": shape " + text(t.sizes()) + ", the call needs " + text(shape));
  if (t.scalar_type() != type) type_error(n + ": " + text(t.scalar_type()) + ", the call needs " + text(type));
  if (t.device() != dev) value_error(n + ": on " + t.device().str() + ", the call is on " + dev.str());
}

// The address of a dense tensor of the shape, type and device that the call needs.
void* dense(PyObject* o, const char* name, IntArrayRef shape, ScalarType type, c10::Device dev) {
  const Tensor& t = tensor(o, name);
  like(t, name, shape, type, dev);
  if (!t.is_contiguous()) value_error(std::string(name) + ": must be contiguous");
  return t.data_ptr();
}
void* dense_or_none(PyObject* o, const char* name, IntArrayRef shape, ScalarType type, c10::Device dev) {
  return none(o) ? nullptr : dense(o, name, shape, type, dev);
}

struct Strided {
  void* p;
  int ld;
};

// A token-major view whose first `lead` dimensions are batch (and row): rows dense, and all
// rows of all batch entries evenly spaced.
Strided strided(PyObject* o, const char* name, IntArrayRef shape, ScalarType type, c10::Device dev, int lead) {
  const Tensor& t = tensor(o, name);
  like(t, name, shape, type, dev);
  const IntArrayRef st = t.strides();
  const std::string n = name;
  int64_t want = shape.back();
  if (want != 1 && st.back() != 1) value_error(n + ": every row must be dense");
  if (static_cast<int>(shape.size()) == lead + 2) {
    if (shape[lead] != 1 && st[lead] != want) value_error(n + ": every row must be dense");
    want *= shape[lead];
  }
  const int64_t B = shape[0];
  int64_t ld;
  if (lead == 1) {
    ld = B > 1 ? st[0] : want;
  } else {
    const int64_t N = shape[1];
    ld = N > 1 ? st[1] : B > 1 ? st[0] : want;
    if (B > 1 && st[0] != N * ld) value_error(n + ": batch entries must be N rows apart");
  }
  if (ld > INT_MAX) value_error(n + ": rows " + std::to_string(ld) + " elements apart, at most " + std::to_string(INT_MAX));
  return {t.data_ptr(), static_cast<int>(ld)};
}

// ---------------------------------------------------------------- the call itself

// The inputs' device, made the current one, and its current stream.
class On {
 public:
  explicit On(const Tensor& t) : dev_(t.device()) {
    if (!t.is_cuda()) value_error("tensors must be on a CUDA device");
    guard_.emplace(dev_);
    stream_ = c10::cuda::getCurrentCUDAStream(dev_.index()).stream();
  }
  void* stream() const { return stream_; }
  Tensor make(IntArrayRef shape, ScalarType type) const { return at::empty(shape, at::TensorOptions().dtype(type).device(dev_)); }

 private:
  c10::Device dev_;
  std::optional<c10::DeviceGuard> guard_;
  void* stream_;
};

// Workspace bytes on the device; none where none are needed.
struct Room {
  Tensor t;
  void* p = nullptr;
  size_t bytes;
  Room(const On& on, size_t n) : bytes(n) {
    if (n > 0) {
      t = on.make({static_cast<int64_t>(n)}, ScalarType::Byte);
      p = t.data_ptr();
    }
  }
};

template <typename... P, typename... A>
void call(la_status (*f)(P...), const char* where, A... args) {
  la_status rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = f(args...);
  Py_END_ALLOW_THREADS;
  if (rc == LA_OK) return;
  if (PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(rc), where)) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

PyObject* held(PyObject* o) {
  Py_INCREF(o);
  return o;
}
PyObject* out(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* out(PyObject* o) { return held(o); }
template <typename... T>
PyObject* tuple(const T&... v) {
  PyObject* r = PyTuple_New(sizeof...(v));
  if (r == nullptr) throw Raised{};
  Py_ssize_t i = 0;
  bool ok = true;
  auto set = [&](PyObject* o) {
    ok = ok && o != nullptr;
    PyTuple_SET_ITEM(r, i++, o);
  };
  (set(out(v)), ...);
  if (!ok) {
    Py_DECREF(r);
    throw Raised{};
  }
  return r;
}

// ---------------------------------------------------------------- gated recurrence

struct Gated {
  Strided x, r, i;
  void *lam, *lengths;
  IntArrayRef shape;
  int B, N, C;
  float scale;
  la_dtype code;
  ScalarType type;
  c10::Device dev;

  Gated(PyObject* const* a, PyObject* length, PyObject* by, int lead) : dev(c10::kCPU) {
    const Tensor& t = tensor(a[0], "x");
    if (t.dim() != lead + 1) value_error("x: " + std::to_string(lead + 1) + " dimensions");
    shape = t.sizes(), type = t.scalar_type(), dev = t.device();
    B = size(shape[0]), N = lead == 2 ? size(shape[1]) : 1, C = size(shape.back());
    const double v = real(by);
    if (!(v > 0 && std::isfinite(v))) value_error("scale: a positive number is needed");
    scale = static_cast<float>(v);
    code = code_of(t);
    x = strided(a[0], "x", shape, type, dev, lead);
    r = strided(a[1], "r", shape, type, dev, lead);
    i = strided(a[2], "i", shape, type, dev, lead);
    lam = dense(a[3], "lam", shape.slice(lead), type, dev);
    lengths = length == nullptr ? nullptr : dense_or_none(length, "lengths", shape.slice(0, 1), ScalarType::Int, dev);
  }
};

// x, r, i, lam, h, scale, lengths, keep
PyObject* gated_fwd(PyObject* const* a) {
  const Gated g(a, a[6], a[5], 2);
  void* h = dense_or_none(a[4], "h", {g.B, g.C}, ScalarType::Float, g.dev);
  const bool keep = truth(a[7]);
  const On on(tensor(a[0], "x"));
  const Tensor y = on.make(g.shape, g.type);
  Tensor kept;
  if (keep) kept = on.make({static_cast<int64_t>(la_gated_kept_bytes(g.B, g.N, g.C, g.code) / 4)}, ScalarType::Float);
  const Room ws(on, la_gated_workspace_bytes(0, g.B, g.N, g.C, g.code));
  call(la_gated_fwd, "la_gated_fwd", g.x.p, g.r.p, g.i.p, g.lam, static_cast<const int*>(g.lengths), static_cast<float*>(h),
       keep ? kept.data_ptr() : nullptr, y.data_ptr(), ws.p, ws.bytes, g.B, g.N, g.C, g.x.ld, g.r.ld, g.i.ld, g.scale, g.code, on.stream());
  return keep ? tuple(y, kept) : out(y);
}

// x, r, i, lam, kept, dy, scale, lengths
PyObject* gated_bwd(PyObject* const* a) {
  const Gated g(a, a[7], a[6], 2);
  void* kept = dense(a[4], "kept", {static_cast<int64_t>(la_gated_kept_bytes(g.B, g.N, g.C, g.code) / 4)}, ScalarType::Float, g.dev);
  void* dy = dense(a[5], "dy", g.shape, g.type, g.dev);
  const On on(tensor(a[0], "x"));
  const Tensor dx = on.make(g.shape, g.type), dr = on.make(g.shape, g.type), di = on.make(g.shape, g.type), dlam = on.make({g.C}, g.type);
  const Room ws(on, la_gated_workspace_bytes(1, g.B, g.N, g.C, g.code));
  call(la_gated_bwd, "la_gated_bwd", g.x.p, g.r.p, g.i.p, g.lam, static_cast<const int*>(g.lengths), kept, dy, dx.data_ptr(), dr.data_ptr(),
       di.data_ptr(), dlam.data_ptr(), ws.p, ws.bytes, g.B, g.N, g.C, g.x.ld, g.r.ld, g.i.ld, g.scale, g.code, on.stream());
  return tuple(dx, dr, di, dlam);
}

// x, r, i, lam, h, scale
PyObject* gated_step(PyObject* const* a) {
  const Gated g(a, nullptr, a[5], 1);
  void* h = dense(a[4], "h", {g.B, g.C}, ScalarType::Float, g.dev);
  const On on(tensor(a[0], "x"));
  const Tensor y = on.make(g.shape, g.type);
  call(la_gated_step, "la_gated_step", g.x.p, g.r.p, g.i.p, g.lam, static_cast<float*>(h), y.data_ptr(), g.B, g.C, g.x.ld, g.r.ld, g.i.ld,
       g.scale, g.code, on.stream());
  return out(y);
}

// ---------------------------------------------------------------- layer norm

struct Norm {
  Strided x;
  void* lengths;
  IntArrayRef shape;
  c10::SmallVector<int64_t, 3> stat;  // of a statistic: one value a group
  int B, N, C, G, lead;
  la_dtype code;
  ScalarType type;
  c10::Device dev;

  Norm(PyObject* o, const char* name, PyObject* groups, PyObject* length) : dev(c10::kCPU) {
    const Tensor& t = tensor(o, name);
    const std::string n = name;
    if (t.dim() != 2 && t.dim() != 3) value_error(n + ": 2 or 3 dimensions");
    lead = static_cast<int>(t.dim()) - 1, shape = t.sizes(), type = t.scalar_type(), dev = t.device();
    if (!none(length) && lead != 2) value_error("lengths: " + n + " must have 3 dimensions");
    const long g = whole(groups);
    if (g < 1 || shape.back() % g != 0)
      value_error("groups: " + std::to_string(g) + " does not divide " + std::to_string(shape.back()) + " columns");
    B = lead == 2 ? size(shape[0]) : 1, N = size(shape[lead - 1]), C = size(shape.back()), G = size(g);
    code = code_of(t);
    x = strided(o, name, shape, type, dev, lead);
    lengths = dense_or_none(length, "lengths", shape.slice(0, 1), ScalarType::Int, dev);
    stat.assign(shape.begin(), shape.end());
    stat.back() = g;
  }
};

// x, w, b, residual, groups, eps, lengths
PyObject* norm_fwd(PyObject* const* a) {
  const Norm n(a[0], "x", a[4], a[6]);
  const bool sum = !none(a[3]);
  const Strided res = sum ? strided(a[3], "residual", n.shape, n.type, n.dev, n.lead) : Strided{nullptr, n.C};
  void *w = dense(a[1], "w", {n.C}, n.type, n.dev), *b = dense_or_none(a[2], "b", {n.C}, n.type, n.dev);
  const float eps = static_cast<float>(real(a[5]));
  const On on(tensor(a[0], "x"));
  const Tensor y = on.make(n.shape, n.type), mean = on.make(n.stat, ScalarType::Float), rstd = on.make(n.stat, ScalarType::Float);
  Tensor s;
  if (sum) s = on.make(n.shape, n.type);
  call(la_norm_fwd, "la_norm_fwd", n.x.p, res.p, w, b, static_cast<const int*>(n.lengths), y.data_ptr(), sum ? s.data_ptr() : nullptr,
       mean.data_ptr<float>(), rstd.data_ptr<float>(), eps, n.B, n.N, n.C, n.G, n.x.ld, res.ld, n.code, on.stream());
  return sum ? tuple(y, s, mean, rstd) : tuple(y, a[0], mean, rstd);
}

// s, w, mean, rstd, dy, ds, groups, bias, lengths
PyObject* norm_bwd(PyObject* const* a) {
  const Norm n(a[0], "s", a[6], a[8]);
  void *w = dense(a[1], "w", {n.C}, n.type, n.dev), *mean = dense(a[2], "mean", n.stat, ScalarType::Float, n.dev),
       *rstd = dense(a[3], "rstd", n.stat, ScalarType::Float, n.dev), *dy = dense(a[4], "dy", n.shape, n.type, n.dev),
       *ds = dense_or_none(a[5], "ds", n.shape, n.type, n.dev);
  const bool bias = truth(a[7]);
  const On on(tensor(a[0], "s"));
  const Tensor dx = on.make(n.shape, n.type), dw = on.make({n.C}, n.type);
  Tensor db;
  if (bias) db = on.make({n.C}, n.type);
  const Room ws(on, la_norm_workspace_bytes(n.B, n.N, n.C, n.G, n.code));
  call(la_norm_bwd, "la_norm_bwd", n.x.p, w, static_cast<const float*>(mean), static_cast<const float*>(rstd),
       static_cast<const int*>(n.lengths), dy, ds, dx.data_ptr(), dw.data_ptr(), bias ? db.data_ptr() : nullptr, ws.p, ws.bytes, n.B, n.N, n.C, n.G, n.x.ld, n.code, on.stream());
  return bias ? tuple(dx, dw, db) : tuple(dx, dw, Py_None);
}

// ---------------------------------------------------------------- rotary positions

// q, k, turns, positions, gain, interleaved, head_major, lengths, inplace, inverse
PyObject* rotary(PyObject* const* a) {
  const Tensor& q = tensor(a[0], "q");
  const bool keys = !none(a[1]), step = q.dim() == 3, head_major = truth(a[6]), inplace = truth(a[8]);
  if ((q.dim() != 3 && q.dim() != 4) || (step && (head_major || !none(a[7]))))
    value_error("q: 4 dimensions, or 3 (one row a stream, token-major, without lengths)");
  const IntArrayRef shape = q.sizes();
  const ScalarType type = q.scalar_type();
  const c10::Device dev = q.device();
  const la_dtype code = code_of(q);
  const int lead = static_cast<int>(q.dim()) - 2, heads = head_major ? 1 : lead;  // the dimension that is the heads'
  c10::SmallVector<int64_t, 4> kshape(shape.begin(), shape.end());
  if (keys) {
    const Tensor& k = tensor(a[1], "k");
    if (k.dim() != q.dim()) value_error("k: " + std::to_string(q.dim()) + " dimensions, as q");
    kshape[heads] = k.size(heads);
  }
  const int B = size(shape[0]), N = step ? 1 : size(shape[head_major ? 2 : 1]), H = size(shape[heads]), D = size(shape.back()),
            Hk = keys ? size(kshape[heads]) : 0;
  Strided pq, pk{nullptr, 0};
  if (head_major) {
    pq = {dense(a[0], "q", shape, type, dev), 0};
    if (keys) pk = {dense(a[1], "k", kshape, type, dev), 0};
  } else {
    pq = strided(a[0], "q", shape, type, dev, lead);
    if (keys) pk = strided(a[1], "k", kshape, type, dev, lead);
  }
  const Tensor& turns = tensor(a[2], "turns");
  if (turns.dim() != 1) value_error("turns: 1 dimension");
  const int R = size(2 * turns.size(0));
  void* pt = dense(a[2], "turns", turns.sizes(), ScalarType::Long, dev);
  const bool per_row = !none(a[3]) && tensor(a[3], "positions").dim() == 2;
  void* pp = per_row ? dense(a[3], "positions", {B, N}, ScalarType::Int, dev) : dense_or_none(a[3], "positions", {B}, ScalarType::Int, dev);
  void* pn = dense_or_none(a[7], "lengths", {B}, ScalarType::Int, dev);
  const float gain = static_cast<float>(real(a[4]));
  const bool interleaved = truth(a[5]), inverse = truth(a[9]);
  if (inplace && pq.p == pk.p) value_error("inplace: q and k must be different tensors");
  const On on(q);
  Tensor oq, ok;
  if (!inplace) oq = on.make(shape, type);
  if (!inplace && keys) ok = on.make(kshape, type);
  void *to_q = inplace ? pq.p : oq.data_ptr(), *to_k = inplace ? pk.p : keys ? ok.data_ptr() : nullptr;
  call(la_rotary, "la_rotary", pq.p, pk.p, to_q, to_k, pt, static_cast<const int*>(pp), static_cast<const int*>(pn), gain,
       B, N, H, Hk, D, R, pq.ld, pk.ld, per_row, interleaved, head_major, inverse, code, on.stream());
  if (inplace) return tuple(a[0], a[1]);
  return keys ? tuple(oq, ok) : tuple(oq, Py_None);
}

// ---------------------------------------------------------------- states in 8 bits

// S, format
PyObject* state_pack(PyObject* const* a) {
  const Tensor& S = tensor(a[0], "S");
  if (S.dim() != 4) value_error("S: 4 dimensions");
  const IntArrayRef s = S.sizes();
  const int B = size(s[0]), H = size(s[1]), D = size(s[2]), M = size(s[3]), fmt = static_cast<int>(whole(a[1]));
  void* p = dense(a[0], "S", s, ScalarType::Float, S.device());
  const On on(S);
  const Tensor codes = on.make(s, fmt == LA_CODE_I8 ? ScalarType::Char : ScalarType::Float8_e4m3fn);
  const Tensor scale = on.make(s.slice(0, 3), ScalarType::Float);
  call(la_state_pack, "la_state_pack", static_cast<const float*>(p), codes.data_ptr(), scale.data_ptr<float>(), B, H, D, M, fmt,
       on.stream());
  return tuple(codes, scale);
}

// codes, scale
PyObject* state_unpack(PyObject* const* a) {
  const Tensor& codes = tensor(a[0], "codes");
  if (codes.dim() != 4) value_error("codes: 4 dimensions");
  const IntArrayRef s = codes.sizes();
  const int B = size(s[0]), H = size(s[1]), D = size(s[2]), M = size(s[3]), fmt = format_of(codes);
  const c10::Device dev = codes.device();
  void *p = dense(a[0], "codes", s, codes.scalar_type(), dev), *scale = dense(a[1], "scale", s.slice(0, 3), ScalarType::Float, dev);
  const On on(codes);
  const Tensor S = on.make(s, ScalarType::Float);
  call(la_state_unpack, "la_state_unpack", p, static_cast<const float*>(scale), S.data_ptr<float>(), B, H, D, M, fmt, on.stream());
  return out(S);
}

// q, codes, scale, Z
PyObject* cross_step_packed(PyObject* const* a) {
  const Tensor &q = tensor(a[0], "q"), &codes = tensor(a[1], "codes");
  if (q.dim() != 3 || codes.dim() != 4) value_error("q: 3 dimensions, codes: 4");
  const int B = size(q.size(0)), H = size(q.size(1)), D = size(q.size(2)), Hk = size(codes.size(1)), M = size(codes.size(3));
  const la_dtype code = code_of(q);
  const int fmt = format_of(codes);
  const c10::Device dev = q.device();
  void *pq = dense(a[0], "q", q.sizes(), q.scalar_type(), dev), *pc = dense(a[1], "codes", {B, Hk, D, M}, codes.scalar_type(), dev),
       *ps = dense(a[2], "scale", {B, Hk, D}, ScalarType::Float, dev), *pz = dense(a[3], "Z", {B, Hk, D}, ScalarType::Float, dev);
  const On on(q);
  const Tensor y = on.make({B, H, M}, q.scalar_type());
  call(la_cross_step_packed, "la_cross_step_packed", pq, pc, static_cast<const float*>(ps), static_cast<const float*>(pz), y.data_ptr(),
       B, H, Hk, D, M, fmt, code, on.stream());
  return out(y);
}

// ---------------------------------------------------------------- the module

template <PyObject* (*f)(PyObject* const*), int count>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != count) {
    PyErr_Format(PyExc_TypeError, "%d arguments, not %zd", count, n);
    return nullptr;
  }
  try {
    return f(args);
  } catch (const Refused& e) {
    PyErr_SetString(e.type, e.what.c_str());
  } catch (const Raised&) {
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

PyObject* setup(PyObject*, PyObject* error) {
  Py_XSETREF(g_error, held(error));
  Py_RETURN_NONE;
}

template <PyObject* (*f)(PyObject* const*), int count>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<f, count>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<gated_fwd, 8>("gated_fwd"),
    method<gated_bwd, 8>("gated_bwd"),
    method<gated_step, 6>("gated_step"),
    method<norm_fwd, 7>("norm_fwd"),
    method<norm_bwd, 9>("norm_bwd"),
    method<rotary, 10>("rotary"),
    method<state_pack, 2>("state_pack"),
    method<state_unpack, 2>("state_unpack"),
    method<cross_step_packed, 4>("cross_step_packed"),
    {"setup", setup, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_front", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__front() { return PyModule_Create(&g_module); }
