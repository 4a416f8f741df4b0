// The Python calls of a speculative decoding step: checks of their tensors, outputs
// and workspaces, then the C ABI.  A call of a few microseconds on the GPU has up to
// twenty tensors, and looking at each from Python took longer than its kernel (a decode
// step's append: 13 us of checks beside 4 us of kernel); here it is a field in memory.
// The module knows torch's tensors and nothing of the GPU: the functions of libwq.so
// are bound by address, and streams come as raw handles.
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <sstream>
#include <stdexcept>
#include <string>

#include "../../include/libwq.h"

namespace {

struct Abi {
  decltype(&wq_kv_append) kv_append;
  decltype(&wq_kv_tree_attention) kv_tree_attention;
  decltype(&wq_kv_tree_attention_workspace_bytes) kv_tree_attention_workspace_bytes;
  decltype(&wq_verify_drafts) verify_drafts;
  decltype(&wq_verify_drafts_workspace_bytes) verify_drafts_workspace_bytes;
  decltype(&wq_kv_keep) kv_keep;
} abi;

// Arguments a refused call names; they become Python's ValueError and TypeError.
[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

struct WrongType : std::runtime_error {
  using std::runtime_error::runtime_error;
};

// Other threads run Python while this one is in the allocator or the GPU's runtime, which may wait.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

template <class F>
int unlocked(F call) {
  const Unlocked u;
  return call();
}

std::string type_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kDouble: return "torch.float64";
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kByte: return "torch.uint8";
    case at::kChar: return "torch.int8";
    case at::kShort: return "torch.int16";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    case at::kBool: return "torch.bool";
    default: return c10::toString(t);
  }
}

std::string shape_of(c10::IntArrayRef s) {
  std::ostringstream o;
  o << "(";
  for (size_t i = 0; i < s.size(); ++i) o << (i ? ", " : "") << s[i];
  o << (s.size() == 1 ? ",)" : ")");
  return o.str();
}

bool is_none(PyObject* o) { return o == Py_None; }

const at::Tensor& tensor(const char* name, PyObject* o) {
  if (!THPVariable_Check(o)) throw WrongType(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// The address of a contiguous tensor of exactly that type and shape on that device.
void* array(const char* name, const at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape,
            const at::Device& dev) {
  if (t.scalar_type() != type || t.sizes() != c10::IntArrayRef(shape) || t.device() != dev || !t.is_contiguous()) {
    std::ostringstream o;
    o << name << " must be a contiguous " << type_of(type) << " tensor of shape " << shape_of(shape) << " on " << dev << " (got "
      << type_of(t.scalar_type()) << ", shape " << shape_of(t.sizes()) << ", on " << t.device() << ")";
    refuse(o.str());
  }
  return t.data_ptr();
}
void* array(const char* name, PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape, const at::Device& dev) {
  return array(name, tensor(name, o), type, shape, dev);
}
void* array_or_null(const char* name, PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape,
                    const at::Device& dev) {
  return is_none(o) ? nullptr : array(name, o, type, shape, dev);
}

int dtype16(at::ScalarType t) { return t == at::kBFloat16 ? WQ_BF16 : t == at::kHalf ? WQ_F16 : -1; }

// [tokens][heads][D] of a 16-bit type, heads and values contiguous; its stride between tokens.
int64_t heads(const char* name, const at::Tensor& x, const at::Tensor* like = nullptr, int64_t T = -1) {
  std::ostringstream o;
  if (x.dim() != 3 || dtype16(x.scalar_type()) < 0) {
    o << name << " must be a bfloat16 or float16 tensor [tokens][heads][D] (got " << type_of(x.scalar_type()) << ", shape "
      << shape_of(x.sizes()) << ")";
    refuse(o.str());
  }
  const int64_t n = x.size(0), h = x.size(1), d = x.size(2);
  if ((d > 1 && x.stride(2) != 1) || (h > 1 && x.stride(1) != d)) {
    o << name << ": the heads and values of a token must be contiguous (strides " << shape_of(x.strides()) << ")";
    refuse(o.str());
  }
  if (like && (x.scalar_type() != like->scalar_type() || x.device() != like->device() || d != like->size(2))) {
    o << name << " is " << type_of(x.scalar_type()) << " on " << x.device() << " with D=" << d << ", expected " << type_of(like->scalar_type())
      << " on " << like->device() << " with D=" << like->size(2);
    refuse(o.str());
  }
  if (T >= 0 && n != T) refuse(std::string(name) + " has " + std::to_string(n) + " tokens, expected " + std::to_string(T));
  return n > 1 ? x.stride(0) : h * d;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
int int32(const char* name, PyObject* o) {
  const int64_t v = integer(o);
  if (v != (int)v) refuse(std::string(name) + " must fit 32 bits (got " + std::to_string(v) + ")");
  return (int)v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

void on_gpu(const at::Device& dev) {
  if (dev.type() != at::kCUDA) refuse("tensors must be on the GPU (got " + dev.str() + ")");
}

at::Tensor make(std::initializer_list<int64_t> shape, at::ScalarType type, const at::Device& dev) {
  const Unlocked u;
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

// A K and a V cache: codes, s, zpacked, S, hd of each, ten arguments.
struct Caches {
  int64_t S, hd;
  void* p[6];
};
void cache_sizes(PyObject* const* a, Caches* c) {
  c->S = integer(a[3]);
  c->hd = integer(a[4]);
  const int64_t S = integer(a[8]), hd = integer(a[9]);
  if (S != c->S || hd != c->hd)
    refuse("caches of " + std::to_string(c->S) + " x " + std::to_string(c->hd) + " and " + std::to_string(S) + " x " +
           std::to_string(hd) + " values");
}
void cache_arrays(PyObject* const* a, const at::Device& dev, Caches* c) {
  static const char* const names[2][3] = {{"k_cache.codes", "k_cache.s", "k_cache.zpacked"},
                                          {"v_cache.codes", "v_cache.s", "v_cache.zpacked"}};
  const int64_t nb = c->hd / 128;
  for (int i = 0; i < 2; ++i) {
    c->p[3 * i] = array(names[i][0], a[5 * i], at::kByte, {c->S, c->hd / 2}, dev);
    c->p[3 * i + 1] = array(names[i][1], a[5 * i + 1], at::kHalf, {c->S, nb}, dev);
    c->p[3 * i + 2] = array(names[i][2], a[5 * i + 2], at::kByte, {c->S, (nb + 1) / 2}, dev);
  }
}

struct Pages {
  int64_t B, width;
  const int32_t *table, *lens;
};
Pages pages(PyObject* table, PyObject* lens, const at::Device& dev) {
  const at::Tensor& t = tensor("block_table", table);
  if (t.dim() != 2) refuse("block_table must be [sequences][pages]");
  const int64_t B = t.size(0), width = t.size(1);
  return {B, width, static_cast<int32_t*>(array("block_table", t, at::kInt, {B, width}, dev)),
          static_cast<int32_t*>(array("context_lens", lens, at::kInt, {B}, dev))};
}

// The caller's workspace, or one of `need` bytes.
struct Workspace {
  at::Tensor own;
  void* p = nullptr;
  size_t bytes = 0;
};
void check_workspace(PyObject* o, const at::Device& dev) {
  if (is_none(o)) return;
  const at::Tensor& t = tensor("workspace", o);
  if (t.device() != dev || !t.is_contiguous()) refuse("workspace must be a contiguous tensor on " + dev.str());
}
Workspace workspace(PyObject* o, size_t need, const at::Device& dev) {
  Workspace w;
  if (!is_none(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    w.p = t.data_ptr();
    w.bytes = (size_t)t.nbytes();
  } else if (need > 0) {
    w.own = make({(int64_t)need}, at::kByte, dev);
    w.p = w.own.data_ptr();
    w.bytes = need;
  }
  return w;
}

// Runs a call's body; what it throws becomes a Python error.
template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t expected, F body) {
  if (n != expected) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", expected, n);
    return nullptr;
  }
  if (!abi.kv_keep) {
    PyErr_SetString(PyExc_RuntimeError, "libwq.so is not loaded");
    return nullptr;
  }
  try {
    return body();
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const WrongType& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (python_error& e) {
    e.restore();
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* const m = PyImport_ImportModule("torch");
    PyObject* const type = m ? PyObject_GetAttrString(m, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(m);
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (k, v, 10 of the caches, block_table, context_lens, cos, sin, page_size, q, q_starts, positions, norm, q_weight,
// k_weight, eps, interleaved, q_out, k_out, stream) -> a status, or (q_out, k_out)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 28, [&]() -> PyObject* {
    const at::Tensor &k = tensor("k", a[0]), &v = tensor("v", a[1]);
    const int64_t ks = heads("k", k), vs = heads("v", v, &k, k.size(0));
    const int64_t T = k.size(0), Hkv = k.size(1), D = k.size(2);
    const at::Device dev = k.device();
    const at::ScalarType dt = k.scalar_type();
    if (v.size(1) != Hkv) refuse("k has " + std::to_string(Hkv) + " heads, v " + std::to_string(v.size(1)));
    Caches c;
    cache_sizes(a + 2, &c);
    if (c.hd != Hkv * D)
      refuse("caches of rows of " + std::to_string(c.hd) + " values, " + std::to_string(Hkv) + " heads of " + std::to_string(D));
    PyObject *oq = a[17], *oqo = a[25], *oko = a[26];
    int64_t Hq = Hkv, qs = 0, qos = 0, kos = Hkv * D;
    const at::Tensor *q = nullptr, *qo = nullptr, *ko = nullptr;
    if (!is_none(oq)) {
      q = &tensor("q", oq);
      qs = heads("q", *q, &k, T);
      Hq = q->size(1);
      qos = Hq * D;
    }
    if (!is_none(oqo)) {
      qo = &tensor("q_out", oqo);
      if (!q || qo->dim() != 3 || qo->size(1) != Hq) refuse("q_out must have the heads of q");
      qos = heads("q_out", *qo, q, T);
    }
    const bool make_ko = oko == Py_True;
    if (!make_ko && oko != Py_False && !is_none(oko)) {
      ko = &tensor("k_out", oko);
      kos = heads("k_out", *ko, &k, T);
      if (ko->size(1) != Hkv) refuse("k_out has " + std::to_string(ko->size(1)) + " heads, expected " + std::to_string(Hkv));
    }
    const at::Tensor& cos = tensor("cos", a[14]);
    if (cos.dim() != 2) refuse("cos must be [positions][pairs]");
    const int64_t P = cos.size(0), half = cos.size(1);
    const void *cp = array("cos", cos, at::kFloat, {P, half}, dev), *sp = array("sin", a[15], at::kFloat, {P, half}, dev);
    const void* pos = array_or_null("positions", a[19], at::kInt, {T}, dev);
    const bool norm = truth(a[20]), inter = truth(a[24]);
    const float eps = (float)number(a[23]);
    const int page = int32("page_size", a[16]);
    void* const stream = reinterpret_cast<void*>(integer(a[27]));
    if (!norm && (!is_none(a[21]) || !is_none(a[22]))) refuse("weights are the norm's: pass norm=True");
    const void *qw = array_or_null("q_weight", a[21], dt, {D}, dev), *kw = array_or_null("k_weight", a[22], dt, {D}, dev);
    cache_arrays(a + 2, dev, &c);
    const Pages pg = pages(a[12], a[13], dev);
    const void* starts = array_or_null("q_starts", a[18], at::kInt, {pg.B + 1}, dev);
    on_gpu(dev);
    at::Tensor new_q, new_k;
    if (q && !qo) new_q = make({T, Hq, D}, dt, dev);
    if (make_ko) new_k = make({T, Hkv, D}, dt, dev);
    void* qp = qo ? qo->data_ptr() : q ? new_q.data_ptr() : nullptr;
    void* kp = ko ? ko->data_ptr() : make_ko ? new_k.data_ptr() : nullptr;
    const int st = unlocked([&] { return abi.kv_append(
        q ? q->data_ptr() : nullptr, k.data_ptr(), v.data_ptr(), dtype16(dt), T, (int)Hq, (int)Hkv, (int)D, qs, ks, vs, norm, qw,
        kw, eps, static_cast<const int32_t*>(pos), static_cast<const float*>(cp),
        static_cast<const float*>(sp), P, (int)(2 * half), inter, static_cast<uint8_t*>(c.p[0]),
        static_cast<uint16_t*>(c.p[1]), static_cast<uint8_t*>(c.p[2]), static_cast<uint8_t*>(c.p[3]),
        static_cast<uint16_t*>(c.p[4]), static_cast<uint8_t*>(c.p[5]), c.S, pg.B, pg.table, pg.width, page, pg.lens,
        static_cast<const int32_t*>(starts), qp, kp, qos, kos, stream); });
    if (st) return PyLong_FromLong(st);
    PyObject* rq = new_q.defined() ? THPVariable_Wrap(new_q) : Py_NewRef(oqo);
    PyObject* rk = new_k.defined() ? THPVariable_Wrap(new_k) : ko ? Py_NewRef(oko) : Py_NewRef(Py_None);
    PyObject* r = PyTuple_Pack(2, rq, rk);
    Py_XDECREF(rq);
    Py_XDECREF(rk);
    return r;
  });
}

// (q, 10 of the caches, block_table, context_lens, tree_mask, page_size, max_context, q_starts, max_queries, scale, out,
// lse, workspace, stream) -> a status, out, or (out, lse)
PyObject* kv_tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 23, [&]() -> PyObject* {
    const at::Tensor& q = tensor("q", a[0]);
    const int64_t qs = heads("q", q), T = q.size(0), Hq = q.size(1), D = q.size(2);
    const at::Device dev = q.device();
    const at::ScalarType dt = q.scalar_type();
    Caches c;
    cache_sizes(a + 1, &c);
    if (D == 0 || c.hd % D != 0) refuse("caches of rows of " + std::to_string(c.hd) + " values, heads of " + std::to_string(D));
    const int64_t Hkv = c.hd / D;
    cache_arrays(a + 1, dev, &c);
    const Pages pg = pages(a[11], a[12], dev);
    const at::Tensor& mask = tensor("tree_mask", a[13]);
    if (mask.dim() != 2) refuse("tree_mask must be [tokens][words]");
    const int64_t words = mask.size(1);
    const void* mp = array("tree_mask", mask, at::kLong, {T, words}, dev);
    const void* starts = array_or_null("q_starts", a[16], at::kInt, {pg.B + 1}, dev);
    int64_t most = T < 1 ? T : 1;
    if (starts) {
      const int64_t room = words < (int64_t)1 << 32 ? 64 * words : T;
      most = is_none(a[17]) ? (T < room ? T : room) : integer(a[17]);
      if (most > T) most = T;
    }
    const int page = int32("page_size", a[14]);
    int64_t ctx = 0;
    if (!is_none(a[15])) {
      ctx = integer(a[15]);
    } else if (__builtin_mul_overflow(pg.width, (int64_t)page, &ctx)) {
      ctx = INT64_MAX;
    }
    const float scale = is_none(a[18]) ? (float)(1.0 / std::sqrt((double)D)) : (float)number(a[18]);
    void* const stream = reinterpret_cast<void*>(integer(a[22]));
    check_workspace(a[21], dev);
    const at::Tensor *out = nullptr, *lse = nullptr;
    if (!is_none(a[19])) {
      out = &tensor("out", a[19]);
      array("out", *out, dt, {T, Hq, D}, dev);
    }
    const bool make_lse = a[20] == Py_True;
    if (!make_lse && a[20] != Py_False && !is_none(a[20])) {
      lse = &tensor("lse", a[20]);
      array("lse", *lse, at::kFloat, {T, Hq}, dev);
    }
    on_gpu(dev);
    at::Tensor new_out, new_lse;
    if (!out) new_out = make({T, Hq, D}, dt, dev);
    if (make_lse) new_lse = make({T, Hq}, at::kFloat, dev);
    const Workspace ws = workspace(
        a[21],
        is_none(a[21]) ? abi.kv_tree_attention_workspace_bytes(T, (int)Hq, (int)Hkv, (int)D, pg.B, page, ctx, most) : 0, dev);
    const int st = unlocked([&] { return abi.kv_tree_attention(
        q.data_ptr(), dtype16(dt), T, (int)Hq, (int)Hkv, (int)D, qs, static_cast<uint8_t*>(c.p[0]),
        static_cast<uint16_t*>(c.p[1]), static_cast<uint8_t*>(c.p[2]), static_cast<uint8_t*>(c.p[3]),
        static_cast<uint16_t*>(c.p[4]), static_cast<uint8_t*>(c.p[5]), c.S, pg.B, pg.table, pg.width, page, pg.lens, ctx,
        static_cast<const int32_t*>(starts), most, static_cast<const uint64_t*>(mp), (int)(words > 65536 ? 65537 : words), scale,
        out ? out->data_ptr() : new_out.data_ptr(),
        lse ? static_cast<float*>(lse->data_ptr()) : make_lse ? static_cast<float*>(new_lse.data_ptr()) : nullptr, ws.p, ws.bytes,
        stream); });
    if (st) return PyLong_FromLong(st);
    PyObject* ro = out ? Py_NewRef(a[19]) : THPVariable_Wrap(new_out);
    if (!lse && !make_lse) return ro;
    PyObject* rl = lse ? Py_NewRef(a[20]) : THPVariable_Wrap(new_lse);
    PyObject* r = PyTuple_Pack(2, ro, rl);
    Py_XDECREF(ro);
    Py_XDECREF(rl);
    return r;
  });
}

int64_t rows(const char* name, const at::Tensor& x) {
  if (x.dim() != 2 || (x.size(1) > 1 && x.stride(1) != 1)) {
    std::ostringstream o;
    o << name << " must be [tokens][vocabulary] with contiguous rows (shape " << shape_of(x.sizes()) << ", strides "
      << shape_of(x.strides()) << ")";
    refuse(o.str());
  }
  return x.size(0) > 1 ? x.stride(0) : x.size(1);
}

// (logits, tokens, uniform, q_starts, max_queries, parents, draft_logits, temperature, out_tokens, path, counts, workspace,
// stream) -> a status, or (out_tokens, path, counts)
PyObject* verify_drafts(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const at::Tensor& logits = tensor("logits", a[0]);
    const at::ScalarType dt = logits.scalar_type();
    const int code = dt == at::kFloat ? WQ_F32 : dtype16(dt);
    if (code < 0) {
      std::ostringstream o;
      o << "logits must be float32, bfloat16 or float16 (got " << type_of(dt) << ")";
      refuse(o.str());
    }
    const int64_t stride = rows("logits", logits), T = logits.size(0), V = logits.size(1);
    const at::Device dev = logits.device();
    const at::Tensor* draft = nullptr;
    int64_t dstride = 0;
    if (!is_none(a[6])) {
      draft = &tensor("draft_logits", a[6]);
      dstride = rows("draft_logits", *draft);
      if (draft->sizes() != logits.sizes() || draft->scalar_type() != dt || draft->device() != dev) {
        std::ostringstream o;
        o << "draft_logits must be like logits (got " << type_of(draft->scalar_type()) << ", shape " << shape_of(draft->sizes()) << ", on "
          << draft->device() << ")";
        refuse(o.str());
      }
    }
    const void *tok = array("tokens", a[1], at::kInt, {T}, dev), *u = array("uniform", a[2], at::kFloat, {T}, dev);
    const void* par = array_or_null("parents", a[5], at::kInt, {T}, dev);
    int64_t B = T;
    const void* starts = nullptr;
    if (!is_none(a[3])) {
      const at::Tensor& s = tensor("q_starts", a[3]);
      if (s.dim() != 1 || s.numel() < 1) refuse("q_starts must hold B + 1 token numbers");
      B = s.numel() - 1;
      starts = array("q_starts", s, at::kInt, {B + 1}, dev);
    }
    const int64_t most = !is_none(a[4]) ? integer(a[4]) : !starts ? 1 : T < 1 ? 1 : T > 1024 ? 1024 : T;
    void* const stream = reinterpret_cast<void*>(integer(a[12]));
    const void* temp = array_or_null("temperature", a[7], at::kFloat, {B}, dev);
    static const char* const names[3] = {"out_tokens", "path", "counts"};
    void* p[3];
    for (int i = 0; i < 3; ++i)
      p[i] = is_none(a[8 + i]) ? nullptr
             : i < 2           ? array(names[i], a[8 + i], at::kInt, {B, most}, dev)
                               : array(names[i], a[8 + i], at::kInt, {B}, dev);
    check_workspace(a[11], dev);
    on_gpu(dev);
    at::Tensor made[3];
    const int64_t width = most > 0 ? most : 0;
    for (int i = 0; i < 3; ++i)
      if (is_none(a[8 + i])) {
        made[i] = i < 2 ? make({B, width}, at::kInt, dev) : make({B}, at::kInt, dev);
        p[i] = made[i].data_ptr();
      }
    const Workspace ws =
        workspace(a[11], is_none(a[11]) ? abi.verify_drafts_workspace_bytes(T, V, B, draft ? 1 : 0) : 0, dev);
    const int st = unlocked([&] { return abi.verify_drafts(
        logits.data_ptr(), code, T, V, stride, draft ? draft->data_ptr() : nullptr, dstride, B,
        static_cast<const int32_t*>(starts), most, static_cast<const int32_t*>(tok), static_cast<const int32_t*>(par),
        static_cast<const float*>(u), static_cast<const float*>(temp), static_cast<int32_t*>(p[0]), static_cast<int32_t*>(p[1]),
        static_cast<int32_t*>(p[2]), ws.p, ws.bytes, stream); });
    if (st) return PyLong_FromLong(st);
    PyObject* r = PyTuple_New(3);
    for (int i = 0; r && i < 3; ++i)
      PyTuple_SET_ITEM(r, i, made[i].defined() ? THPVariable_Wrap(made[i]) : Py_NewRef(a[8 + i]));
    return r;
  });
}

// (10 of the caches, block_table, context_lens, path, counts, page_size, q_starts, stream) -> a status
PyObject* kv_keep(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    const at::Device dev = tensor("k_cache.codes", a[0]).device();
    Caches c;
    cache_sizes(a, &c);
    cache_arrays(a, dev, &c);
    const Pages pg = pages(a[10], a[11], dev);
    const void* starts = array("q_starts", a[15], at::kInt, {pg.B + 1}, dev);
    const at::Tensor& path = tensor("path", a[12]);
    if (path.dim() != 2) refuse("path must be [sequences][nodes]");
    const void *pp = array("path", path, at::kInt, {pg.B, path.size(1)}, dev), *cn = array("counts", a[13], at::kInt, {pg.B}, dev);
    const int page = int32("page_size", a[14]);
    void* const stream = reinterpret_cast<void*>(integer(a[16]));
    on_gpu(dev);
    // (how many tokens the call had is on the device: all that q_starts names)
    const int st = unlocked([&] { return abi.kv_keep(static_cast<uint8_t*>(c.p[0]), static_cast<uint16_t*>(c.p[1]), static_cast<uint8_t*>(c.p[2]),
                       static_cast<uint8_t*>(c.p[3]), static_cast<uint16_t*>(c.p[4]), static_cast<uint8_t*>(c.p[5]), c.S, c.hd,
                       ((int64_t)1 << 31) - 1, pg.B, pg.table, pg.width, page, pg.lens, static_cast<const int32_t*>(starts),
                       static_cast<const int32_t*>(pp), path.size(1), static_cast<const int32_t*>(cn), stream); });
    return PyLong_FromLong(st);
  });
}

// (addresses of libwq's functions, in Abi's order)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "expected 6 addresses");
    return nullptr;
  }
  void* p[6];
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i] && PyErr_Occurred()) return nullptr;
  }
  abi.kv_append = reinterpret_cast<decltype(abi.kv_append)>(p[0]);
  abi.kv_tree_attention = reinterpret_cast<decltype(abi.kv_tree_attention)>(p[1]);
  abi.kv_tree_attention_workspace_bytes = reinterpret_cast<decltype(abi.kv_tree_attention_workspace_bytes)>(p[2]);
  abi.verify_drafts = reinterpret_cast<decltype(abi.verify_drafts)>(p[3]);
  abi.verify_drafts_workspace_bytes = reinterpret_cast<decltype(abi.verify_drafts_workspace_bytes)>(p[4]);
  abi.kv_keep = reinterpret_cast<decltype(abi.kv_keep)>(p[5]);
  Py_RETURN_NONE;
}

#define WQ_CALL(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {WQ_CALL(kv_append), WQ_CALL(kv_tree_attention), WQ_CALL(verify_drafts), WQ_CALL(kv_keep), WQ_CALL(bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
