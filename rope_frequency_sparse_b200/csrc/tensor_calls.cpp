// tensor_calls.cpp -- the paged serving calls on torch tensors: argument checks,
// allocation of outputs that the caller did not pass, the argument structures of
// include/atf.h and the call on the tensors' device and current stream.
//
// A call checks up to 16 tensors.  As Python over ctypes that took 23 to 44 us a
// call, three times the kernels of a single-token step, so it is compiled.  The
// kernels stay in libatf.so, whose loaded handle `bind` is given.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <initializer_list>
#include <optional>
#include <string>

#include "../../include/atf.h"

namespace {

struct Refusal {  // raised as a TypeError
  std::string what;
};
struct PythonError {};  // already set

atf_status (*f_norm_rope)(const atf_qk_norm_rope_args*, void*) = nullptr;
atf_status (*f_append)(const atf_paged_append_args*, void*) = nullptr;
atf_status (*f_decode)(const atf_paged_decode_args*, void*) = nullptr;
atf_status (*f_select)(const atf_page_select_args*, void*) = nullptr;
size_t (*f_decode_bytes)(int, int, int, int) = nullptr;
size_t (*f_select_bytes)(int, int, int) = nullptr;
PyObject* raise_status = nullptr;  // Python: raises the library's last error as AtfError(status)

std::string describe(const at::Tensor& x) {
  std::string s = "(";
  for (int64_t i = 0; i < x.dim(); ++i) s += (i ? ", " : "") + std::to_string(x.size(i));
  return s + ") " + c10::toString(x.scalar_type());
}

// The tensor of a Python argument; null for None where that is allowed.
const at::Tensor* tensor(const char* name, PyObject* o, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw Refusal{std::string(name) + ": a tensor is expected"};
  return &THPVariable_Unpack(o);
}

// x must be contiguous, of this type and shape (-1: any extent).
const at::Tensor& dense(const char* name, const at::Tensor& x, at::ScalarType type, std::initializer_list<int64_t> shape) {
  bool ok = x.scalar_type() == type && x.dim() == static_cast<int64_t>(shape.size()) && x.is_contiguous();
  int i = 0;
  for (const int64_t n : shape) {
    ok = ok && (n < 0 || x.size(i) == n);
    ++i;
  }
  if (ok) return x;
  std::string want;
  for (const int64_t n : shape) want += (want.empty() ? "" : ", ") + (n < 0 ? std::string("*") : std::to_string(n));
  throw Refusal{std::string(name) + ": a contiguous " + c10::toString(type) + " tensor of shape (" + want +
                ") is expected, got " + describe(x)};
}

// Token stride of x [T][H][d], whose heads are contiguous (a slice of a fused
// projection is fine); heads and d -1: any.
long long head_rows(const char* name, const at::Tensor& x, at::ScalarType type, int64_t heads, int64_t d) {
  if (x.dim() != 3 || x.scalar_type() != type || (heads >= 0 && x.size(1) != heads) || (d >= 0 && x.size(2) != d))
    throw Refusal{std::string(name) + ": a [tokens][heads][d] tensor of " + c10::toString(type) + " is expected, got " +
                  describe(x)};
  const int64_t T = x.size(0), H = x.size(1), n = x.size(2);
  if (T * H * n && (x.stride(2) != 1 || (H > 1 && x.stride(1) != n)))
    throw Refusal{std::string(name) + ": the heads of a token must be contiguous"};
  return T > 1 ? x.stride(0) : H * n;
}

int extent(const char* name, int64_t n) {
  if (n > INT_MAX) throw Refusal{std::string(name) + " does not fit 32 bits"};
  return static_cast<int>(n);
}

void* address(const at::Tensor* x) { return x ? x->data_ptr() : nullptr; }

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw PythonError{};
  return x;
}

long long whole(const char* name, PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw PythonError{};
  if (x > INT_MAX || x < INT_MIN) throw Refusal{std::string(name) + " does not fit 32 bits"};
  return x;
}

// The position axis of each pair, from bytes or a sequence of small integers.
struct PairAxis {
  unsigned char axis[64];
  const unsigned char* get(PyObject* o, int64_t d) {
    if (o == Py_None) return nullptr;
    PyObject* seq = PySequence_Fast(o, "pair_axis: a sequence is expected");
    if (!seq) throw PythonError{};
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
    std::string refused;
    if (n != d / 2) {
      refused = "pair_axis: " + std::to_string(d / 2) + " entries are expected, got " + std::to_string(n);
    } else {
      for (Py_ssize_t i = 0; i < n && refused.empty(); ++i) {
        const long a = PyLong_AsLong(PySequence_Fast_GET_ITEM(seq, i));
        if (a == -1 && PyErr_Occurred()) {
          Py_DECREF(seq);
          throw PythonError{};
        }
        if (a < 0 || a > 255) refused = "pair_axis: an entry of " + std::to_string(a);
        if (i < 64) axis[i] = static_cast<unsigned char>(a);
      }
    }
    Py_DECREF(seq);
    if (!refused.empty()) throw Refusal{refused};
    return axis;
  }
};

// Positions [axes][tokens] (None: the slots); returns the axes.
int positions(const at::Tensor* pos, int64_t tokens) {
  return pos ? extent("pos", dense("pos", *pos, at::kLong, {-1, tokens}).size(0)) : 1;
}

void* weight(const char* name, const at::Tensor* w, at::ScalarType type, int64_t d) {
  return w ? dense(name, *w, type, {d}).data_ptr() : nullptr;
}

struct Named {
  const char* name;
  const at::Tensor* x;
};

// All tensors on one CUDA device.
void on_device(const at::Tensor& first, std::initializer_list<Named> others) {
  const c10::Device dev = first.device();
  if (!dev.is_cuda()) throw Refusal{"tensors of a CUDA device are expected, got " + dev.str()};
  for (const Named& t : others)
    if (t.x && t.x->device() != dev)
      throw Refusal{std::string(t.name) + " is on " + t.x->device().str() + ", the queries or keys on " + dev.str()};
}

// Where a call runs: the tensors' device, and `stream` or that device's current
// one.  While it lives both are current, so that what the call allocates belongs to
// the stream that uses it (a scratch freed on return is reused in stream order only).
class Target {
 public:
  Target(const at::Tensor& x, PyObject* stream) {
    if (!x.is_cuda()) return;  // refused by on_device, after the checks of types and shapes
    const c10::DeviceIndex dev = x.device().index();
    if (stream == Py_None) {
      device_.emplace(dev);
      stream_ = c10::cuda::getCurrentCUDAStream(dev).stream();
      return;
    }
    PyObject* v = PyLong_Check(stream) ? Py_NewRef(stream) : PyObject_GetAttrString(stream, "cuda_stream");
    if (!v) throw PythonError{};
    void* s = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (!s && PyErr_Occurred()) throw PythonError{};
    stream_ = static_cast<cudaStream_t>(s);
    if (stream_ == cudaStreamPerThread) throw Refusal{"stream: the per-thread default stream has no torch stream"};
    // torch tells its own streams from handles by the low bit, which the legacy default's has set
    guard_.emplace(stream_ == nullptr || stream_ == cudaStreamLegacy ? c10::cuda::getDefaultCUDAStream(dev)
                                                                     : c10::cuda::getStreamFromExternal(stream_, dev));
  }

  template <typename Args>
  void launch(atf_status (*fn)(const Args*, void*), const Args& args) const {
    if (!fn) throw Refusal{"the library is not bound"};
    atf_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = fn(&args, stream_);
    Py_END_ALLOW_THREADS;
    if (st == ATF_OK) return;
    PyObject* r = PyObject_CallFunction(raise_status, "i", static_cast<int>(st));
    if (!r) throw PythonError{};
    Py_DECREF(r);
    throw Refusal{"status " + std::to_string(static_cast<int>(st))};
  }

 private:
  std::optional<c10::cuda::CUDAGuard> device_;
  std::optional<c10::cuda::CUDAStreamGuard> guard_;
  cudaStream_t stream_ = nullptr;
};

template <typename Body>
PyObject* guarded(const char* who, Py_ssize_t got, Py_ssize_t want, Body body) {
  try {
    if (got != want) throw Refusal{std::string(who) + ": " + std::to_string(want) + " arguments are expected"};
    return body();
  } catch (const Refusal& e) {
    PyErr_SetString(PyExc_TypeError, e.what.c_str());
  } catch (const PythonError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// ------------------------------------------------------------------ the calls

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("bind", n, 2, [&]() -> PyObject* {
    void* lib = PyLong_AsVoidPtr(a[0]);
    if (!lib && PyErr_Occurred()) throw PythonError{};
    auto sym = [&](const char* name) {
      void* p = dlsym(lib, name);
      if (!p) throw Refusal{std::string("the library has no ") + name};
      return p;
    };
    f_norm_rope = reinterpret_cast<decltype(f_norm_rope)>(sym("atf_qk_norm_rope"));
    f_append = reinterpret_cast<decltype(f_append)>(sym("atf_paged_append"));
    f_decode = reinterpret_cast<decltype(f_decode)>(sym("atf_paged_decode"));
    f_select = reinterpret_cast<decltype(f_select)>(sym("atf_page_select"));
    f_decode_bytes = reinterpret_cast<decltype(f_decode_bytes)>(sym("atf_paged_decode_workspace_bytes"));
    f_select_bytes = reinterpret_cast<decltype(f_select_bytes)>(sym("atf_page_select_workspace_bytes"));
    Py_XSETREF(raise_status, Py_NewRef(a[1]));
    Py_RETURN_NONE;
  });
}

// q, k, theta, pos, q_weight, k_weight, eps, pair_axis, pairing, q_out, k_out, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded("qk_norm_rope", n, 12, [&]() -> PyObject* {
    const at::Tensor &q = *tensor("q", o[0]), &k = *tensor("k", o[1]);
    const at::Tensor* pos = tensor("pos", o[3]);
    const at::Tensor *qw = tensor("q_weight", o[4], true), *kw = tensor("k_weight", o[5], true);
    const at::ScalarType type = q.scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat)
      throw Refusal{std::string("unsupported dtype ") + c10::toString(type)};
    atf_qk_norm_rope_args a{};
    a.q_stride = head_rows("q", q, type, -1, -1);
    const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2);
    a.k_stride = head_rows("k", k, type, -1, d);
    const int64_t Hkv = k.size(1);
    if (k.size(0) != T) throw Refusal{"q has " + std::to_string(T) + " tokens, k " + std::to_string(k.size(0))};
    PairAxis axis;
    a.pair_axis = axis.get(o[7], d);
    a.n_axes = positions(pos, T);
    const Target target(q, o[11]);
    at::Tensor q_new, k_new;
    const at::Tensor *qo = tensor("q_out", o[9], true), *ko = tensor("k_out", o[10], true);
    if (!qo) q_new = at::empty({T, Hq, d}, q.options()), qo = &q_new;
    if (!ko) k_new = at::empty({T, Hkv, d}, q.options()), ko = &k_new;
    dense("q_out", *qo, type, {T, Hq, d});
    dense("k_out", *ko, type, {T, Hkv, d});
    a.q_weight = weight("q_weight", qw, type, d);
    a.k_weight = weight("k_weight", kw, type, d);
    on_device(q, {{"k", &k}, {"pos", pos}, {"q_weight", qw}, {"k_weight", kw}, {"q_out", qo}, {"k_out", ko}});
    a.q = q.data_ptr();
    a.k = k.data_ptr();
    a.q_out = qo->data_ptr();
    a.k_out = ko->data_ptr();
    a.pos = static_cast<const long long*>(pos->data_ptr());
    a.tokens = extent("tokens", T);
    a.heads = extent("heads", Hq);
    a.kv_heads = extent("kv_heads", Hkv);
    a.d = extent("d", d);
    a.pairing = static_cast<int>(whole("pairing", o[8]));
    a.dtype = type == at::kFloat ? ATF_FP32 : ATF_BF16;
    a.theta = number(o[2]);
    a.eps = static_cast<float>(number(o[6]));
    target.launch(f_norm_rope, a);
    PyObject* r = PyTuple_New(2);
    if (!r) throw PythonError{};
    PyTuple_SET_ITEM(r, 0, o[9] == Py_None ? THPVariable_Wrap(*qo) : Py_NewRef(o[9]));
    PyTuple_SET_ITEM(r, 1, o[10] == Py_None ? THPVariable_Wrap(*ko) : Py_NewRef(o[10]));
    return r;
  });
}

// Sizes of a paged cache.
struct Pool {
  int64_t pages, hkv, d, page, batch, max_pages;
  Pool(const at::Tensor& k, const at::Tensor& v, const at::Tensor& table) {
    if (k.dim() != 5) throw Refusal{"k_pages: [pages][kv heads][d/16][page size][16] is expected, got " + describe(k)};
    pages = k.size(0), hkv = k.size(1), d = k.size(2) * 16, page = k.size(3);
    dense("k_pages", k, at::kBFloat16, {pages, hkv, d / 16, page, 16});
    dense("v_pages", v, at::kBFloat16, {pages, hkv, page, d});
    dense("page_table", table, at::kInt, {-1, -1});
    batch = table.size(0), max_pages = table.size(1);
  }
};

// q, k, v, k_pages, v_pages, page_table, start, theta, cu, pos, q_weight, k_weight, eps, pair_axis, pairing, bounds,
// q_out, stream
PyObject* paged_append(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded("paged_append", n, 18, [&]() -> PyObject* {
    const at::Tensor* q = tensor("q", o[0], true);
    const at::Tensor &k = *tensor("k", o[1]), &v = *tensor("v", o[2]), &kp = *tensor("k_pages", o[3]),
                     &vp = *tensor("v_pages", o[4]), &table = *tensor("page_table", o[5]), &start = *tensor("start", o[6]);
    const at::Tensor *cu = tensor("cu", o[8], true), *pos = tensor("pos", o[9], true),
                     *qw = tensor("q_weight", o[10], true), *kw = tensor("k_weight", o[11], true),
                     *bounds = tensor("bounds", o[15], true), *qo = tensor("q_out", o[16], true);
    const Pool c(kp, vp, table);
    const at::ScalarType bf16 = at::kBFloat16;
    atf_paged_append_args a{};
    a.k_stride = head_rows("k", k, bf16, c.hkv, c.d);
    a.v_stride = head_rows("v", v, bf16, c.hkv, c.d);
    const int64_t T = k.size(0);
    if (v.size(0) != T || (q && q->size(0) != T)) throw Refusal{"q, k and v must have the same tokens"};
    PairAxis axis;
    a.pair_axis = axis.get(o[13], c.d);
    const Target target(k, o[17]);
    at::Tensor q_new;
    int64_t Hq = c.hkv;
    if (q) {
      a.q_stride = head_rows("q", *q, bf16, -1, c.d);
      Hq = q->size(1);
      if (!qo) q_new = at::empty({T, Hq, c.d}, q->options()), qo = &q_new;
      dense("q_out", *qo, bf16, {T, Hq, c.d});
    }
    dense("start", start, at::kInt, {c.batch});
    if (cu) dense("cu", *cu, at::kInt, {c.batch + 1});
    if (bounds) dense("bounds", *bounds, bf16, {c.pages, c.hkv, 2, c.d});
    a.n_axes = positions(pos, T);
    a.q_weight = weight("q_weight", qw, bf16, c.d);
    a.k_weight = weight("k_weight", kw, bf16, c.d);
    on_device(k, {{"q", q}, {"v", &v}, {"k_pages", &kp}, {"v_pages", &vp}, {"page_table", &table}, {"start", &start},
                  {"cu", cu}, {"pos", pos}, {"q_weight", qw}, {"k_weight", kw}, {"bounds", bounds}, {"q_out", qo}});
    a.q = address(q);
    a.k = k.data_ptr();
    a.v = v.data_ptr();
    a.q_out = address(qo);
    a.k_pages = kp.data_ptr();
    a.v_pages = vp.data_ptr();
    a.bounds = address(bounds);
    a.page_table = static_cast<const int*>(table.data_ptr());
    a.start = static_cast<const int*>(start.data_ptr());
    a.cu = static_cast<const int*>(address(cu));
    a.pos = static_cast<const long long*>(address(pos));
    a.num_pages = c.pages;
    a.tokens = extent("tokens", T);
    a.batch = extent("batch", c.batch);
    a.heads = extent("heads", Hq);
    a.kv_heads = extent("kv_heads", c.hkv);
    a.d = extent("d", c.d);
    a.page_size = extent("page size", c.page);
    a.max_pages = extent("max_pages", c.max_pages);
    a.pairing = static_cast<int>(whole("pairing", o[14]));
    a.theta = number(o[7]);
    a.eps = static_cast<float>(number(o[12]));
    target.launch(f_append, a);
    if (q && o[16] == Py_None) return THPVariable_Wrap(q_new);
    return Py_NewRef(o[16]);
  });
}

const at::Tensor* scratch(PyObject* o, size_t need, const at::Tensor& like, at::Tensor* own) {
  const at::Tensor* ws = tensor("workspace", o, true);
  if (!ws) {
    *own = at::empty({static_cast<int64_t>(need < 16 ? 16 : need)}, like.options().dtype(at::kByte));
    return own;
  }
  if (!ws->is_contiguous()) throw Refusal{"workspace: a contiguous tensor is expected"};
  return ws;
}

// Queries [batch][heads][d]; returns the row stride.
long long queries(const at::Tensor& q, int64_t batch, int64_t d) {
  const long long stride = head_rows("q", q, at::kBFloat16, -1, d);
  if (q.size(0) != batch)
    throw Refusal{"q has " + std::to_string(q.size(0)) + " sequences, page_table " + std::to_string(batch)};
  return stride;
}

// q, k_pages, v_pages, page_table, kv_len, theta, alpha, selected, lse, out, workspace, stream
PyObject* paged_decode(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded("paged_decode", n, 12, [&]() -> PyObject* {
    const at::Tensor &q = *tensor("q", o[0]), &kp = *tensor("k_pages", o[1]), &vp = *tensor("v_pages", o[2]),
                     &table = *tensor("page_table", o[3]), &len = *tensor("kv_len", o[4]);
    const at::Tensor *sel = tensor("selected", o[7], true), *lse = tensor("lse", o[8], true),
                     *out = tensor("out", o[9], true);
    const Pool c(kp, vp, table);
    atf_paged_decode_args a{};
    a.q_stride = queries(q, c.batch, c.d);
    const int64_t Hq = q.size(1);
    dense("kv_len", len, at::kInt, {c.batch});
    if (sel) a.n_select = extent("n_select", dense("selected", *sel, at::kInt, {c.batch, c.hkv, -1}).size(2));
    const Target target(q, o[11]);
    at::Tensor out_new, ws_new;
    if (!out) out_new = at::empty({c.batch, Hq, c.d}, q.options()), out = &out_new;
    dense("out", *out, at::kBFloat16, {c.batch, Hq, c.d});
    if (lse) dense("lse", *lse, at::kFloat, {c.batch, Hq});
    a.batch = extent("batch", c.batch);
    a.heads = extent("heads", Hq);
    a.kv_heads = extent("kv_heads", c.hkv);
    a.d = extent("d", c.d);
    a.page_size = extent("page size", c.page);
    a.max_pages = extent("max_pages", c.max_pages);
    const at::Tensor& ws =
        *scratch(o[10], f_decode_bytes ? f_decode_bytes(a.batch, a.heads, a.kv_heads, a.d) : 0, q, &ws_new);
    on_device(q, {{"k_pages", &kp}, {"v_pages", &vp}, {"page_table", &table}, {"kv_len", &len}, {"selected", sel},
                  {"out", out}, {"lse", lse}, {"workspace", &ws}});
    a.q = q.data_ptr();
    a.k_pages = kp.data_ptr();
    a.v_pages = vp.data_ptr();
    a.page_table = static_cast<const int*>(table.data_ptr());
    a.kv_len = static_cast<const int*>(len.data_ptr());
    a.selected = static_cast<const int*>(address(sel));
    a.out = out->data_ptr();
    a.lse = static_cast<float*>(address(lse));
    a.num_pages = c.pages;
    a.theta = number(o[5]);
    a.alpha = number(o[6]);
    a.workspace = ws.data_ptr();
    a.workspace_bytes = ws.nbytes();
    target.launch(f_decode, a);
    return o[9] == Py_None ? THPVariable_Wrap(out_new) : Py_NewRef(o[9]);
  });
}

// q, bounds, page_table, kv_len, page_size, n_select, theta, alpha, n_first, n_last, selected, workspace, stream
PyObject* page_select(PyObject*, PyObject* const* o, Py_ssize_t n) {
  return guarded("page_select", n, 13, [&]() -> PyObject* {
    const at::Tensor &q = *tensor("q", o[0]), &bounds = *tensor("bounds", o[1]), &table = *tensor("page_table", o[2]),
                     &len = *tensor("kv_len", o[3]);
    const at::Tensor* sel = tensor("selected", o[10], true);
    if (bounds.dim() != 4) throw Refusal{"bounds: [pages][kv heads][2][d] is expected, got " + describe(bounds)};
    const int64_t N = bounds.size(0), Hkv = bounds.size(1), d = bounds.size(3);
    dense("bounds", bounds, at::kBFloat16, {N, Hkv, 2, d});
    dense("page_table", table, at::kInt, {-1, -1});
    const int64_t B = table.size(0), P = table.size(1);
    atf_page_select_args a{};
    a.q_stride = queries(q, B, d);
    dense("kv_len", len, at::kInt, {B});
    a.n_select = static_cast<int>(whole("n_select", o[5]));
    const Target target(q, o[12]);
    at::Tensor sel_new, ws_new;
    if (!sel) {
      if (a.n_select < 0) throw Refusal{"n_select " + std::to_string(a.n_select)};
      sel_new = at::empty({B, Hkv, a.n_select}, q.options().dtype(at::kInt)), sel = &sel_new;
    }
    dense("selected", *sel, at::kInt, {B, Hkv, a.n_select});
    a.batch = extent("batch", B);
    a.heads = extent("heads", q.size(1));
    a.kv_heads = extent("kv_heads", Hkv);
    a.d = extent("d", d);
    a.page_size = static_cast<int>(whole("page_size", o[4]));
    a.max_pages = extent("max_pages", P);
    a.n_first = static_cast<int>(whole("n_first", o[8]));
    a.n_last = static_cast<int>(whole("n_last", o[9]));
    const at::Tensor& ws = *scratch(o[11], f_select_bytes ? f_select_bytes(a.batch, a.kv_heads, a.max_pages) : 0, q, &ws_new);
    on_device(q, {{"bounds", &bounds}, {"page_table", &table}, {"kv_len", &len}, {"selected", sel}, {"workspace", &ws}});
    a.q = q.data_ptr();
    a.bounds = bounds.data_ptr();
    a.page_table = static_cast<const int*>(table.data_ptr());
    a.kv_len = static_cast<const int*>(len.data_ptr());
    a.selected = static_cast<int*>(sel->data_ptr());
    a.num_pages = N;
    a.theta = number(o[6]);
    a.alpha = number(o[7]);
    a.workspace = ws.data_ptr();
    a.workspace_bytes = ws.nbytes();
    target.launch(f_select, a);
    return o[10] == Py_None ? THPVariable_Wrap(sel_new) : Py_NewRef(o[10]);
  });
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyMethodDef def(const char* name, Fast f) { return {name, reinterpret_cast<PyCFunction>(f), METH_FASTCALL, nullptr}; }
PyMethodDef methods[] = {def("bind", bind), def("qk_norm_rope", qk_norm_rope), def("paged_append", paged_append),
                         def("paged_decode", paged_decode), def("page_select", page_select), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_calls(void) { return PyModule_Create(&module); }
