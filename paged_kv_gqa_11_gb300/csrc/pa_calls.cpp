// Python entry of the calls that run once per layer and step: norm + rotation,
// rotating append, cache reads, shared-prefix decode.
//
// The kernels behind them take a few microseconds; checking a dozen tensors and
// passing two dozen arguments through Python and ctypes took 8 to 20 (measured:
// 28 us a shared-prefix decode against 6.5 us for the library's call).  So the
// checks are made here, on the tensors themselves, and the library is called
// directly.  What may be refused is raised as the package's PaError before
// anything is launched: types, shapes, strides, devices here, the rest by the
// library.
//
// Nothing is kept from one call for the next.  Memory that a call needs comes
// from torch's allocator on the stream that the call runs on, so calls on several
// streams, and captured ones, each have their own.  What stands on a stream passed in
// is ordered there: the caller lets it wait for what makes the arguments, and waits for
// it before using the results elsewhere.
#include <Python.h>

#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ATen.h>

#include <initializer_list>
#include <optional>
#include <string>

#include "pa.h"

namespace {

constexpr int64_t kD = 256;
PyObject* g_error = nullptr;  // the package's PaError

struct Refused {
  int status;
  std::string what;
};

[[noreturn]] void refuse(const std::string& what, int status = PA_ERR_INVALID) { throw Refused{status, what}; }
void check(bool ok, const char* what) {
  if (!ok) refuse(what);
}

int dtype_of(const at::Tensor& x) {
  switch (x.scalar_type()) {
    case at::kFloat: return PA_DT_F32;
    case at::kHalf: return PA_DT_F16;
    case at::kBFloat16: return PA_DT_BF16;
    default: refuse(std::string("values of type ") + c10::toString(x.scalar_type()), PA_ERR_UNSUPPORTED);
  }
}

// A CUDA tensor, or (where it may be) an undefined one for None.
const at::Tensor& tensor(PyObject* o, const char* name, bool optional = false) {
  static const at::Tensor none;
  if (optional && o == Py_None) return none;
  if (!THPVariable_Check(o)) refuse(std::string(name) + ": a tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(std::string(name) + ": on a GPU");
  return t;
}

void on(int device, const at::Tensor& t, const char* name) {
  if (t.defined() && t.get_device() != device) refuse(std::string(name) + ": on the other tensors' device");
}

void index(const at::Tensor& t, int64_t n, const char* name) {
  if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    refuse(std::string(name) + ": int32 [" + std::to_string(n) + "]");
}

void block_table(const at::Tensor& t) {
  check(t.scalar_type() == at::kInt && t.dim() == 2 && t.is_contiguous(), "block_table: int32 [n_seq][pages], contiguous");
}

// Elements between rows of [n][heads][256] whose heads are packed (a single row's own
// length, whatever stride its tensor has there).
int64_t row_stride(const at::Tensor& x, const char* name) {
  if (x.dim() != 3 || x.size(2) != kD || x.stride(2) != 1 || (x.size(1) > 1 && x.stride(1) != kD))
    refuse(std::string(name) + ": rows [n][heads][256] of packed heads");
  return x.size(0) > 1 ? x.stride(0) : x.size(1) * kD;
}

void same_shape(const at::Tensor& a, const at::Tensor& b, const char* what) { check(a.sizes() == b.sizes(), what); }

int weight_type(const at::Tensor& a, const at::Tensor& b) {
  int t = PA_DT_F32;
  for (const at::Tensor* w : {&a, &b}) {
    if (!w->defined()) continue;
    check(w->dim() == 1 && w->size(0) == kD && w->is_contiguous(), "weights: [256]");
    t = dtype_of(*w);
  }
  check(!a.defined() || !b.defined() || a.scalar_type() == b.scalar_type(), "weights of one type");
  return t;
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// The device and stream of a call: both are current while this lives.
struct Place {
  std::optional<c10::cuda::CUDAGuard> device;
  std::optional<c10::cuda::CUDAStreamGuard> stream_guard;
  std::optional<c10::cuda::CUDAStream> other, current;  // a stream passed in that is not the current one, and that
  pa_stream_t stream;

  Place(int dev, PyObject* s) {
    if (s == Py_None) {
      device.emplace(static_cast<c10::DeviceIndex>(dev));
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
      return;
    }
    unsigned long long v = 0;
    if (PyLong_Check(s)) {
      v = PyLong_AsUnsignedLongLong(s);
    } else {
      PyObject* a = PyObject_GetAttrString(s, "cuda_stream");
      if (a) {
        v = PyLong_AsUnsignedLongLong(a);
        Py_DECREF(a);
      }
    }
    if (PyErr_Occurred()) {
      PyErr_Clear();
      refuse("stream: a torch stream or its address");
    }
    stream = reinterpret_cast<pa_stream_t>(v);
    const auto device_index = static_cast<c10::DeviceIndex>(dev);
    const auto passed = c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(v), device_index);
    const auto now = c10::cuda::getCurrentCUDAStream(device_index);
    if (passed.stream() != now.stream()) {
      other = passed;
      current = now;
    }
    stream_guard.emplace(passed);
  }

  // Tensors that the call reads or writes: torch's allocator gives their memory out again
  // only after what is on the stream by then.
  void uses(std::initializer_list<const at::Tensor*> tensors) const {
    if (!other) return;
    for (const at::Tensor* t : tensors)
      if (t->defined()) c10::cuda::CUDACachingAllocator::recordStream(t->storage().data_ptr(), *other);
  }

  // A result made on the stream passed in, which the caller will use on the current one.
  const at::Tensor& made(const at::Tensor& t) const {
    if (other) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), *current);
    return t;
  }
};

at::Tensor like(const at::Tensor& x, at::ScalarType t) { return at::empty(x.sizes(), x.options().dtype(t)); }

std::optional<at::ScalarType> dtype_arg(PyObject* o) {
  if (o == Py_None) return std::nullopt;
  if (!THPDtype_Check(o)) refuse("dtype: a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

void* address(PyObject* o, const char* name) {
  void* p = PyLong_AsVoidPtr(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + ": an address");
  }
  return p;
}

void status(pa_status s, const char* what) {
  if (s != PA_OK) refuse(what, s);
}

PyObject* wrap(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  PyObject* x = wrap(a);
  PyObject* y = wrap(b);
  PyObject* r = PyTuple_Pack(2, x, y);
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// Runs a call's body: refusals become PaError, anything else a RuntimeError.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& body) {
  try {
    if (n != want) refuse("wrong number of arguments");
    return body();
  } catch (const Refused& r) {
    PyErr_Clear();  // of a conversion whose result was then refused
    PyObject* e = PyObject_CallFunction(g_error ? g_error : PyExc_RuntimeError, "is", r.status, r.what.c_str());
    if (e) {
      PyErr_SetObject(reinterpret_cast<PyObject*>(Py_TYPE(e)), e);
      Py_DECREF(e);
    }
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (rope, q, k, row_pos, q_weight, k_weight, q_out, k_out, out_dtype, stream) -> (q_out, k_out)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 10, [&]() -> PyObject* {
    const auto* rope = static_cast<const pa_rope_desc*>(address(a[0], "rope"));
    const at::Tensor &q = tensor(a[1], "q", true), &k = tensor(a[2], "k", true), &pos = tensor(a[3], "row_pos"),
                     &wq = tensor(a[4], "q_weight", true), &wk = tensor(a[5], "k_weight", true);
    at::Tensor qo = tensor(a[6], "q_out", true), ko = tensor(a[7], "k_out", true);
    check(q.defined() || k.defined(), "q or k");
    const at::Tensor& some = q.defined() ? q : k;
    check(some.dim() == 3, "rows [n][heads][256]");
    const int64_t n = some.size(0);
    const int dev = some.get_device();
    index(pos, n, "row_pos");
    on(dev, pos, "row_pos"); on(dev, k, "k"); on(dev, wq, "q_weight"); on(dev, wk, "k_weight");
    on(dev, qo, "q_out"); on(dev, ko, "k_out");
    check(!k.defined() || (k.scalar_type() == some.scalar_type() && k.dim() == 3 && k.size(0) == n), "q and k of one type and row count");
    check((q.defined() || !qo.defined()) && (k.defined() || !ko.defined()), "an output without its input");
    const auto want = dtype_arg(a[8]);
    const at::ScalarType type = want ? *want : qo.defined() ? qo.scalar_type() : ko.defined() ? ko.scalar_type() : some.scalar_type();
    const Place place(dev, a[9]);
    place.uses({&q, &k, &pos, &wq, &wk, &qo, &ko});
    if (q.defined() && !qo.defined()) qo = place.made(like(q, type));
    if (k.defined() && !ko.defined()) ko = place.made(like(k, type));
    int64_t s[4] = {0, 0, 0, 0}, h[2] = {0, 0};
    const at::Tensor *in[2] = {&q, &k}, *out[2] = {&qo, &ko};
    for (int i = 0; i < 2; ++i) {
      if (!in[i]->defined()) continue;
      same_shape(*in[i], *out[i], "outputs of the inputs' shape");
      check(out[i]->scalar_type() == type, "outputs of one type");
      s[2 * i] = row_stride(*in[i], "q, k");
      s[2 * i + 1] = row_stride(*out[i], "outputs");
      h[i] = in[i]->size(1);
    }
    check(n <= UINT32_MAX, "rows");
    const int it = dtype_of(some), ot = dtype_of(qo.defined() ? qo : ko);
    if (n > 0)
      status(pa_norm_rope(rope, ptr(q), s[0], (uint32_t)h[0], ptr(k), s[2], (uint32_t)h[1], it, ptr(wq), ptr(wk), weight_type(wq, wk),
                          pos.data_ptr<int32_t>(), (uint32_t)n, ptr(qo), s[1], ptr(ko), s[3], ot, place.stream),
             "pa_norm_rope");
    return pair(qo, ko);
  });
}

// (pool, n_kv_heads, k_pool, v_pool, rope, k, v, row_seq, row_pos, table, k_weight, q, q_weight, q_out, q_dtype, err,
//  stream) -> q_out
PyObject* append_rope(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 17, [&]() -> PyObject* {
    const auto* pool = static_cast<const pa_pool*>(address(a[0], "pool"));
    const int64_t heads = PyLong_AsLongLong(a[1]);
    const at::Tensor &kp = tensor(a[2], "k_pool"), &vp = tensor(a[3], "v_pool"), &k = tensor(a[5], "k"), &v = tensor(a[6], "v"),
                     &seq = tensor(a[7], "row_seq"), &pos = tensor(a[8], "row_pos"), &table = tensor(a[9], "block_table"),
                     &wk = tensor(a[10], "k_weight", true), &q = tensor(a[11], "q", true), &wq = tensor(a[12], "q_weight", true),
                     &err = tensor(a[15], "err");
    const auto* rope = static_cast<const pa_rope_desc*>(address(a[4], "rope"));
    at::Tensor qo = tensor(a[13], "q_out", true);
    const int dev = kp.get_device();
    check(k.dim() == 3 && k.size(1) == heads, "k: rows [n][n_kv_heads][256]");
    const int64_t n = k.size(0);
    same_shape(k, v, "v: rows of k's shape");
    check(k.scalar_type() == v.scalar_type(), "k and v of one type");
    index(seq, n, "row_seq");
    index(pos, n, "row_pos");
    block_table(table);
    on(dev, vp, "v_pool"); on(dev, k, "k"); on(dev, v, "v"); on(dev, seq, "row_seq"); on(dev, pos, "row_pos");
    on(dev, table, "block_table"); on(dev, wk, "k_weight"); on(dev, q, "q"); on(dev, wq, "q_weight"); on(dev, qo, "q_out"); on(dev, err, "err");
    const auto want = dtype_arg(a[14]);
    const Place place(dev, a[16]);
    place.uses({&kp, &vp, &k, &v, &seq, &pos, &table, &wk, &q, &wq, &qo, &err});
    int64_t qs = 0, qos = 0, hq = 0;
    if (q.defined()) {
      check(q.dim() == 3 && q.size(0) == n && q.scalar_type() == k.scalar_type(), "q of k's type and row count");
      if (!qo.defined()) qo = place.made(like(q, want ? *want : q.scalar_type()));
      same_shape(q, qo, "q_out of q's shape");
      check(!want || qo.scalar_type() == *want, "q_out of q_dtype");
      qs = row_stride(q, "q");
      qos = row_stride(qo, "q_out");
      hq = q.size(1);
    } else {
      check(!qo.defined(), "q_out without q");
    }
    check(n <= UINT32_MAX && table.size(0) <= UINT32_MAX && table.size(1) <= INT32_MAX, "rows and table");
    const int it = dtype_of(k), ot = qo.defined() ? dtype_of(qo) : it;
    if (n > 0)
      status(pa_append_rows_rope(pool, ptr(kp), ptr(vp), rope, ptr(k), row_stride(k, "k"), ptr(v), row_stride(v, "v"), it, ptr(wk),
                                 weight_type(wq, wk), ptr(q), qs, (uint32_t)hq, ptr(wq), ptr(qo), qos, ot, seq.data_ptr<int32_t>(),
                                 pos.data_ptr<int32_t>(), (uint32_t)n, table.data_ptr<int32_t>(), (uint32_t)table.size(1),
                                 (uint32_t)table.size(0), err.data_ptr<int32_t>(), place.stream),
             "pa_append_rows_rope");
    return wrap(qo);
  });
}

// (pool, n_kv_heads, k_pool, v_pool, row_seq, row_pos, table, dtype, k_out, v_out, err, stream) -> (k_out, v_out)
PyObject* read_rows(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 12, [&]() -> PyObject* {
    const auto* pool = static_cast<const pa_pool*>(address(a[0], "pool"));
    const int64_t heads = PyLong_AsLongLong(a[1]);
    const at::Tensor &kp = tensor(a[2], "k_pool"), &vp = tensor(a[3], "v_pool"), &seq = tensor(a[4], "row_seq"), &pos = tensor(a[5], "row_pos"),
                     &table = tensor(a[6], "block_table"), &err = tensor(a[10], "err");
    at::Tensor ko = tensor(a[8], "k_out", true), vo = tensor(a[9], "v_out", true);
    const int dev = kp.get_device();
    const int64_t n = seq.dim() == 1 ? seq.size(0) : 0;
    index(seq, n, "row_seq");
    index(pos, n, "row_pos");
    block_table(table);
    on(dev, vp, "v_pool"); on(dev, seq, "row_seq"); on(dev, pos, "row_pos"); on(dev, table, "block_table");
    on(dev, ko, "k_out"); on(dev, vo, "v_out"); on(dev, err, "err");
    const auto want = dtype_arg(a[7]);
    const Place place(dev, a[11]);
    place.uses({&kp, &vp, &seq, &pos, &table, &ko, &vo, &err});
    if (!ko.defined() && !vo.defined()) {
      const auto opt = kp.options().dtype(want ? *want : at::kHalf);
      ko = place.made(at::empty({n, heads, kD}, opt));
      vo = place.made(at::empty({n, heads, kD}, opt));
    }
    const at::Tensor& some = ko.defined() ? ko : vo;
    for (const at::Tensor* x : {&ko, &vo})
      check(!x->defined() || (x->dim() == 3 && x->size(0) == n && x->size(1) == heads && x->size(2) == kD && x->is_contiguous() &&
                              x->scalar_type() == some.scalar_type()),
            "outputs [n][n_kv_heads][256] of one type, contiguous");
    check(n <= UINT32_MAX && table.size(0) <= UINT32_MAX && table.size(1) <= INT32_MAX, "rows and table");
    const int ot = dtype_of(some);
    if (n > 0)
      status(pa_read_rows(pool, ptr(kp), ptr(vp), seq.data_ptr<int32_t>(), pos.data_ptr<int32_t>(), (uint32_t)n, table.data_ptr<int32_t>(),
                          (uint32_t)table.size(1), (uint32_t)table.size(0), ptr(ko), ptr(vo), ot, err.data_ptr<int32_t>(), place.stream),
             "pa_read_rows");
    return pair(ko, vo);
  });
}

// A host array of 32-bit whole numbers, held while this lives.
struct Ints {
  Py_buffer b{};
  bool held = false;
  Ints(PyObject* o, const char* name) {
    held = PyObject_GetBuffer(o, &b, PyBUF_C_CONTIGUOUS | PyBUF_FORMAT) == 0;
    if (!held) PyErr_Clear();
    const char* f = held ? b.format : nullptr;
    if (f && (*f == '<' || *f == '=' || *f == '@')) ++f;
    if (!held || b.ndim != 1 || b.itemsize != 4 || !f || !(*f == 'i' || *f == 'I' || *f == 'l' || *f == 'L')) {
      if (held) PyBuffer_Release(&b);
      held = false;
      refuse(std::string(name) + ": a contiguous host array of 32-bit whole numbers");
    }
  }
  ~Ints() {
    if (held) PyBuffer_Release(&b);
  }
  int64_t size() const { return b.shape ? b.shape[0] : b.len / 4; }
};

// (pool, q, k_pool, v_pool, table, seq_lens_dev, seq_lens_host, group_sizes, prefix_lens, n_qtok, scale, out, lse,
//  want_lse, workspace, err, stream) -> (out, lse)
PyObject* decode_prefix(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 17, [&]() -> PyObject* {
    const auto* pool = static_cast<const pa_pool*>(address(a[0], "pool"));
    const at::Tensor &q = tensor(a[1], "q"), &kp = tensor(a[2], "k_pool"), &vp = tensor(a[3], "v_pool"), &table = tensor(a[4], "block_table"),
                     &lens_dev = tensor(a[5], "seq_lens_dev"), &err = tensor(a[15], "err");
    const Ints lens(a[6], "seq_lens_host"), sizes(a[7], "group_sizes"), pre(a[8], "prefix_lens");
    at::Tensor out = tensor(a[11], "out", true), lse = tensor(a[12], "lse", true), ws = tensor(a[14], "workspace", true);
    const int dev = kp.get_device();
    check(q.dim() == 4 && q.size(1) == PyLong_AsLongLong(a[9]) && q.size(3) == kD && q.is_contiguous(),
          "q [n_seq][n_qtok][heads][256], contiguous");
    const int64_t n = q.size(0), t = q.size(1), hq = q.size(2), g = sizes.size();
    block_table(table);
    index(lens_dev, n, "seq_lens_dev");
    check(lens.size() == n && table.size(0) == n, "a table row and a length per sequence");
    check(pre.size() == g, "a size and a prefix per group");
    on(dev, q, "q"); on(dev, vp, "v_pool"); on(dev, table, "block_table"); on(dev, lens_dev, "seq_lens_dev"); on(dev, out, "out");
    on(dev, lse, "lse"); on(dev, ws, "workspace"); on(dev, err, "err");
    check(n <= UINT32_MAX && g <= UINT32_MAX && t <= UINT32_MAX && hq <= UINT32_MAX && table.size(1) <= INT32_MAX, "sizes");
    const Place place(dev, a[16]);
    place.uses({&q, &kp, &vp, &table, &lens_dev, &out, &lse, &ws, &err});
    if (!out.defined()) out = place.made(like(q, q.scalar_type()));
    if (!lse.defined() && PyObject_IsTrue(a[13]) == 1) lse = place.made(at::empty({n, t, hq}, q.options().dtype(at::kFloat)));
    same_shape(q, out, "out of q's shape");
    check(out.is_contiguous(), "out: contiguous");
    check(!lse.defined() || (lse.scalar_type() == at::kFloat && lse.is_contiguous() && lse.dim() == 3 && lse.size(0) == n && lse.size(1) == t &&
                             lse.size(2) == hq),
          "lse: float32 [n_seq][n_qtok][heads]");
    if (!ws.defined())
      ws = at::empty({(int64_t)pa_decode_prefix_workspace_size(pool, (uint32_t)n, (uint32_t)g, (uint32_t)t, dev)}, kp.options().dtype(at::kByte));
    check(ws.is_contiguous(), "workspace: contiguous");
    status(pa_decode_prefix(pool, ptr(q), dtype_of(q), ptr(kp), ptr(vp), table.data_ptr<int32_t>(), (uint32_t)table.size(1),
                            lens_dev.data_ptr<int32_t>(), static_cast<const int32_t*>(lens.b.buf), (uint32_t)n,
                            static_cast<const uint32_t*>(sizes.b.buf), static_cast<const int32_t*>(pre.b.buf), (uint32_t)g, (uint32_t)t,
                            (uint32_t)hq, (float)PyFloat_AsDouble(a[10]), ptr(out), dtype_of(out), lse.defined() ? lse.data_ptr<float>() : nullptr,
                            ptr(ws), (size_t)ws.nbytes(), err.data_ptr<int32_t>(), place.stream),
           "pa_decode_prefix");
    return pair(out, lse);
  });
}

uint32_t count_arg(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (PyErr_Occurred() || v < 0 || v > UINT32_MAX) {
    PyErr_Clear();
    refuse(std::string(name) + ": a whole number from 0 on");
  }
  return (uint32_t)v;
}

float float_arg(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + ": a number");
  }
  return (float)v;
}

// (pool, q, k_pool, v_pool, table, seq_lens_dev, seq_lens_host, n_new, window, sinks, scale, out, lse, want_lse, workspace,
//  err, stream) -> (out, lse)
PyObject* attend_window(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 17, [&]() -> PyObject* {
    const auto* pool = static_cast<const pa_pool*>(address(a[0], "pool"));
    const at::Tensor &q = tensor(a[1], "q"), &kp = tensor(a[2], "k_pool"), &vp = tensor(a[3], "v_pool"), &table = tensor(a[4], "block_table"),
                     &lens_dev = tensor(a[5], "seq_lens_dev"), &err = tensor(a[15], "err");
    const Ints lens(a[6], "seq_lens_host"), n_new(a[7], "n_new");
    const uint32_t window = count_arg(a[8], "window"), sinks = count_arg(a[9], "sinks");
    const float scale = float_arg(a[10], "scale");
    at::Tensor out = tensor(a[11], "out", true), lse = tensor(a[12], "lse", true), ws = tensor(a[14], "workspace", true);
    const int dev = kp.get_device();
    block_table(table);
    const int64_t n = table.size(0);
    index(lens_dev, n, "seq_lens_dev");
    check(lens.size() == n && n_new.size() == n, "a table row, a length and a number of new tokens per sequence");
    const int64_t qs = row_stride(q, "q"), rows = q.size(0), hq = q.size(1);
    const auto* fresh = static_cast<const int32_t*>(n_new.b.buf);
    int64_t tokens = 0;
    for (int64_t i = 0; i < n; ++i) {
      check(fresh[i] >= 0, "n_new: from 0 on");
      tokens += fresh[i];
    }
    check(tokens <= rows, "q: a row per new token");
    on(dev, q, "q"); on(dev, vp, "v_pool"); on(dev, table, "block_table"); on(dev, lens_dev, "seq_lens_dev"); on(dev, out, "out");
    on(dev, lse, "lse"); on(dev, ws, "workspace"); on(dev, err, "err");
    check(n <= UINT32_MAX && hq <= UINT32_MAX && table.size(1) <= INT32_MAX, "sizes");
    const Place place(dev, a[16]);
    place.uses({&q, &kp, &vp, &table, &lens_dev, &out, &lse, &ws, &err});
    if (!out.defined()) {
      out = place.made(at::empty({rows, hq, kD}, q.options()));
      if (tokens < rows) out.narrow(0, tokens, rows - tokens).zero_();
    }
    const int want = PyObject_IsTrue(a[13]);
    if (want < 0) PyErr_Clear();
    if (!lse.defined() && want == 1) {
      lse = place.made(at::empty({rows, hq}, q.options().dtype(at::kFloat)));
      if (tokens < rows) lse.narrow(0, tokens, rows - tokens).zero_();
    }
    same_shape(q, out, "out of q's shape");
    check(!lse.defined() || (lse.scalar_type() == at::kFloat && lse.is_contiguous() && lse.dim() == 2 && lse.size(0) == rows && lse.size(1) == hq),
          "lse: float32 [tokens][heads], contiguous");
    if (tokens > 0 && !ws.defined())
      ws = at::empty({(int64_t)pa_attend_window_workspace_size(pool, static_cast<const int32_t*>(lens.b.buf), fresh, (uint32_t)n, window,
                                                               sinks, dev)},
                     kp.options().dtype(at::kByte));
    check(!ws.defined() || ws.is_contiguous(), "workspace: contiguous");
    const int qt = dtype_of(q), ot = dtype_of(out);
    const int64_t os = row_stride(out, "out");
    status(pa_attend_window(pool, ptr(q), qs, qt, ptr(kp), ptr(vp), table.data_ptr<int32_t>(), (uint32_t)table.size(1),
                            lens_dev.data_ptr<int32_t>(), static_cast<const int32_t*>(lens.b.buf), fresh, (uint32_t)n, (uint32_t)hq, window,
                            sinks, scale, ptr(out), os, ot, lse.defined() ? lse.data_ptr<float>() : nullptr, ptr(ws),
                            ws.defined() ? (size_t)ws.nbytes() : 0, err.data_ptr<int32_t>(), place.stream),
           "pa_attend_window");
    return pair(out, lse);
  });
}

// (pool, k_pool, v_pool, rope, rope_from, src_seq, src_pos, dst_seq, dst_pos, table, dst_table, disjoint, workspace, err,
//  stream) -> None
PyObject* move_rows(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 15, [&]() -> PyObject* {
    const auto* pool = static_cast<const pa_pool*>(address(a[0], "pool"));
    const at::Tensor &kp = tensor(a[1], "k_pool"), &vp = tensor(a[2], "v_pool"), &from_seq = tensor(a[5], "src_seq"),
                     &from = tensor(a[6], "src_pos"), &to_seq = tensor(a[7], "dst_seq"), &to = tensor(a[8], "dst_pos"),
                     &table = tensor(a[9], "block_table"), &other = tensor(a[10], "dst_table", true), &err = tensor(a[13], "err");
    const auto* rope = static_cast<const pa_rope_desc*>(address(a[3], "rope"));
    const auto* was = static_cast<const pa_rope_desc*>(address(a[4], "rope_from"));
    at::Tensor ws = tensor(a[12], "workspace", true);
    const int dev = kp.get_device();
    const int64_t n = from_seq.dim() == 1 ? from_seq.size(0) : 0;
    index(from_seq, n, "src_seq"); index(from, n, "src_pos"); index(to_seq, n, "dst_seq"); index(to, n, "dst_pos");
    block_table(table);
    if (other.defined()) block_table(other);
    const at::Tensor& dst_table = other.defined() ? other : table;
    on(dev, vp, "v_pool"); on(dev, from_seq, "src_seq"); on(dev, from, "src_pos"); on(dev, to_seq, "dst_seq"); on(dev, to, "dst_pos");
    on(dev, table, "block_table"); on(dev, other, "dst_table"); on(dev, ws, "workspace"); on(dev, err, "err");
    const int disjoint = PyObject_IsTrue(a[11]);
    if (disjoint < 0) {
      PyErr_Clear();
      refuse("disjoint: true or false");
    }
    check(n <= UINT32_MAX && table.size(0) <= INT32_MAX && table.size(1) <= INT32_MAX && dst_table.size(0) <= INT32_MAX &&
              dst_table.size(1) <= INT32_MAX,
          "rows and tables");
    const Place place(dev, a[14]);
    place.uses({&kp, &vp, &from_seq, &from, &to_seq, &to, &table, &other, &ws, &err});
    if (!disjoint && !ws.defined()) {
      const size_t bytes = pa_move_rows_workspace_size(pool, (uint32_t)n);
      if (bytes > 0) ws = at::empty({(int64_t)bytes}, kp.options().dtype(at::kByte));
    }
    check(!ws.defined() || ws.is_contiguous(), "workspace: contiguous");
    status(pa_move_rows(pool, ptr(kp), ptr(vp), rope, was, from_seq.data_ptr<int32_t>(), from.data_ptr<int32_t>(), to_seq.data_ptr<int32_t>(),
                        to.data_ptr<int32_t>(), (uint32_t)n, table.data_ptr<int32_t>(), (uint32_t)table.size(1), (uint32_t)table.size(0),
                        dst_table.data_ptr<int32_t>(), (uint32_t)dst_table.size(1), (uint32_t)dst_table.size(0), disjoint, ptr(ws),
                        ws.defined() ? (size_t)ws.nbytes() : 0, err.data_ptr<int32_t>(), place.stream),
           "pa_move_rows");
    Py_RETURN_NONE;
  });
}

// (pool, k_pool, v_pool, src, dst, table, table_out, err, stream) -> table_out
PyObject* move_blocks(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  return guarded(n_args, 9, [&]() -> PyObject* {
    const auto* pool = static_cast<const pa_pool*>(address(a[0], "pool"));
    const at::Tensor &kp = tensor(a[1], "k_pool"), &vp = tensor(a[2], "v_pool"), &src = tensor(a[3], "src"), &dst = tensor(a[4], "dst"),
                     &table = tensor(a[5], "block_table", true), &err = tensor(a[7], "err");
    at::Tensor out = tensor(a[6], "table_out", true);
    const int dev = kp.get_device();
    const int64_t n = src.dim() == 1 ? src.size(0) : 0;
    index(src, n, "src"); index(dst, n, "dst");
    if (table.defined()) block_table(table);
    check(table.defined() || !out.defined(), "table_out without block_table");
    on(dev, vp, "v_pool"); on(dev, src, "src"); on(dev, dst, "dst"); on(dev, table, "block_table"); on(dev, out, "table_out"); on(dev, err, "err");
    check(n <= INT32_MAX, "blocks");
    const Place place(dev, a[8]);
    place.uses({&kp, &vp, &src, &dst, &table, &out, &err});
    if (table.defined() && !out.defined()) out = place.made(at::empty(table.sizes(), table.options()));
    if (out.defined()) {
      same_shape(table, out, "table_out of the table's shape");
      check(out.scalar_type() == at::kInt && out.is_contiguous(), "table_out: int32, contiguous");
    }
    status(pa_move_blocks(pool, ptr(kp), ptr(vp), src.data_ptr<int32_t>(), dst.data_ptr<int32_t>(), (uint32_t)n,
                          table.defined() ? table.data_ptr<int32_t>() : nullptr, out.defined() ? out.data_ptr<int32_t>() : nullptr,
                          table.defined() ? (uint64_t)table.numel() : 0, err.data_ptr<int32_t>(), place.stream),
           "pa_move_blocks");
    return wrap(out);
  });
}

PyObject* set_error(PyObject*, PyObject* e) {
  Py_INCREF(e);
  Py_XDECREF(g_error);
  g_error = e;
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(norm_rope)), METH_FASTCALL, ""},
    {"append_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(append_rope)), METH_FASTCALL, ""},
    {"read_rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(read_rows)), METH_FASTCALL, ""},
    {"decode_prefix", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(decode_prefix)), METH_FASTCALL, ""},
    {"attend_window", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(attend_window)), METH_FASTCALL, ""},
    {"move_rows", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(move_rows)), METH_FASTCALL, ""},
    {"move_blocks", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(move_blocks)), METH_FASTCALL, ""},
    {"set_error", set_error, METH_O, ""},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "pa_calls", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit_pa_calls() { return PyModule_Create(&g_module); }
