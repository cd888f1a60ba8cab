// Torch front end of the operators around the mixer (see include/gdr.h).
//
// A decode loop calls these operators once per layer and token, and their
// kernels take a few microseconds.  Checks, allocation and marshalling in Python
// took 12 us a call beside the launch's 4 (pooled step); here they take about 2, so this
// part is compiled: it looks at the tensors, allocates what the caller did not
// pass, and calls the C ABI with raw pointers.  It holds no arithmetic and no
// state but the ABI's addresses.
//
// The functions take every argument by position (binding.py gives them names,
// defaults and documentation) and return the status of the ABI call as an int
// where it is not GDR_OK.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/Stream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <exception>
#include <string>

#include "gdr.h"

namespace {

struct Abi {
  decltype(&gdr_step_slots) step_slots;
  decltype(&gdr_slot_map) slot_map;
  decltype(&gdr_group_norm_fwd) group_norm_fwd;
  decltype(&gdr_group_norm_bwd) group_norm_bwd;
  decltype(&gdr_group_norm_bwd_workspace_bytes) group_norm_bwd_ws;
  decltype(&gdr_prologue_fwd) prologue_fwd;
  decltype(&gdr_prologue_bwd) prologue_bwd;
  decltype(&gdr_prologue_bwd_workspace_bytes) prologue_bwd_ws;
} abi;

// A refused argument: becomes the Python exception `type`.
struct Refused : std::exception {
  PyObject *type;
  std::string text;
  Refused(PyObject *t, std::string s) : type(t), text(std::move(s)) {}
  const char *what() const noexcept override { return text.c_str(); }
};

[[noreturn]] void refuse(PyObject *type, const char *fmt, ...) {
  char buf[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  throw Refused(type, buf);
}

std::string text(at::IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + ")";
}

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

// The first tensor of a call: what the others have to go with.
const at::Tensor &first_tensor(PyObject *o, const char *name, int64_t least_dims,
                               const char *layout) {
  const at::Tensor &t = tensor(o, name);
  if (t.dim() < least_dims) refuse(PyExc_ValueError, "%s must be a %s tensor", name, layout);
  if (!t.is_cuda())
    refuse(PyExc_ValueError, "%s must be on a CUDA device (no CPU path exists)", name);
  return t;
}

void look(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef size,
          c10::Device device) {
  if (!t.is_cuda())
    refuse(PyExc_ValueError, "%s must be on a CUDA device (no CPU path exists)", name);
  if (t.device() != device)
    refuse(PyExc_ValueError, "%s is on %s, expected %s", name, t.device().str().c_str(),
           device.str().c_str());
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, "%s has dtype %s, expected %s", name, c10::toString(t.scalar_type()),
           c10::toString(type));
  if (t.sizes() != size)
    refuse(PyExc_ValueError, "%s has shape %s, expected %s", name, text(t.sizes()).c_str(),
           text(size).c_str());
}

// A dense tensor of this type and shape.
template <typename P = void>
P *dense(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef size,
         c10::Device device) {
  const at::Tensor &t = tensor(o, name);
  look(t, name, type, size, device);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
  return static_cast<P *>(t.data_ptr());
}

template <typename P = void>
P *dense_or_null(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef size,
                 c10::Device device) {
  return o == Py_None ? nullptr : dense<P>(o, name, type, size, device);
}

// Elements between the rows of t [..., H, d]: the last two dimensions are
// dense, those before them advance by one distance (a slice of a fused
// projection, for example).
int64_t row_stride(const at::Tensor &t, const char *name) {
  const auto size = t.sizes();
  const auto stride = t.strides();
  const int64_t n = t.dim(), width = size[n - 1] * size[n - 2];
  if (t.is_contiguous()) return width;
  bool ok = (size[n - 1] == 1 || stride[n - 1] == 1) &&
            (size[n - 2] == 1 || stride[n - 2] == size[n - 1]);
  int64_t row = -1, count = 1;  // count: rows of the dimensions behind this one
  for (int64_t i = n - 3; i >= 0; --i) {
    if (size[i] == 1) continue;
    if (row < 0) row = stride[i];
    ok = ok && stride[i] == row * count;
    count *= size[i];
  }
  if (!ok || (row >= 0 && row < width))
    refuse(PyExc_ValueError,
           "%s must have dense last two dimensions and rows one distance apart (strides %s of "
           "shape %s)",
           name, text(stride).c_str(), text(size).c_str());
  return row < 0 ? width : row;
}

gdr_dtype in_dtype(const at::Tensor &t, const char *name) {
  if (t.scalar_type() == at::kBFloat16) return GDR_BF16;
  if (t.scalar_type() == at::kFloat) return GDR_F32;
  refuse(PyExc_TypeError, "%s dtype must be bfloat16 or float32, got %s", name,
         c10::toString(t.scalar_type()));
}

int64_t whole(PyObject *o, const char *name, int64_t least, int64_t most) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, "%s must be a whole number", name);
  }
  if (v < least || v > most)
    refuse(PyExc_ValueError, "%s must be in [%lld, %lld], got %lld", name, (long long)least,
           (long long)most, v);
  return v;
}

bool flag(PyObject *o, const char *name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse(PyExc_TypeError, "%s must be a truth value", name);
  }
  return v;
}

float real(PyObject *o, const char *name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, "%s must be a number", name);
  }
  return static_cast<float>(v);
}

int fits(int64_t v, const char *name) {
  if (v > INT32_MAX) refuse(PyExc_ValueError, "%s is too large (%lld)", name, (long long)v);
  return static_cast<int>(v);
}

// The device of a call made current, its stream, and what it allocates: from
// the memory of the call's own stream, on which alone the order of a block's last
// user and of the kernel that writes it next is given; what the caller gets is
// kept, once freed, until the current stream is done with it too.
class Call {
 public:
  Call(c10::Device device, PyObject *stream)
      : guard_(device), stream_(c10::cuda::getCurrentCUDAStream(device.index())),
        caller_(stream_) {
    if (stream == Py_None) return;
    if (!THPStream_Check(stream)) refuse(PyExc_TypeError, "stream must be a torch.cuda.Stream");
    const auto *s = reinterpret_cast<THPStream *>(stream);
    if (s->device_type != static_cast<int64_t>(c10::DeviceType::CUDA) ||
        s->device_index != device.index())
      refuse(PyExc_ValueError, "stream is on device %lld, the tensors are on %s",
             (long long)s->device_index, device.str().c_str());
    const auto given = c10::cuda::CUDAStream(
        c10::Stream::unpack3(s->stream_id, s->device_index, c10::DeviceType::CUDA));
    stream_ = given;
  }

  at::Tensor make(at::IntArrayRef size, at::ScalarType type) {
    if (stream_ == caller_) return empty(size, type);
    const c10::cuda::CUDAStreamGuard of_the_call(stream_);
    at::Tensor t = empty(size, type);
    if (t.numel()) t.record_stream(caller_.unwrap());
    return t;
  }

  // The caller's `o`, looked at, or a new tensor.
  at::Tensor given_or_made(PyObject *o, const char *name, at::IntArrayRef size,
                           at::ScalarType type) {
    if (o == Py_None) return make(size, type);
    dense(o, name, type, size, guard_.current_device());
    return THPVariable_Unpack(o);
  }

  // The caller's workspace of any type, or a new one.
  std::pair<at::Tensor, size_t> workspace(PyObject *o, size_t need) {
    if (o == Py_None) return {make({static_cast<int64_t>(need)}, at::kByte), need};
    const at::Tensor &t = tensor(o, "workspace");
    if (t.device() != guard_.current_device() || !t.is_contiguous())
      refuse(PyExc_ValueError, "workspace must be a contiguous tensor on the inputs' device");
    return {t, t.nbytes()};
  }

  gdr_stream_t stream() const { return reinterpret_cast<gdr_stream_t>(stream_.stream()); }

 private:
  at::Tensor empty(at::IntArrayRef size, at::ScalarType type) const {
    // at::empty's own way where somebody looks at it (a dispatch mode) or fills new memory;
    // else without the dispatcher: 1 us of 2.
    if (c10::impl::dispatch_mode_enabled() || at::globalContext().deterministicAlgorithms())
      return at::empty(size, at::TensorOptions(type).device(guard_.current_device()));
    return at::detail::empty_cuda(size, type, guard_.current_device(), std::nullopt);
  }

  c10::cuda::CUDAGuard guard_;
  c10::cuda::CUDAStream stream_, caller_;  // the call's, and the one that is current
};

// n elements of a new one-dimensional tensor's memory, from `at` on.
at::Tensor piece(const at::Tensor &whole, int64_t at, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()),
                                                          whole.key_set(), whole.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return t;
}

PyObject *wrap(const at::Tensor &t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

PyObject *entry(PyObject *dict, const char *name) {
  PyObject *v = PyDict_GetItemString(dict, name);  // (borrowed)
  if (!v) refuse(PyExc_KeyError, "out has no entry %s", name);
  return v;
}

// A call's results: a new dict, or the caller's, whose entries that were None become the
// tensors made for them.
PyObject *dictionary(PyObject *given,
                     std::initializer_list<std::pair<const char *, const at::Tensor &>> items) {
  PyObject *d = given;
  if (given == Py_None)
    d = PyDict_New();
  else
    Py_INCREF(given);
  for (const auto &it : items) {
    if (d == given && !(it.second.defined() && PyDict_GetItemString(d, it.first) == Py_None))
      continue;
    PyObject *v = wrap(it.second);
    PyDict_SetItemString(d, it.first, v);
    Py_DECREF(v);
  }
  return d;
}

void check_out(PyObject *out) {
  if (out != Py_None && !PyDict_Check(out)) refuse(PyExc_TypeError, "out must be a dict");
}

// Runs `f` on exactly `n` arguments and turns what it throws into a Python error.
template <typename F>
PyObject *guarded(Py_ssize_t have, Py_ssize_t n, F f) {
  if (have != n) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", n, have);
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused &r) {
    PyErr_SetString(r.type, r.what());
  } catch (...) {  // torch's own errors (out of memory, ...)
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// The interpreter is free for other threads while a launch may wait for room.
template <typename F>
gdr_status launch(F f) {
  struct Free {
    PyThreadState *state = PyEval_SaveThread();
    ~Free() { PyEval_RestoreThread(state); }
  } free;
  return f();
}

// q, k, v, g, beta, pool, src, dst, cu_seqlens, gate_scale, norm_q, norm_k, o, stream
PyObject *step_slots(PyObject *, PyObject *const *x, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject * {
    const at::Tensor &q = first_tensor(x[0], "q", 3, "[total, Hk, dk]");
    const at::Tensor &v = first_tensor(x[2], "v", 3, "[total, H, dv]");
    if (q.dim() != 3 || v.dim() != 3) refuse(PyExc_ValueError, "q and v must have 3 dimensions");
    const auto dev = q.device();
    const auto type = q.scalar_type();
    const gdr_dtype dt = in_dtype(q, "q/k/v");
    const int64_t total = q.size(0), Hk = q.size(1), dk = q.size(2), H = v.size(1), dv = v.size(2);
    const at::Tensor &k = tensor(x[1], "k");
    look(k, "k", type, q.sizes(), dev);
    look(v, "v", type, {total, H, dv}, dev);
    const int64_t qs = row_stride(q, "q"), ks = row_stride(k, "k"), vs = row_stride(v, "v");
    const bool per = tensor(x[3], "g").dim() == 3;
    const int64_t gate_size[3] = {total, H, dk};
    const auto *g = dense<float>(x[3], "g", at::kFloat, {gate_size, per ? 3u : 2u}, dev);
    const auto *beta = dense<float>(x[4], "beta", at::kFloat, {total, H}, dev);
    const auto *scale = dense_or_null<float>(x[9], "gate_scale", at::kFloat, {H}, dev);
    const at::Tensor &pool = tensor(x[5], "pool");
    if (pool.dim() != 4) refuse(PyExc_ValueError, "pool must be a [slots, H, dv, dk] tensor");
    const int64_t slots = pool.size(0);
    look(pool, "pool", at::kFloat, {slots, H, dv, dk}, dev);
    int64_t slot_stride = H * dv * dk;
    if (!pool.is_contiguous()) {
      if (pool.stride(3) != 1 || pool.stride(2) != dk || pool.stride(1) != dv * dk ||
          pool.stride(0) < slot_stride)
        refuse(PyExc_ValueError, "the slots of pool [slots, H, dv, dk] must be dense");
      slot_stride = pool.stride(0);
    }
    const at::Tensor &src = tensor(x[6], "src");
    const int64_t R = src.dim() == 1 ? src.size(0) : -1;
    const auto *psrc = dense<int>(x[6], "src", at::kInt, {R}, dev);
    const auto *dst = dense_or_null<int>(x[7], "dst", at::kInt, {total}, dev);
    const auto *cu = dense_or_null<int>(x[8], "cu_seqlens", at::kInt, {R + 1}, dev);
    if (!cu && R != total)
      refuse(PyExc_ValueError, "without cu_seqlens src must hold one slot for each of %lld tokens",
             (long long)total);
    const int norm = (flag(x[10], "norm_q") ? GDR_NORM_Q : 0) |
                     (flag(x[11], "norm_k") ? GDR_NORM_K : 0);
    Call call(dev, x[13]);
    const at::Tensor o = call.given_or_made(x[12], "o", {total, H, dv}, type);
    const gdr_status st = launch([&] {
      return abi.step_slots(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), dt, qs, ks, vs, g,
        per ? GDR_GATE_PER_CHANNEL : GDR_GATE_SCALAR, beta, scale, norm,
        static_cast<float *>(pool.data_ptr()), fits(slots, "slots"), slot_stride, psrc, dst, cu,
        o.data_ptr(), fits(R, "R"), fits(total, "total"), fits(Hk, "Hk"), fits(H, "H"),
        fits(dk, "dk"), fits(dv, "dv"), call.stream());
    });
    return st == GDR_OK ? wrap(o) : PyLong_FromLong(st);
  });
}

// lens, kept, table, slots, max_tokens, keep_all, out, stream
PyObject *slot_map(PyObject *, PyObject *const *x, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject * {
    const at::Tensor &lens = first_tensor(x[0], "lens", 1, "[R]");
    const auto dev = lens.device();
    const at::Tensor &table = tensor(x[2], "table");
    if (table.dim() != 2) refuse(PyExc_ValueError, "table must be a [R, W] tensor");
    const int64_t R = table.size(0), W = table.size(1);
    const auto *plens = dense<int>(x[0], "lens", at::kInt, {R}, dev);
    const auto *kept = dense<int>(x[1], "kept", at::kInt, {R}, dev);
    look(table, "table", at::kInt, {R, W}, dev);
    int64_t ts = W;
    if (!table.is_contiguous()) {
      if ((W != 1 && table.stride(1) != 1) || (R > 1 && table.stride(0) < W))
        refuse(PyExc_ValueError, "the rows of table [R, W] must be dense");
      ts = R > 1 ? table.stride(0) : W;
    }
    const int64_t slots = whole(x[3], "slots", 0, INT32_MAX);
    const int64_t room = whole(x[4], "max_tokens", 0, INT32_MAX);
    const bool keep_all = flag(x[5], "keep_all");
    check_out(x[6]);
    Call call(dev, x[7]);
    at::Tensor cu, src, request, dst;
    if (x[6] == Py_None) {  // four pieces of one allocation
      const at::Tensor all = call.make({2 * R + 1 + 2 * room}, at::kInt);
      cu = piece(all, 0, R + 1);
      src = piece(all, R + 1, R);
      request = piece(all, 2 * R + 1, room);
      dst = piece(all, 2 * R + 1 + room, room);
    } else {
      cu = call.given_or_made(entry(x[6], "cu_seqlens"), "cu_seqlens", {R + 1}, at::kInt);
      src = call.given_or_made(entry(x[6], "src"), "src", {R}, at::kInt);
      request = call.given_or_made(entry(x[6], "request"), "request", {room}, at::kInt);
      dst = call.given_or_made(entry(x[6], "dst"), "dst", {room}, at::kInt);
    }
    const gdr_status st = launch([&] {
      return abi.slot_map(
        plens, kept, static_cast<int *>(table.data_ptr()), ts, fits(R, "R"), fits(W, "W"),
        static_cast<int>(slots), static_cast<int>(room), keep_all, static_cast<int *>(cu.data_ptr()),
        static_cast<int *>(request.data_ptr()), static_cast<int *>(src.data_ptr()),
        static_cast<int *>(dst.data_ptr()), call.stream());
    });
    if (st != GDR_OK) return PyLong_FromLong(st);
    return dictionary(x[6], {{"cu_seqlens", cu}, {"src", src}, {"request", request}, {"dst", dst}});
  });
}

// What both directions of the output norm look at: x, z, weight, bias, act, center, eps.
struct NormInputs {
  const at::Tensor &x;
  c10::Device dev;
  gdr_dtype dt;
  int64_t G, D, rows, xs, zs = 0;
  int64_t affine[2];
  size_t affine_dims = 1;
  void *z = nullptr;
  float *weight = nullptr, *bias = nullptr;
  gdr_act act;
  int center;
  float eps;

  explicit NormInputs(PyObject *const *a)
      : x(first_tensor(a[0], "x", 2, "[..., G, D]")), dev(x.device()), dt(in_dtype(x, "x")) {
    G = x.size(-2);
    D = x.size(-1);
    rows = G * D ? x.numel() / (G * D) : 0;
    xs = row_stride(x, "x");
    if (a[1] != Py_None) {
      const at::Tensor &t = tensor(a[1], "z");
      look(t, "z", x.scalar_type(), x.sizes(), dev);
      zs = row_stride(t, "z");
      z = t.data_ptr();
    }
    PyObject *any = a[2] != Py_None ? a[2] : a[3];
    if (any != Py_None && tensor(any, "weight/bias").dim() == 2) affine_dims = 2;
    affine[0] = affine_dims == 2 ? G : D;
    affine[1] = D;
    weight = dense_or_null<float>(a[2], "weight", at::kFloat, affine_size(), dev);
    bias = dense_or_null<float>(a[3], "bias", at::kFloat, affine_size(), dev);
    act = static_cast<gdr_act>(whole(a[4], "act", 0, 2));
    center = flag(a[5], "center");
    eps = real(a[6], "eps");
  }
  at::IntArrayRef affine_size() const { return {affine, affine_dims}; }
  int per_channel() const { return affine_dims == 2; }
};

// x, z, weight, bias, act, center, eps, y, stream
PyObject *group_norm_fwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject * {
    const NormInputs i(a);
    Call call(i.dev, a[8]);
    const at::Tensor y = call.given_or_made(a[7], "y", i.x.sizes(), i.x.scalar_type());
    const gdr_status st = launch([&] {
      return abi.group_norm_fwd(
        i.x.data_ptr(), i.z, i.dt, i.xs, i.zs, i.weight, i.bias, i.per_channel(), i.act, i.center,
        i.eps, y.data_ptr(), i.rows, fits(i.G, "G"), fits(i.D, "D"), call.stream());
    });
    return st == GDR_OK ? wrap(y) : PyLong_FromLong(st);
  });
}

// x, z, weight, bias, act, center, eps, dy, workspace, out, stream
PyObject *group_norm_bwd(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject * {
    const NormInputs i(a);
    const auto type = i.x.scalar_type();
    const void *dy = dense(a[7], "dy", type, i.x.sizes(), i.dev);
    check_out(a[9]);
    PyObject *out = a[9];
    Call call(i.dev, a[10]);
    const auto place = [&](bool wanted, const char *name, at::IntArrayRef size,
                           at::ScalarType t) -> at::Tensor {
      if (!wanted) return {};
      return call.given_or_made(out == Py_None ? out : entry(out, name), name, size, t);
    };
    const at::Tensor dx = place(true, "dx", i.x.sizes(), at::kFloat);
    const at::Tensor dz = place(i.z || a[1] != Py_None, "dz", i.x.sizes(), type);
    const at::Tensor dw = place(a[2] != Py_None, "dweight", i.affine_size(), at::kFloat);
    const at::Tensor db = place(a[3] != Py_None, "dbias", i.affine_size(), at::kFloat);
    std::pair<at::Tensor, size_t> ws{{}, 0};
    if (dw.defined() || db.defined())
      ws = call.workspace(a[8], abi.group_norm_bwd_ws(i.rows, fits(i.G, "G"), fits(i.D, "D"), i.dt,
                                                      i.per_channel()));
    const auto f = [](const at::Tensor &t) {
      return t.defined() ? static_cast<float *>(t.data_ptr()) : nullptr;
    };
    const gdr_status st = launch([&] {
      return abi.group_norm_bwd(
        dy, i.x.data_ptr(), i.z, i.dt, i.xs, i.zs, i.weight, i.bias, i.per_channel(), i.act,
        i.center, i.eps, f(dx), dz.defined() ? dz.data_ptr() : nullptr, f(dw), f(db), i.rows,
        fits(i.G, "G"), fits(i.D, "D"), ws.first.defined() ? ws.first.data_ptr() : nullptr,
        ws.second, call.stream());
    });
    if (st != GDR_OK) return PyLong_FromLong(st);
    return dictionary(out, {{"dx", dx}, {"dz", dz}, {"dweight", dw}, {"dbias", db}});
  });
}

// What both directions of the prologue look at: q, k, a, b, gate_scale, norm_q, norm_k.
struct PrologueInputs {
  const at::Tensor &q, &k;
  c10::Device dev;
  gdr_dtype dt;
  int64_t Hk, H, d, tokens, qs, ks;
  c10::SmallVector<int64_t, 6> full, heads;  // [..., H, d] and [..., H]
  bool per_channel;
  float *a, *b, *scale;
  int norm;

  explicit PrologueInputs(PyObject *const *x)
      : q(first_tensor(x[0], "q", 3, "[..., Hk, dk]")), k(tensor(x[1], "k")), dev(q.device()),
        dt(in_dtype(q, "q/k")) {
    const int64_t n = q.dim();
    look(k, "k", q.scalar_type(), q.sizes(), dev);
    const at::Tensor &tb = tensor(x[3], "b");
    if (tb.dim() != n - 1)
      refuse(PyExc_ValueError, "b must be a [..., H] tensor beside q [..., Hk, dk]");
    Hk = q.size(n - 2);
    d = q.size(n - 1);
    H = tb.size(n - 2);
    heads.append(q.sizes().begin(), q.sizes().end() - 2);
    heads.push_back(H);
    full = heads;
    full.push_back(d);
    qs = row_stride(q, "q");
    ks = row_stride(k, "k");
    per_channel = tensor(x[2], "a").dim() == n;
    a = dense<float>(x[2], "a", at::kFloat, gate_size(), dev);
    b = dense<float>(x[3], "b", at::kFloat, heads, dev);
    scale = dense<float>(x[4], "gate_scale", at::kFloat, {H}, dev);
    norm = (flag(x[5], "norm_q") ? GDR_NORM_Q : 0) | (flag(x[6], "norm_k") ? GDR_NORM_K : 0);
    tokens = H ? tb.numel() / H : 0;
  }
  at::IntArrayRef gate_size() const { return per_channel ? full : heads; }
  gdr_gate_kind gate() const { return per_channel ? GDR_GATE_PER_CHANNEL : GDR_GATE_SCALAR; }
};

// q, k, a, b, gate_scale, norm_q, norm_k, out, stream
PyObject *prologue_fwd(PyObject *, PyObject *const *x, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject * {
    const PrologueInputs i(x);
    const auto type = i.q.scalar_type();
    PyObject *out = x[7];
    if (out != Py_None && (!PyTuple_Check(out) || PyTuple_GET_SIZE(out) != 4))
      refuse(PyExc_TypeError, "out must be a tuple (q, k, g, beta)");
    const auto at = [&](int j) { return out == Py_None ? out : PyTuple_GET_ITEM(out, j); };
    Call call(i.dev, x[8]);
    const at::Tensor qn = call.given_or_made(at(0), "q out", i.full, type);
    const at::Tensor kn = call.given_or_made(at(1), "k out", i.full, type);
    const at::Tensor g = call.given_or_made(at(2), "g out", i.gate_size(), at::kFloat);
    const at::Tensor beta = call.given_or_made(at(3), "beta out", i.heads, at::kFloat);
    const gdr_status st = launch([&] {
      return abi.prologue_fwd(
        i.q.data_ptr(), i.k.data_ptr(), i.dt, i.qs, i.ks, i.a, i.gate(), i.b, i.scale, i.norm,
        qn.data_ptr(), kn.data_ptr(), static_cast<float *>(g.data_ptr()),
        static_cast<float *>(beta.data_ptr()), i.tokens, fits(i.Hk, "Hk"), fits(i.H, "H"),
        fits(i.d, "dk"), call.stream());
    });
    if (st != GDR_OK) return PyLong_FromLong(st);
    PyObject *all = PyTuple_New(4);
    PyTuple_SET_ITEM(all, 0, wrap(qn));
    PyTuple_SET_ITEM(all, 1, wrap(kn));
    PyTuple_SET_ITEM(all, 2, wrap(g));
    PyTuple_SET_ITEM(all, 3, wrap(beta));
    return all;
  });
}

// q, k, a, b, gate_scale, norm_q, norm_k, dq, dk, dg, dbeta, workspace, out, stream
PyObject *prologue_bwd(PyObject *, PyObject *const *x, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject * {
    const PrologueInputs i(x);
    const auto type = i.q.scalar_type();
    const auto *dqn = dense<float>(x[7], "dq", at::kFloat, i.full, i.dev);
    const auto *dkn = dense<float>(x[8], "dk", at::kFloat, i.full, i.dev);
    const auto *dg = dense<float>(x[9], "dg", at::kFloat, i.gate_size(), i.dev);
    const auto *dbeta = dense<float>(x[10], "dbeta", at::kFloat, i.heads, i.dev);
    PyObject *out = x[12];
    check_out(out);
    Call call(i.dev, x[13]);
    const auto place = [&](const char *name, at::IntArrayRef size, at::ScalarType t) {
      return call.given_or_made(out == Py_None ? out : entry(out, name), name, size, t);
    };
    const at::Tensor dq = place("dq", i.q.sizes(), type);
    const at::Tensor dk = place("dk", i.q.sizes(), type);
    const at::Tensor da = place("da", i.gate_size(), at::kFloat);
    const at::Tensor db = place("db", i.heads, at::kFloat);
    const at::Tensor ds = place("dgate_scale", {i.H}, at::kFloat);
    const auto ws = call.workspace(
        x[11], abi.prologue_bwd_ws(i.tokens, fits(i.H, "H"), fits(i.d, "dk"), i.gate()));
    const auto f = [](const at::Tensor &t) { return static_cast<float *>(t.data_ptr()); };
    const gdr_status st = launch([&] {
      return abi.prologue_bwd(
        i.q.data_ptr(), i.k.data_ptr(), i.dt, i.qs, i.ks, i.a, i.gate(), i.b, i.scale, i.norm, dqn,
        dkn, dg, dbeta, dq.data_ptr(), dk.data_ptr(), f(da), f(db), f(ds), i.tokens,
        fits(i.Hk, "Hk"), fits(i.H, "H"), fits(i.d, "dk"), ws.first.data_ptr(), ws.second,
        call.stream());
    });
    if (st != GDR_OK) return PyLong_FromLong(st);
    return dictionary(out, {{"dq", dq}, {"dk", dk}, {"da", da}, {"db", db}, {"dgate_scale", ds}});
  });
}

// t, name: the distance of t's rows (for tests of the layouts, on any device)
PyObject *rows_apart(PyObject *, PyObject *const *x, Py_ssize_t n) {
  return guarded(n, 2, [&]() -> PyObject * {
    const at::Tensor &t = tensor(x[0], "t");
    if (t.dim() < 2) refuse(PyExc_ValueError, "t must have 2 dimensions or more");
    return PyLong_FromLongLong(row_stride(t, PyUnicode_AsUTF8(x[1])));
  });
}

// The addresses of the ABI's functions, in the order of Abi.
PyObject *connect(PyObject *, PyObject *const *x, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject * {
    void *p[8];
    for (int i = 0; i < 8; ++i) {
      p[i] = PyLong_AsVoidPtr(x[i]);
      if (!p[i]) {
        PyErr_Clear();
        refuse(PyExc_ValueError, "address %d is missing", i);
      }
    }
    abi.step_slots = reinterpret_cast<decltype(abi.step_slots)>(p[0]);
    abi.slot_map = reinterpret_cast<decltype(abi.slot_map)>(p[1]);
    abi.group_norm_fwd = reinterpret_cast<decltype(abi.group_norm_fwd)>(p[2]);
    abi.group_norm_bwd = reinterpret_cast<decltype(abi.group_norm_bwd)>(p[3]);
    abi.group_norm_bwd_ws = reinterpret_cast<decltype(abi.group_norm_bwd_ws)>(p[4]);
    abi.prologue_fwd = reinterpret_cast<decltype(abi.prologue_fwd)>(p[5]);
    abi.prologue_bwd = reinterpret_cast<decltype(abi.prologue_bwd)>(p[6]);
    abi.prologue_bwd_ws = reinterpret_cast<decltype(abi.prologue_bwd_ws)>(p[7]);
    Py_RETURN_NONE;
  });
}

#define GDR_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    GDR_METHOD(connect),        GDR_METHOD(rows_apart),     GDR_METHOD(step_slots),
    GDR_METHOD(slot_map),       GDR_METHOD(group_norm_fwd), GDR_METHOD(group_norm_bwd),
    GDR_METHOD(prologue_fwd),   GDR_METHOD(prologue_bwd),   {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_gdr_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__gdr_torch(void) { return PyModule_Create(&module); }
