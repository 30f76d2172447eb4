// The stand-alone operators for Python: checks of torch tensors, outputs, stream
// and device, and the C call, in one step. A call on one token spends most of
// its time on the host, and most of that on looking at tensors from Python
// (moe_block_norm of one token: 4.7 us of host time so, 9.2 us there).
// Argument marshalling only; the calls are those of moe_layer.h.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

#include "../../include/moe_layer.h"

namespace {

PyObject* g_error = nullptr;  // MoEError

struct Refused {
  int status;
};
void require(bool ok) {
  if (!ok) throw Refused{MOE_ERR_INVALID_ARG};
}
bool given(PyObject* o) { return o != Py_None; }
const at::Tensor& tensor(PyObject* o) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), "expected a torch.Tensor, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)v;
}
int code_of(at::ScalarType t) {
  return t == at::kBFloat16 ? MOE_BF16 : t == at::kHalf ? MOE_FP16 : t == at::kFloat ? MOE_FP32 : -1;
}
int as_int(int64_t v) {
  if (v > INT32_MAX) throw Refused{MOE_ERR_TOO_LARGE};
  return (int)v;
}

// Row stride of a matrix [n (-1: any), width] on a device whose rows are contiguous
long long rows_of(const at::Tensor& t, int device, int64_t n, int64_t width) {
  require(t.get_device() == device && t.dim() == 2 && t.size(1) == width && (n < 0 || t.size(0) == n));
  if (t.is_contiguous()) return width;
  require(t.stride(1) == 1 || width == 1);
  return t.stride(0);
}
// A contiguous tensor of the given type and shape
template <typename T>
T* flat(const at::Tensor& t, int device, at::ScalarType type, at::IntArrayRef shape) {
  require(t.get_device() == device && t.scalar_type() == type && t.sizes() == shape && t.is_contiguous());
  return static_cast<T*>(t.data_ptr());
}

// Device and stream of a call: outputs come from the pool of the stream that
// writes them, and the device is current while the call is made.
class Place {
 public:
  Place(const at::Tensor& lead, PyObject* stream) : device_(lead.device()) {
    if (device_.index() != c10::cuda::current_device()) guard_.emplace(device_);
    if (given(stream)) {
      void* s = PyLong_AsVoidPtr(stream);
      if (!s && PyErr_Occurred()) throw python_error();
      stream_ = static_cast<cudaStream_t>(s);
      on_stream_.emplace(c10::cuda::getStreamFromExternal(stream_, device_.index()));
    } else {
      stream_ = c10::cuda::getCurrentCUDAStream(device_.index()).stream();
    }
  }
  at::Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
    return at::empty(shape, at::TensorOptions().dtype(type).device(device_));
  }
  cudaStream_t stream() const { return stream_; }

 private:
  c10::Device device_;
  std::optional<c10::cuda::CUDAGuard> guard_;
  std::optional<c10::cuda::CUDAStreamGuard> on_stream_;
  cudaStream_t stream_ = nullptr;
};

// the C call, without the interpreter's lock
template <typename Call>
void run(Call call) {
  moe_status_t s;
  Py_BEGIN_ALLOW_THREADS;
  s = call();
  Py_END_ALLOW_THREADS;
  if (s != MOE_OK) throw Refused{(int)s};
}

// the Python side of a call: where() names it in errors
template <typename Body>
PyObject* guarded(const char* where, Body body) {
  HANDLE_TH_ERRORS
  try {
    return body();
  } catch (const Refused& r) {
    PyObject* e = PyObject_CallFunction(g_error, "is", r.status, where);
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}
// a tensor that the call wrote into: a change in place, as autograd counts them
PyObject* written(PyObject* o) {
  if (given(o)) {
    const at::Tensor& t = tensor(o);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  }
  return o;
}
PyObject* keep(PyObject* o) {
  Py_INCREF(o);
  return o;
}
PyObject* pair(PyObject* a, PyObject* b) {  // takes over both references
  PyObject* t = a && b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return t;
}
bool arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

// (residual, branch, w_pre, w_post, gate, gate_sigmoid, residual_scale, branch_scale, eps, weight_offset, inv_pos,
//  pair_weights, residual_out, h_out, stream)
PyObject* block_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arguments(n, 15)) return nullptr;
  PyObject *const residual = args[0], *const branch = args[1], *const w_pre = args[2], *const w_post = args[3],
           *const gate = args[4], *const inv_pos = args[10], *const pair_weights = args[11], *const residual_out = args[12],
           *const h_out = args[13];
  return guarded("moe_block_norm", [&]() -> PyObject* {
    require(given(residual) || given(branch));
    const at::Tensor& lead = tensor(given(residual) ? residual : branch);
    require(lead.dim() == 2 && lead.is_cuda());
    const int device = lead.get_device();
    const Place place(lead, args[14]);
    int64_t T = lead.size(0);
    const int64_t K = lead.size(1);
    if (!given(residual) && given(inv_pos)) {
      require(tensor(inv_pos).dim() == 2);
      T = tensor(inv_pos).size(0);
    }
    const at::ScalarType dt = given(branch)  ? tensor(branch).scalar_type()
                              : given(w_pre) ? tensor(w_pre).scalar_type()
                                             : lead.scalar_type();
    const at::ScalarType rdt = given(residual)       ? lead.scalar_type()
                               : given(residual_out) ? tensor(residual_out).scalar_type()
                                                     : dt;
    moe_block_norm_t a = {};
    a.tokens = as_int(T);
    a.width = as_int(K);
    a.dtype = (moe_dtype_t)code_of(dt);
    a.residual_dtype = (moe_dtype_t)code_of(rdt);
    a.residual_scale = number(args[6]);
    a.branch_scale = number(args[7]);
    a.eps = number(args[8]);
    a.weight_offset = number(args[9]);
    if (given(residual)) {
      a.residual = lead.data_ptr();
      a.residual_stride = rows_of(lead, device, T, K);
    }
    require(given(inv_pos) == given(pair_weights));
    if (given(branch)) {
      const at::Tensor& y = tensor(branch);
      a.branch_stride = rows_of(y, device, given(inv_pos) ? -1 : T, K);
      a.branch = y.data_ptr();
      a.branch_rows = as_int(y.size(0));
    }
    if (given(inv_pos)) {
      const at::Tensor& p = tensor(inv_pos);
      require(p.dim() == 2 && p.size(1) >= 1);
      a.pairs = as_int(p.size(1));
      a.inv_pos = flat<int>(p, device, at::kInt, {T, p.size(1)});
      a.pair_weights = flat<float>(tensor(pair_weights), device, at::kFloat, {T, p.size(1)});
    }
    if (given(w_post)) a.post_weight = flat<void>(tensor(w_post), device, dt, {K});
    if (given(w_pre)) a.pre_weight = flat<void>(tensor(w_pre), device, dt, {K});
    if (given(gate)) {
      const at::Tensor& g = tensor(gate);
      if (g.dim() == 1) {
        a.gate = flat<void>(g, device, dt, {K});
        a.gate_channel_stride = 1;
      } else {
        require(g.dim() == 2 && g.scalar_type() == dt && (g.size(1) == 1 || g.size(1) == K));
        a.gate_token_stride = rows_of(g, device, T, g.size(1));
        a.gate_channel_stride = g.size(1) == 1 ? 0 : 1;
        a.gate = g.data_ptr();
      }
      const int on = PyObject_IsTrue(args[5]);
      if (on < 0) throw python_error();
      a.gate_sigmoid = on;
    }
    at::Tensor r, h;  // outputs made here
    if (given(residual_out)) {
      const at::Tensor& o = tensor(residual_out);
      require(o.scalar_type() == rdt);
      a.residual_out_stride = rows_of(o, device, T, K);
      a.residual_out = o.data_ptr();
    } else if (given(branch)) {
      r = place.make({T, K}, rdt);
      a.residual_out_stride = K;
      a.residual_out = r.data_ptr();
    }
    if (given(h_out)) {
      const at::Tensor& o = tensor(h_out);
      require(o.scalar_type() == dt);
      a.h_stride = rows_of(o, device, T, K);
      a.h = o.data_ptr();
    } else if (given(w_pre)) {
      h = place.make({T, K}, dt);
      a.h_stride = K;
      a.h = h.data_ptr();
    }
    if (T > 0) run([&] { return moe_block_norm(&a, place.stream()); });
    return pair(r.defined() ? THPVariable_Wrap(r) : keep(written(residual_out)),
                h.defined() ? THPVariable_Wrap(h) : keep(written(h_out)));
  });
}

// (x, src_rows, codes, scales, stream)
PyObject* quantize_rows(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arguments(n, 5)) return nullptr;
  return guarded("moe_quantize_rows", [&]() -> PyObject* {
    const at::Tensor& x = tensor(args[0]);
    require(x.dim() == 2 && x.is_cuda());
    const int device = x.get_device();
    const Place place(x, args[4]);
    const int64_t M = x.size(0), K = x.size(1);
    const long long ldx = rows_of(x, device, M, K);
    int64_t R = M;
    const int* src = nullptr;
    if (given(args[1])) {
      const at::Tensor& s = tensor(args[1]);
      require(s.dim() == 1);
      R = s.size(0);
      src = flat<int>(s, device, at::kInt, {R});
    }
    at::Tensor q, s;
    long long ldq = K;
    if (given(args[2])) {
      q = tensor(args[2]);
      require(q.scalar_type() == at::kChar);
      ldq = rows_of(q, device, R, K);
    } else {
      q = place.make({R, K}, at::kChar);
    }
    s = given(args[3]) ? tensor(args[3]) : place.make({R}, at::kFloat);
    float* scales = flat<float>(s, device, at::kFloat, {R});
    const int m = as_int(M), rows = as_int(R), width = as_int(K);
    run([&] {
      return moe_quantize_rows(x.data_ptr(), ldx, m, (moe_dtype_t)code_of(x.scalar_type()), src, rows, width,
                               static_cast<signed char*>(q.data_ptr()), ldq, scales, place.stream());
    });
    return pair(given(args[2]) ? keep(written(args[2])) : THPVariable_Wrap(q),
                given(args[3]) ? keep(written(args[3])) : THPVariable_Wrap(s));
  });
}

// what the products share
struct Product {
  long long ldx, ldw, ldwe = 0, ldy;
  const int* offsets = nullptr;
  int rows, experts = 1, K, N;
  at::Tensor y;
  Product(const Place& place, const at::Tensor& x, const at::Tensor& w, PyObject* off, at::ScalarType default_type,
          PyObject* out_dtype, PyObject* out) {
    const int device = x.get_device();
    require(w.scalar_type() == x.scalar_type() && w.get_device() == device && (w.dim() == 2 || w.dim() == 3));
    const int64_t R = x.size(0), k = x.size(1), d = w.dim(), E = d == 3 ? w.size(0) : 1, n = w.size(d - 2);
    ldx = rows_of(x, device, R, k);
    require(w.size(d - 1) == k && (w.stride(d - 1) == 1 || k == 1));
    ldw = w.stride(d - 2);
    if (d == 3) ldwe = w.stride(0);
    rows = as_int(R);
    K = as_int(k);
    N = as_int(n);
    experts = as_int(E);
    if (given(off)) offsets = flat<int>(tensor(off), device, at::kInt, {E + 1});
    at::ScalarType type = default_type;
    if (given(out_dtype)) {
      TORCH_CHECK_TYPE(THPDtype_Check(out_dtype), "out_dtype is a torch.dtype");
      type = reinterpret_cast<THPDtype*>(out_dtype)->scalar_type;
    }
    if (given(out)) {
      y = tensor(out);
      require(!given(out_dtype) || y.scalar_type() == type);
      ldy = rows_of(y, device, R, n);
    } else {
      require(code_of(type) >= 0);
      y = place.make({R, n}, type);
      ldy = n;
    }
  }
  moe_dtype_t type() const { return (moe_dtype_t)code_of(y.scalar_type()); }
};

// (x, row_scales, w, channel_scales, offsets, out_dtype, out, stream)
PyObject* int8_matmul(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arguments(n, 8)) return nullptr;
  return guarded("moe_int8_matmul", [&]() -> PyObject* {
    const at::Tensor &x = tensor(args[0]), &w = tensor(args[2]);
    require(x.dim() == 2 && x.is_cuda() && x.scalar_type() == at::kChar);
    const Place place(x, args[7]);
    const Product p(place, x, w, args[4], at::kBFloat16, args[5], args[6]);
    const float* xs = flat<float>(tensor(args[1]), x.get_device(), at::kFloat, {x.size(0)});
    const float* ws = flat<float>(tensor(args[3]), x.get_device(), at::kFloat, w.sizes().slice(0, w.dim() - 1));
    run([&] {
      return moe_int8_matmul(static_cast<const signed char*>(x.data_ptr()), p.ldx, xs,
                             static_cast<const signed char*>(w.data_ptr()), p.ldw, p.ldwe, ws, p.offsets, p.rows, p.experts,
                             p.K, p.N, p.y.data_ptr(), p.ldy, p.type(), place.stream());
    });
    return given(args[6]) ? keep(written(args[6])) : THPVariable_Wrap(p.y);
  });
}

// (x, w, offsets, out_dtype, out, stream)
PyObject* grouped_matmul(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arguments(n, 6)) return nullptr;
  return guarded("moe_grouped_matmul", [&]() -> PyObject* {
    const at::Tensor &x = tensor(args[0]), &w = tensor(args[1]);
    require(x.dim() == 2 && x.is_cuda());
    const Place place(x, args[5]);
    const Product p(place, x, w, args[2], x.scalar_type(), args[3], args[4]);
    run([&] {
      return moe_grouped_matmul(x.data_ptr(), p.ldx, w.data_ptr(), p.ldw, p.ldwe, p.offsets, p.rows, p.experts, p.K, p.N,
                                (moe_dtype_t)code_of(x.scalar_type()), p.y.data_ptr(), p.ldy, p.type(), place.stream());
    });
    return given(args[4]) ? keep(written(args[4])) : THPVariable_Wrap(p.y);
  });
}

// the class of the errors raised: called with (status, where)
PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyMethodDef method(const char* name, Fast f) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method("block_norm", block_norm),
                         method("quantize_rows", quantize_rows),
                         method("int8_matmul", int8_matmul),
                         method("grouped_matmul", grouped_matmul),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Calls of the stand-alone operators on torch tensors.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
