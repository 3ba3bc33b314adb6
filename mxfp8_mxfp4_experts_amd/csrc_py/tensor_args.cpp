// Argument checks of the calls around the experts, for the Python binding.
//
// In a decode step those calls take a few microseconds each, launch included,
// and asking a tensor for its dtype, shape, device and layout from Python costs
// about 0.3 us per tensor; here it is one call of 0.05 us (moe_add_rmsnorm of one
// row of 7168 with a residual: 8.5 -> 6.3 us a call).  These functions only
// answer; what is wrong is said by the binding.  A tensor that has no plain
// memory (sparse, nested, fake) throws when asked for it: that is a no as well,
// and no exception leaves an entry.
//
// The calls beside the experts go one step further: with every buffer given and everything plainly
// right, one function checks the tensors and makes the C call (at the address that the binding
// gives) and answers its status; else it answers None, nothing has been launched, and the binding
// checks and calls step by step.  (A call, launch included: moe_fp8_linear of one token 5.1 -> 3.7
// us, moe_fp8_grouped 6.1 -> 4.1, moe_quant_fp8 4.0 -> 3.3, moe_sort_tokens 4.6 -> 3.3; the binding
// itself takes 0.3 us of that.)
#include <Python.h>

#include <climits>
#include <cstdint>
#include <exception>

#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mi355moe.h"

namespace {

// head(t) -> (device index, rows, columns) of a two-dimensional tensor on the
// current GPU, else None.
PyObject* head(PyObject*, PyObject* obj) {
  if (!THPVariable_Check(obj)) Py_RETURN_NONE;
  const at::Tensor& t = THPVariable_Unpack(obj);
  try {
    if (!t.is_cuda() || t.dim() != 2) Py_RETURN_NONE;
    const long idx = t.get_device();
    const c10::impl::VirtualGuardImpl gpu(c10::DeviceType::CUDA);
    if (gpu.getDevice().index() != idx) Py_RETURN_NONE;
    return Py_BuildValue("(lLL)", idx, (long long)t.size(0), (long long)t.size(1));
  } catch (const std::exception&) {
    Py_RETURN_NONE;
  }
}

// plain(t, dtype, rows, columns, device index) -> the address of a contiguous
// GPU tensor of just that dtype, shape (columns -1: one-dimensional) and
// device, else -1.
PyObject* plain(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5 || !THPDtype_Check(a[1])) {
    PyErr_SetString(PyExc_TypeError, "plain(tensor, dtype, rows, columns, device index)");
    return nullptr;
  }
  const long long rows = PyLong_AsLongLong(a[2]), cols = PyLong_AsLongLong(a[3]);
  const long idx = PyLong_AsLong(a[4]);
  if (PyErr_Occurred()) return nullptr;
  if (!THPVariable_Check(a[0])) return PyLong_FromLong(-1);
  const at::Tensor& t = THPVariable_Unpack(a[0]);
  try {
    const bool ok = t.scalar_type() == reinterpret_cast<THPDtype*>(a[1])->scalar_type &&
                    t.is_cuda() && t.get_device() == idx && t.dim() == (cols < 0 ? 1 : 2) &&
                    t.size(0) == rows && (cols < 0 || t.size(1) == cols) && t.is_contiguous();
    return ok ? PyLong_FromVoidPtr(t.data_ptr()) : PyLong_FromLong(-1);
  } catch (const std::exception&) {
    return PyLong_FromLong(-1);
  }
}

// ---------------------------------------------------------------------------
// Check and call.  Arguments: the C function's address, the binding's function for the current
// stream of a device, then the Python call's own.

using at::ScalarType;
constexpr ScalarType kBf16 = ScalarType::BFloat16, kF32 = ScalarType::Float, kI32 = ScalarType::Int;

struct No {};                                 // thrown where something is not plainly right
inline void need(bool ok) {
  if (!ok) throw No();
}

// A call's tensors, all on one GPU, which has to be the current one.
class Args {
 public:
  explicit Args(PyObject* first) {
    need(THPVariable_Check(first));
    const at::Tensor& t = THPVariable_Unpack(first);
    need(t.is_cuda());
    idx_ = t.get_device();
    const c10::impl::VirtualGuardImpl gpu(c10::DeviceType::CUDA);
    need(gpu.getDevice().index() == idx_);
  }
  const at::Tensor& tensor(PyObject* o, int dim) const {
    need(THPVariable_Check(o));
    const at::Tensor& t = THPVariable_Unpack(o);
    need(t.is_cuda() && t.get_device() == idx_ && t.dim() == dim);
    return t;
  }
  // Rows of unit column stride, `rows` and `cols` of them (-1: any number).
  struct Rows {
    void* p;
    int64_t ld;
    int rows, cols;
    ScalarType type;
  };
  Rows rows(PyObject* o, int64_t rows, int64_t cols) const {
    const at::Tensor& t = tensor(o, 2);
    const int64_t r = t.size(0), c = t.size(1);
    need(r <= INT_MAX && c <= INT_MAX && (rows < 0 || r == rows) && (cols < 0 || c == cols) &&
         (t.stride(1) == 1 || c == 1));
    return {t.data_ptr(), r > 1 ? t.stride(0) : c, (int)r, (int)c, t.scalar_type()};
  }
  Rows rows(PyObject* o, int64_t n, int64_t cols, ScalarType type) const {
    const Rows r = rows(o, n, cols);
    need(r.type == type);
    return r;
  }
  Rows codes(PyObject* o, int64_t n, int64_t cols) const {
    const Rows r = rows(o, n, cols);
    need(is_code(r.type));
    return r;
  }
  static bool is_code(ScalarType t) {
    return t == ScalarType::Byte || t == ScalarType::Float8_e4m3fn;
  }
  // Contiguous, of one dimension (`n` elements, -1: any number) or of two.
  void* flat(PyObject* o, ScalarType type, int64_t n, int* count = nullptr) const {
    const at::Tensor& t = tensor(o, 1);
    need(t.scalar_type() == type && (n < 0 || t.size(0) == n) && t.size(0) <= INT_MAX &&
         t.is_contiguous());
    if (count) *count = (int)t.size(0);
    return t.data_ptr();
  }
  void* whole(PyObject* o, ScalarType type, int64_t rows, int64_t cols) const {
    const at::Tensor& t = tensor(o, 2);
    need(t.scalar_type() == type && t.size(0) == rows && t.size(1) == cols && t.is_contiguous());
    return t.data_ptr();
  }
  // route_row: [T, top_k], in one dimension or two; T -1: any that fits.
  const int32_t* routes(PyObject* o, int64_t T, int top_k, int* tokens = nullptr) const {
    need(THPVariable_Check(o));
    const at::Tensor& t = tensor(o, (int)THPVariable_Unpack(o).dim());
    const int64_t n = t.numel();
    need(top_k >= 1 && n % top_k == 0 && n <= INT_MAX && t.scalar_type() == kI32 &&
         t.is_contiguous() && (T < 0 || n == T * top_k) &&
         (t.dim() == 1 || (t.dim() == 2 && t.size(1) == top_k)));
    if (tokens) *tokens = (int)(n / top_k);
    return static_cast<const int32_t*>(t.data_ptr());
  }
  // An E4M3 weight [N, K] or [E, N, K] and its scales.
  struct Weight {
    const uint8_t* w;
    const float* s;
    int E, N;
  };
  Weight weight(PyObject* w, PyObject* w_s, int K, int dim) const {
    const at::Tensor &t = tensor(w, dim), &u = tensor(w_s, dim);
    const int64_t E = dim == 3 ? t.size(0) : 1, N = t.size(dim - 2);
    need(is_code(t.scalar_type()) && t.size(dim - 1) == K && E <= INT_MAX && N <= INT_MAX &&
         t.is_contiguous());
    need(u.scalar_type() == kF32 && (dim == 2 || u.size(0) == E) &&
         u.size(dim - 2) == (N + 127) / 128 && u.size(dim - 1) == ((int64_t)K + 127) / 128 &&
         u.is_contiguous());
    return {static_cast<const uint8_t*>(t.data_ptr()), static_cast<const float*>(u.data_ptr()),
            (int)E, (int)N};
  }
  hipStream_t stream(PyObject* current) const {
    PyObject* index = PyLong_FromLong(idx_);
    PyObject* got = index ? PyObject_CallOneArg(current, index) : nullptr;
    Py_XDECREF(index);
    void* s = got ? PyLong_AsVoidPtr(got) : nullptr;
    Py_XDECREF(got);
    need(!PyErr_Occurred());
    return static_cast<hipStream_t>(s);
  }

 private:
  int64_t idx_;
};

// The C call, during which other Python threads run (it may load code or wait for a full queue).
template <class F, class... A>
moe_status_t call(PyObject* address, A... args) {
  F* const f = reinterpret_cast<F*>(PyLong_AsVoidPtr(address));
  need(f != nullptr);
  moe_status_t status;
  Py_BEGIN_ALLOW_THREADS
  status = f(args...);
  Py_END_ALLOW_THREADS
  return status;
}
int whole_number(PyObject* o) {
  const long v = PyLong_Check(o) ? PyLong_AsLong(o) : -1;
  need(!PyErr_Occurred() && v >= 0 && v <= INT_MAX);
  return (int)v;
}
template <class T>
T* as(void* p) {
  return static_cast<T*>(p);
}
int row_type(ScalarType t) {
  need(t == kBf16 || t == kF32);
  return t == kBf16 ? MOE_ROWS_BF16 : MOE_ROWS_F32;
}

// Runs f(a) with n arguments; what is thrown, or an error left by Python, is None.
template <class F>
PyObject* answer(Py_ssize_t n, Py_ssize_t wanted, F f) {
  if (n != wanted) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return PyLong_FromLong((long)f());
  } catch (const No&) {
  } catch (const std::exception&) {
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

// (address, stream, x, xq, xs)
PyObject* quant_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return answer(n, 5, [&] {
    const Args g(a[2]);
    const auto x = g.rows(a[2], -1, -1, kBf16);
    const auto q = g.codes(a[3], x.rows, x.cols);
    need(q.ld == x.cols);
    const auto s = g.rows(a[4], (x.cols + 127LL) / 128, x.rows, kF32);
    return call<decltype(moe_quant_fp8)>(
        a[0], as<uint16_t>(x.p), x.ld, x.rows, x.cols, as<uint8_t>(q.p), as<float>(s.p), s.ld,
        g.stream(a[1]));
  });
}

// (address, stream, xq, xs, w, w_s, out, workspace)
PyObject* fp8_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return answer(n, 8, [&] {
    const Args g(a[2]);
    const auto q = g.codes(a[2], -1, -1);
    const auto s = g.rows(a[3], (q.cols + 127LL) / 128, q.rows, kF32);
    const auto w = g.weight(a[4], a[5], q.cols, 2);
    const auto o = g.rows(a[6], q.rows, w.N, kBf16);
    int bytes;
    void* ws = g.flat(a[7], ScalarType::Byte, -1, &bytes);
    return call<decltype(moe_fp8_matmul)>(
        a[0], as<uint8_t>(q.p), q.ld, as<float>(s.p), s.ld, w.w, w.s, q.rows, w.N, q.cols,
        as<uint16_t>(o.p), o.ld, ws, (size_t)bytes, g.stream(a[1]));
  });
}

// (address, stream, x, w, w_s, out, workspace)
PyObject* fp8_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return answer(n, 7, [&] {
    const Args g(a[2]);
    const auto x = g.rows(a[2], -1, -1, kBf16);
    const auto w = g.weight(a[3], a[4], x.cols, 2);
    const auto o = g.rows(a[5], x.rows, w.N, kBf16);
    int bytes;
    void* ws = g.flat(a[6], ScalarType::Byte, -1, &bytes);
    return call<decltype(moe_fp8_linear)>(
        a[0], as<uint16_t>(x.p), x.ld, w.w, w.s, x.rows, w.N, x.cols, as<uint16_t>(o.p), o.ld, ws,
        (size_t)bytes, g.stream(a[1]));
  });
}

// (address, stream, xq, xs, w, w_s, expert_offsets, sorted_route or None, top_k, out)
PyObject* fp8_grouped(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return answer(n, 10, [&] {
    const Args g(a[2]);
    const auto q = g.codes(a[2], -1, -1);
    const auto s = g.rows(a[3], (q.cols + 127LL) / 128, q.rows, kF32);
    const auto w = g.weight(a[4], a[5], q.cols, 3);
    void* offs = g.flat(a[6], kI32, w.E + 1LL);
    int R = q.rows;
    void* route = a[7] == Py_None ? nullptr : g.flat(a[7], kI32, -1, &R);
    const auto o = g.rows(a[9], R, w.N, kBf16);
    return call<decltype(moe_fp8_grouped)>(
        a[0], as<uint8_t>(q.p), q.ld, as<float>(s.p), s.ld, q.rows, w.w, w.s, w.E, w.N, q.cols,
        as<int32_t>(offs), as<int32_t>(route), whole_number(a[8]), R, as<uint16_t>(o.p), o.ld,
        g.stream(a[1]));
  });
}

// (address, stream, x, route_row, top_k, rows)
PyObject* sort_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return answer(n, 6, [&] {
    const Args g(a[2]);
    const auto x = g.rows(a[2], -1, -1);
    const int k = whole_number(a[4]);
    const int32_t* route = g.routes(a[3], x.rows, k);
    const auto r = g.rows(a[5], -1, x.cols, x.type);
    return call<decltype(moe_sort_tokens)>(
        a[0], x.p, x.ld, x.rows, x.cols, k, route, row_type(x.type), r.p, r.ld, r.rows,
        g.stream(a[1]));
  });
}

// (address, stream, rows, route_row, topk_w or None, top_k, out)
PyObject* unsort_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return answer(n, 7, [&] {
    const Args g(a[2]);
    const auto r = g.rows(a[2], -1, -1);
    const int k = whole_number(a[5]);
    int T;
    const int32_t* route = g.routes(a[3], -1, k, &T);
    void* w = a[4] == Py_None ? nullptr : g.whole(a[4], kF32, T, k);
    const auto o = g.rows(a[6], T, r.cols, r.type);
    return call<decltype(moe_unsort_tokens)>(
        a[0], r.p, r.ld, r.rows, T, r.cols, k, route, as<float>(w), row_type(r.type), o.p, o.ld,
        g.stream(a[1]));
  });
}

// (address, stream, dout, rows, route_row, topk_w, drows, dw)
PyObject* unsort_tokens_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return answer(n, 8, [&] {
    const Args g(a[2]);
    const auto d = g.rows(a[2], -1, -1);
    const auto r = g.rows(a[3], -1, d.cols, d.type);
    const at::Tensor& wt = g.tensor(a[5], 2);
    need(wt.size(1) <= INT_MAX);
    const int k = (int)wt.size(1);
    void* w = g.whole(a[5], kF32, d.rows, k);
    const int32_t* route = g.routes(a[4], d.rows, k);
    const auto o = g.rows(a[6], r.rows, d.cols, d.type);
    void* dw = g.whole(a[7], kF32, d.rows, k);
    return call<decltype(moe_unsort_tokens_grad)>(
        a[0], d.p, d.ld, r.p, r.ld, r.rows, d.rows, d.cols, k, route, as<float>(w),
        row_type(d.type), o.p, o.ld, as<float>(dw), g.stream(a[1]));
  });
}

// (address, stream, topk_idx, expert_offset, E_local, workspace, expert_offsets, sorted_route,
// route_row)
PyObject* permute(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return answer(n, 9, [&] {
    const Args g(a[2]);
    const at::Tensor& idx = g.tensor(a[2], 2);
    const int64_t T = idx.size(0), k = idx.size(1);
    need(T <= INT_MAX && k <= INT_MAX && T * k <= INT_MAX);
    void* ids = g.whole(a[2], kI32, T, k);
    const int first = whole_number(a[3]), E = whole_number(a[4]);
    int bytes;
    void* ws = g.flat(a[5], ScalarType::Byte, -1, &bytes);
    void* offs = g.flat(a[6], kI32, E + 1LL);
    void* sorted = g.flat(a[7], kI32, T * k);
    void* row = g.flat(a[8], kI32, T * k);
    return call<decltype(moe_permute)>(
        a[0], as<int32_t>(ids), (int)T, (int)k, first, E, as<int32_t>(offs), as<int32_t>(sorted),
        as<int32_t>(row), ws, (size_t)bytes, g.stream(a[1]));
  });
}

#define CALL(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, \
   "status of moe_" #name " with these tensors, or None where they are not plainly right"}
PyMethodDef methods[] = {
    {"head", head, METH_O, "(device index, rows, columns) of a 2-D tensor on the current GPU"},
    {"plain", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(plain)), METH_FASTCALL,
     "address of a contiguous tensor of this dtype, shape and device, or -1"},
    CALL(quant_fp8), CALL(fp8_matmul), CALL(fp8_linear), CALL(fp8_grouped), CALL(sort_tokens),
    CALL(unsort_tokens), CALL(unsort_tokens_grad), CALL(permute),
    {nullptr, nullptr, 0, nullptr}};
#undef CALL
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_args() { return PyModule_Create(&module); }
