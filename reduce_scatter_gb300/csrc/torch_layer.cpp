// torch_layer.cpp -- the Python extension behind reduce_scatter_gb300.layer:
// checks and marshals torch tensors for include/dg_layer.h and allocates the
// outputs.  In C++ because small calls are bound by the host: checking,
// allocating and launching took 15-28 us a call through ctypes, against 2-4 us
// on the GPU.
//
// Errors: ValueError / TypeError for arguments, dg.DGError (set_error) for a
// dg_status.  No call synchronizes except check().

#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/full.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <mutex>
#include <unordered_map>

#include "dg_layer.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;  // dg.DGError

struct StatusError {
  int code;
};
void check_status(int rc) {
  if (rc != DG_OK) throw StatusError{rc};
}

// Runs a body, turning its exceptions into Python's.
template <class F>
PyObject* guarded(F body) {
  HANDLE_TH_ERRORS
  try {
    return body();
  } catch (const StatusError& e) {
    if (PyObject* args = Py_BuildValue("(is)", e.code, dg_layer_last_error())) {
      PyErr_SetObject(g_error ? g_error : PyExc_RuntimeError, args);
      Py_DECREF(args);
    }
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

void want_args(Py_ssize_t got, Py_ssize_t want) {
  TORCH_CHECK_TYPE(got == want, "expected ", want, " arguments, got ", got);
}
// (No call has a forward-mode derivative, and outputs without one would pass for constants.)
const Tensor& tensor(PyObject* o, const char* what) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), what, " must be a tensor");
  const Tensor& t = THPVariable_Unpack(o);
  TORCH_CHECK_VALUE(!t._fw_grad(0).defined(), what, " has a forward-mode tangent, which this operator does not carry on");
  return t;
}
// A tensor or None (an undefined tensor).
Tensor maybe(PyObject* o, const char* what) { return o == Py_None ? Tensor() : tensor(o, what); }
at::ScalarType dtype(PyObject* o) {
  TORCH_CHECK_TYPE(THPDtype_Check(o), "out_dtype must be a torch dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}
PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

// The dg_type of a torch type, or -1.
int type_of(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return DG_TYPE_BF16;
    case at::kFloat: return DG_TYPE_F32;
    case at::kFloat8_e4m3fn: return DG_TYPE_E4M3;
    case at::kFloat8_e5m2: return DG_TYPE_E5M2;
    default: return -1;
  }
}
bool is8(at::ScalarType t) { return t == at::kFloat8_e4m3fn || t == at::kFloat8_e5m2; }
bool bf16_or_f32(at::ScalarType t) { return t == at::kBFloat16 || t == at::kFloat; }

void same_device(const Tensor& x, std::initializer_list<const Tensor*> others) {
  TORCH_CHECK_VALUE(x.is_cuda(), "inputs must be CUDA tensors");
  for (const Tensor* t : others)
    TORCH_CHECK_VALUE(!t->defined() || t->device() == x.device(), "all tensors must be on the same CUDA device");
}

// The tensors' device made current, and its current stream.
struct Site {
  c10::cuda::CUDAGuard guard;
  c10::cuda::CUDAStream stream;
  explicit Site(const Tensor& x) : guard(x.device()), stream(c10::cuda::getCurrentCUDAStream(x.device().index())) {}
  void* handle() const { return stream.stream(); }
};

// An output or workspace on x's device, without the dispatcher (0.4 us a tensor).
Tensor fresh(const Tensor& x, at::IntArrayRef sizes, at::ScalarType type) {
  return at::detail::empty_cuda(sizes, type, x.device(), std::nullopt);
}

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// (..., hidden) as a matrix whose rows are contiguous; copies only where the
// strides leave no other way.
Tensor as_rows(const Tensor& t, int64_t hidden) {
  int64_t rows = 1;
  for (int64_t d = 0; d + 1 < t.dim(); ++d) rows *= t.size(d);
  Tensor r = t.dim() == 2 ? t : t.reshape({rows, hidden});
  return r.stride(1) == 1 || hidden <= 1 ? r : r.contiguous();
}
bool aligned(const Tensor& t, int64_t pitch) {
  return reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0 && pitch * t.element_size() % 16 == 0;
}
// A matrix with contiguous, 16-byte aligned rows that do not overlap; a copy
// only where it is not.
Tensor as_operand(const Tensor& t) {
  if (t.size(0) == 0 || (t.stride(1) == 1 && t.stride(0) >= t.size(1) && aligned(t, t.stride(0)))) return t;
  return fresh(t, t.sizes(), t.scalar_type()).copy_(t);
}

// Rows in memory, to tell whether two tensors share some.
struct Rows {
  uintptr_t at;
  int64_t count, pitch, bytes;  // from row to row, and of one
  Rows(const Tensor& t, int64_t count_, int64_t pitch_, int64_t length)
      : at(reinterpret_cast<uintptr_t>(t.data_ptr())), count(count_), pitch(pitch_ * t.element_size()),
        bytes(length * t.element_size()) {}
  uintptr_t end() const { return at + (count - 1) * pitch + bytes; }
  bool same(const Rows& o) const { return at == o.at && bytes == o.bytes && (pitch == o.pitch || count == 1); }
  // (starts and ends ascend in both)
  bool meet(const Rows& o) const {
    if (count == 0 || bytes == 0 || o.count == 0 || o.bytes == 0 || end() <= o.at || o.end() <= at) return false;
    for (int64_t i = 0, j = 0; i < count && j < o.count;) {
      const uintptr_t a = at + i * pitch, b = o.at + j * o.pitch;
      if (a + bytes <= b)
        ++i;
      else if (b + o.bytes <= a)
        ++j;
      else
        return true;
    }
    return false;
  }
};

// ------------------------------------------------------------- device state

// The status word of each device, and the products' workspace of each stream:
// the calls of one stream run one after another.  Inside a stream capture a
// call takes a workspace of the graph's own, since its replays may run beside
// the stream's later calls.
struct State {
  std::mutex mu;
  std::unordered_map<int, Tensor> status;
  std::unordered_map<uint64_t, Tensor> workspace;
};
State& state() {
  static State* s = new State;  // lives as long as the process: CUDA may be gone before static destructors
  return *s;
}
bool capturing() { return c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None; }

void* status_word(const Site& at, const Tensor& like) {
  State& st = state();
  std::lock_guard<std::mutex> lk(st.mu);
  Tensor& t = st.status[(int)like.device().index()];
  if (!t.defined()) {
    TORCH_CHECK(!capturing(), "make one call outside of stream capture first");
    Tensor fresh = at::zeros({16}, like.options().dtype(at::kLong));
    at.stream.synchronize();  // zero before any stream uses it
    t = fresh;
  }
  return t.data_ptr();
}
Tensor new_workspace(const Tensor& like) {
  const size_t bytes = dg_layer_products_workspace();
  if (bytes == 0) throw StatusError{DG_ERR_CUDA};
  Tensor t = fresh(like, {(int64_t)bytes}, at::kByte);
  t.narrow(0, 0, (int64_t)DG_LAYER_COUNTER_BYTES).zero_();
  return t;
}
Tensor products_workspace(const Site& at, const Tensor& like) {
  if (capturing()) return new_workspace(like);
  const uint64_t key = (uint64_t)at.stream.id() * 64u + (uint64_t)like.device().index();
  State& st = state();
  std::lock_guard<std::mutex> lk(st.mu);
  Tensor& t = st.workspace[key];
  if (!t.defined()) t = new_workspace(like);
  return t;
}

// --------------------------------------------------------------------- norm

PyObject* add_rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want_args(n, 8);
    const Tensor &x = tensor(a[0], "x"), &weight = tensor(a[1], "weight");
    const Tensor residual = maybe(a[2], "residual");
    Tensor scale_in = THPVariable_Check(a[5]) ? tensor(a[5], "scale") : Tensor();
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) return nullptr;
    const at::ScalarType out = dtype(a[4]);
    const bool keep_rstd = a[6] == Py_True, inplace = a[7] == Py_True;
    TORCH_CHECK_TYPE(x.dim() >= 1 && x.scalar_type() == at::kBFloat16,
                     "x must be a bfloat16 tensor with a last dimension to normalise");
    const int64_t hidden = x.size(-1);
    TORCH_CHECK_VALUE(weight.dim() == 1 && weight.size(0) == hidden && weight.is_contiguous(),
                      "weight must be a contiguous vector of ", hidden, " values");
    TORCH_CHECK_TYPE(bf16_or_f32(weight.scalar_type()), "weight must be bfloat16 or float32");
    if (residual.defined()) {
      TORCH_CHECK_VALUE(residual.sizes() == x.sizes(), "residual must have x's shape");
      TORCH_CHECK_TYPE(bf16_or_f32(residual.scalar_type()), "residual must be bfloat16 or float32");
    }
    TORCH_CHECK_VALUE(!inplace || residual.defined(), "inplace needs a residual");
    TORCH_CHECK_VALUE(out == at::kBFloat16 || is8(out), "out_dtype must be bfloat16 or a float8 type, got ", out);
    TORCH_CHECK_VALUE(a[5] == Py_None || is8(out), "a scale needs a float8 out_dtype");
    same_device(x, {&weight, &residual});
    const Site at(x);
    const Tensor x2 = as_rows(x, hidden);
    const int64_t rows = x2.size(0);
    Tensor row_scale, rstd, h, r2;
    if (is8(out)) {
      if (a[5] == Py_None) {
        row_scale = fresh(x, x.sizes().slice(0, x.dim() - 1), at::kFloat);
      } else if (scale_in.defined()) {
        TORCH_CHECK_VALUE(scale_in.numel() == 1 && scale_in.scalar_type() == at::kFloat,
                          "a given scale is a number or a one-element float32 tensor");
        same_device(x, {&scale_in});
      } else {
        const double s = PyFloat_AsDouble(a[5]);
        if (s == -1.0 && PyErr_Occurred()) return nullptr;
        scale_in = at::full({1}, s, x.options().dtype(at::kFloat));
      }
    }
    const Tensor y = fresh(x, x.sizes(), out);
    if (keep_rstd) rstd = fresh(x, x.sizes().slice(0, x.dim() - 1), at::kFloat);
    int64_t h_ld = hidden;
    if (residual.defined()) {
      r2 = as_rows(residual, hidden);
      if (inplace) {
        TORCH_CHECK_VALUE(r2.data_ptr() == residual.data_ptr(), "an in-place residual must have rows that are contiguous");
        h = residual;
        h_ld = r2.stride(0);
        // rows are summed in no particular order
        TORCH_CHECK_VALUE(rows <= 1 || h_ld >= hidden, "the rows of an in-place residual must not overlap");
        const Rows out(r2, rows, h_ld, hidden), in(x2, rows, x2.stride(0), hidden);
        TORCH_CHECK_VALUE((x2.scalar_type() == r2.scalar_type() && out.same(in)) || !out.meet(in),
                          "an in-place residual must not share memory with other values of x");
        TORCH_CHECK_VALUE(!out.meet(Rows(weight, 1, 0, hidden)) && !(scale_in.defined() && out.meet(Rows(scale_in, 1, 0, 1))),
                          "an in-place residual must not share memory with the weight or the scale");
        // as torch's in-place operations: a graph that saved the tensor finds it changed
        h.unsafeGetTensorImpl()->bump_version();
      } else {
        h = fresh(x, x.sizes(), residual.scalar_type());
      }
    }
    check_status(dg_layer_add_rms_norm(
        x2.data_ptr(), x2.stride(0), ptr(r2), r2.defined() ? r2.stride(0) : 0,
        r2.defined() ? type_of(r2.scalar_type()) : DG_TYPE_BF16, weight.data_ptr(), type_of(weight.scalar_type()),
        y.data_ptr(), type_of(out), ptr(h), h_ld, static_cast<float*>(ptr(row_scale)),
        static_cast<const float*>(ptr(scale_in)), static_cast<float*>(ptr(rstd)), rows, hidden, (float)eps, at.handle()));
    return Py_BuildValue("(NNNN)", wrap(y), wrap(h.defined() ? h : x), wrap(row_scale), wrap(rstd));
  });
}

PyObject* add_rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want_args(n, 5);
    const Tensor &dy = tensor(a[0], "dy"), &h = tensor(a[1], "h");
    const Tensor weight = tensor(a[2], "weight").contiguous(), rstd = tensor(a[3], "rstd").contiguous();
    const Tensor dh = maybe(a[4], "d_residual");
    TORCH_CHECK_VALUE(h.dim() >= 1, "h must have a last dimension");
    const int64_t hidden = h.size(-1);
    TORCH_CHECK_VALUE(dy.sizes() == h.sizes() && rstd.sizes() == h.sizes().slice(0, h.dim() - 1) && weight.dim() == 1 &&
                          weight.size(0) == hidden,
                      "dy must have h's shape, rstd that of its rows, weight that of one row");
    TORCH_CHECK_VALUE(!dh.defined() || (dh.sizes() == h.sizes() && dh.scalar_type() == h.scalar_type()),
                      "d_residual must have h's shape and type");
    TORCH_CHECK_TYPE(dy.scalar_type() == at::kBFloat16 && rstd.scalar_type() == at::kFloat,
                     "dy must be bfloat16 and rstd float32");
    TORCH_CHECK_TYPE(bf16_or_f32(h.scalar_type()) && bf16_or_f32(weight.scalar_type()),
                     "h and weight must be bfloat16 or float32");
    same_device(h, {&dy, &weight, &rstd, &dh});
    const Site at(h);
    const Tensor dy2 = as_rows(dy, hidden), h2 = as_rows(h, hidden), d2 = dh.defined() ? as_rows(dh, hidden) : dh;
    const int64_t rows = h2.size(0);
    const Tensor dx = fresh(h, h.sizes(), h.scalar_type()), dw = fresh(h, weight.sizes(), weight.scalar_type());
    const Tensor ws = fresh(h, {(int64_t)dg_layer_add_rms_norm_backward_workspace(rows, hidden)}, at::kByte);
    check_status(dg_layer_add_rms_norm_backward(
        dy2.data_ptr(), dy2.stride(0), h2.data_ptr(), h2.stride(0), type_of(h2.scalar_type()), weight.data_ptr(),
        type_of(weight.scalar_type()), static_cast<const float*>(rstd.data_ptr()), ptr(d2),
        d2.defined() ? d2.stride(0) : 0, dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), rows, hidden, at.handle()));
    return Py_BuildValue("(NN)", wrap(dx), wrap(dw));
  });
}

// ----------------------------------------------------------------- products

void check_grouped(const Tensor& A, const Tensor& B, const Tensor& ends) {
  TORCH_CHECK_VALUE(A.dim() == 2 && B.dim() == 3 && B.size(1) == A.size(1), "A must be (T, K) and B (experts, K, N), got ",
                    A.sizes(), " and ", B.sizes());
  TORCH_CHECK_VALUE(ends.scalar_type() == at::kInt && ends.dim() == 1 && ends.size(0) == B.size(0),
                    "group_ends must be an int32 vector with one ascending end for each expert");
  same_device(A, {&B, &ends});
}

// How a (experts, K, N) B (`swapped`: its transpose) is read: in place when its K
// rows (or, in bf16, its N rows) are contiguous, aligned and apart from each
// other, else from a copy with K rows.
struct Experts {
  Tensor B;
  int64_t K, N, ld, ld_e;
  int n_major;
  Experts(const Tensor& b, bool f8, bool swapped) : B(b) {
    const int dk = swapped ? 2 : 1, dn = swapped ? 1 : 2;
    const int64_t E = b.size(0), sk = b.stride(dk), sn = b.stride(dn);
    K = b.size(dk), N = b.size(dn), ld_e = b.stride(0);
    const bool apart = E == 1 || (ld_e > 0 && ld_e * b.element_size() % 16 == 0);
    if (apart && sk == 1 && sn >= K && aligned(b, sn)) {
      ld = sn, n_major = 0;
    } else if (apart && !f8 && sn == 1 && sk >= N && aligned(b, sk)) {
      ld = sk, n_major = 1;
    } else {
      B = fresh(b, {E, N, K}, b.scalar_type()).copy_(swapped ? b : b.transpose(1, 2));
      ld = K, ld_e = N * K, n_major = 0;
    }
  }
};

Tensor grouped(const Tensor& A_, const Tensor& B, bool swapped, const Tensor& ends_, const Tensor& sa, const Tensor& sb,
               at::ScalarType out, const Site& at) {
  const int64_t T = A_.size(0), E = B.size(0);
  const Tensor A = as_operand(A_), ends = ends_.contiguous();
  const Experts ex(B, is8(B.scalar_type()), swapped);
  const Tensor D = fresh(A, {T, ex.N}, out);
  const Tensor ws = products_workspace(at, A);
  auto stride = [](const Tensor& t, int d) { return t.defined() && t.size(d) > 1 ? t.stride(d) : 0; };
  check_status(dg_layer_grouped_matmul(
      A.data_ptr(), A.stride(0), type_of(A.scalar_type()), ex.B.data_ptr(), ex.ld, ex.ld_e, type_of(B.scalar_type()),
      ex.n_major, static_cast<const int32_t*>(ends.data_ptr()), (int)E, static_cast<const float*>(ptr(sa)), stride(sa, 0),
      static_cast<const float*>(ptr(sb)), stride(sb, 0), stride(sb, 1), D.data_ptr(), type_of(out), T, ex.N, ex.K,
      ws.data_ptr(), status_word(at, A), at.handle()));
  return D;
}

// A fp32 scale or None.
Tensor scale_of(PyObject* o, const char* what) {
  if (o == Py_None) return Tensor();
  TORCH_CHECK_TYPE(THPVariable_Check(o) && THPVariable_Unpack(o).scalar_type() == at::kFloat, what,
                   " must be a float32 tensor");
  return tensor(o, what);
}
// The same seen as `shape` (stride 0 where it is shared).
Tensor scale_as(Tensor t, at::IntArrayRef shape, const char* what) {
  if (!t.defined() || t.sizes() == shape) return t;
  if (shape.size() == 2 && t.dim() == 1) t = t.unsqueeze(1);  // one for each expert
  bool fits = t.dim() <= (int64_t)shape.size();
  for (int64_t d = 1; fits && d <= t.dim(); ++d) fits = t.size(-d) == 1 || t.size(-d) == shape[shape.size() - d];
  TORCH_CHECK_VALUE(fits, what, " of shape ", t.sizes(), " does not broadcast to ", shape);
  return t.expand(shape);
}

PyObject* grouped_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want_args(n, 6);
    const Tensor &A = tensor(a[0], "A"), &B = tensor(a[1], "B"), &ends = tensor(a[2], "group_ends");
    const Tensor scale_a = scale_of(a[3], "scale_a"), scale_b = scale_of(a[4], "scale_b");
    const at::ScalarType out = dtype(a[5]), ta = A.scalar_type(), tb = B.scalar_type();
    check_grouped(A, B, ends);
    TORCH_CHECK_TYPE((ta == at::kBFloat16 && tb == at::kBFloat16) || (is8(ta) && is8(tb)),
                     "A and B must be both bfloat16 or both float8, got ", ta, " and ", tb);
    TORCH_CHECK_VALUE(bf16_or_f32(out), "out_dtype must be bfloat16 or float32, got ", out);
    const Tensor sa = scale_as(scale_a, {A.size(0)}, "scale_a"), sb = scale_as(scale_b, {B.size(0), B.size(2)}, "scale_b");
    same_device(A, {&sa, &sb});
    const Site at(A);
    return wrap(grouped(A, B, false, ends, sa, sb, out, at));
  });
}

// (experts, rows' columns, feats' columns): the sum over each group of
// rows[t, :, None] * feats[t, None, :]; `swapped`: seen as its transpose.
Tensor weight_grad(const Tensor& rows_, const Tensor& feats_, bool swapped, const Tensor& ends_, const Site& at) {
  const Tensor rows = as_operand(rows_), feats = as_operand(feats_), ends = ends_.contiguous();
  const int64_t T = rows.size(0), N = rows.size(1), K = feats.size(1), E = ends.size(0);
  const Tensor out = swapped ? at::detail::empty_strided_cuda({E, K, N}, {N * K, 1, K}, rows.scalar_type(), rows.device())
                             : at::detail::empty_cuda({E, N, K}, rows.scalar_type(), rows.device(), std::nullopt);
  const Tensor ws = fresh(rows, {(int64_t)dg_layer_grouped_grad_workspace((int)E, N, K)}, at::kByte);
  check_status(dg_layer_grouped_weight_grad(rows.data_ptr(), rows.stride(0), feats.data_ptr(), feats.stride(0),
                                            static_cast<const int32_t*>(ends.data_ptr()), (int)E, out.data_ptr(),
                                            DG_TYPE_BF16, T, N, K, ws.data_ptr(), products_workspace(at, rows).data_ptr(),
                                            status_word(at, rows), at.handle()));
  return out;
}

PyObject* grouped_matmul_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want_args(n, 6);
    const Tensor &dD = tensor(a[0], "dD"), &A = tensor(a[1], "A"), &B = tensor(a[2], "B"), &ends = tensor(a[3], "group_ends");
    check_grouped(A, B, ends);
    TORCH_CHECK_VALUE(dD.dim() == 2 && dD.size(0) == A.size(0) && dD.size(1) == B.size(2), "dD must be (", A.size(0), ", ",
                      B.size(2), "), got ", dD.sizes());
    TORCH_CHECK_TYPE(dD.scalar_type() == at::kBFloat16 && A.scalar_type() == at::kBFloat16 &&
                         B.scalar_type() == at::kBFloat16,
                     "dD, A and B must be bfloat16");
    same_device(A, {&dD});
    const Site at(A);
    Tensor dA, dB;
    if (a[4] == Py_True) dA = grouped(dD, B, true, ends, Tensor(), Tensor(), at::kBFloat16, at);
    if (a[5] == Py_True)
      dB = B.stride(2) == 1 && B.stride(1) != 1 ? weight_grad(A, dD, false, ends, at)  // contiguous along N
                                                : weight_grad(dD, A, true, ends, at);
    return Py_BuildValue("(NN)", wrap(dA), wrap(dB));
  });
}

// ------------------------------------------------------- microscaled 4 bits

PyObject* quantize_mx4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want_args(n, 1);
    const Tensor& x = tensor(a[0], "x");
    TORCH_CHECK_TYPE(bf16_or_f32(x.scalar_type()), "x must be bfloat16 or float32, got ", x.scalar_type());
    TORCH_CHECK_VALUE(x.dim() >= 1, "x must have a last dimension");
    const int64_t cols = x.size(-1);
    same_device(x, {});
    TORCH_CHECK_VALUE(cols % 32 == 0, "the last dimension (", cols, ") must be a multiple of 32");
    const Site at(x);
    Tensor x2 = as_rows(x, cols);
    if (!aligned(x2, x2.stride(0))) x2 = fresh(x2, x2.sizes(), x2.scalar_type()).copy_(x2);
    const int64_t rows = x2.size(0);
    const Tensor codes = fresh(x, {rows, cols / 2}, at::kByte);
    const Tensor scales = fresh(x, {(rows + 127) / 128, (cols + 255) / 256 * 2, 512}, at::kByte);
    check_status(dg_layer_mx4_quantize(x2.data_ptr(), x2.stride(0), type_of(x2.scalar_type()), codes.data_ptr(),
                                       scales.data_ptr(), rows, cols, at.handle()));
    return Py_BuildValue("(NNLL)", wrap(codes), wrap(scales), (long long)rows, (long long)cols);
  });
}

// A (codes, scales, rows, cols) tuple.
struct Mx4 {
  Tensor codes, scales;
  int64_t rows, cols;
  Mx4(PyObject* o, const char* what) {
    TORCH_CHECK_TYPE(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 4, what, " must be an MX4Tensor");
    codes = tensor(PyTuple_GET_ITEM(o, 0), "codes");
    scales = tensor(PyTuple_GET_ITEM(o, 1), "scales");
    rows = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 2));
    cols = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 3));
    TORCH_CHECK_TYPE(!PyErr_Occurred(), what, ".rows and .cols must be whole numbers");
    TORCH_CHECK_VALUE(rows >= 0 && cols >= 0 && cols % 32 == 0, what, ".cols must be a multiple of 32");
    TORCH_CHECK_VALUE(codes.scalar_type() == at::kByte && codes.is_contiguous() && codes.dim() == 2 &&
                          codes.size(0) == rows && codes.size(1) == cols / 2,
                      what, ".codes must be contiguous uint8 of shape (", rows, ", ", cols / 2, ")");
    const int64_t rt = (rows + 127) / 128, ct = (cols + 255) / 256 * 2;
    TORCH_CHECK_VALUE(scales.scalar_type() == at::kByte && scales.is_contiguous() && scales.dim() == 3 &&
                          scales.size(0) == rt && scales.size(1) == ct && scales.size(2) == 512,
                      what, ".scales must be contiguous uint8 of shape (", rt, ", ", ct, ", 512)");
    same_device(codes, {&scales});
  }
};

PyObject* dequantize_mx4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want_args(n, 2);
    const Mx4 q(a[0], "q");
    const at::ScalarType out = dtype(a[1]);
    TORCH_CHECK_VALUE(bf16_or_f32(out), "out_dtype must be bfloat16 or float32, got ", out);
    const Site at(q.codes);
    const Tensor y = fresh(q.codes, {q.rows, q.cols}, out);
    check_status(dg_layer_mx4_dequantize(q.codes.data_ptr(), q.scales.data_ptr(), y.data_ptr(), type_of(out), q.rows,
                                         q.cols, at.handle()));
    return wrap(y);
  });
}

PyObject* mx4_matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want_args(n, 3);
    const Mx4 p(a[0], "a"), q(a[1], "b");
    const at::ScalarType out = dtype(a[2]);
    TORCH_CHECK_VALUE(p.cols == q.cols, "a has ", p.cols, " columns, b ", q.cols);
    TORCH_CHECK_VALUE(bf16_or_f32(out), "out_dtype must be bfloat16 or float32, got ", out);
    same_device(p.codes, {&q.codes});
    const Site at(p.codes);
    const Tensor D = fresh(p.codes, {p.rows, q.rows}, out);
    const Tensor ws = products_workspace(at, p.codes);
    check_status(dg_layer_mx4_matmul(p.codes.data_ptr(), p.scales.data_ptr(), q.codes.data_ptr(), q.scales.data_ptr(),
                                     D.data_ptr(), type_of(out), p.rows, q.rows, p.cols, ws.data_ptr(),
                                     status_word(at, p.codes), at.handle()));
    return wrap(D);
  });
}

// ------------------------------------------------------------------- module

PyObject* check(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want_args(n, 1);
    const long index = PyLong_AsLong(a[0]);
    if (index == -1 && PyErr_Occurred()) return nullptr;
    const Tensor like = at::empty({0}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, (c10::DeviceIndex)index));
    const Site at(like);
    void* word = status_word(at, like);
    int rc;
    Py_BEGIN_ALLOW_THREADS rc = dg_layer_check(word, at.handle());
    Py_END_ALLOW_THREADS if (rc != DG_OK) {
      // a product that gave up leaves its counters as they were
      State& st = state();
      std::lock_guard<std::mutex> lk(st.mu);
      st.workspace.clear();
    }
    check_status(rc);
    Py_RETURN_NONE;
  });
}

PyObject* clear_workspaces(PyObject*, PyObject* const*, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    State& st = state();
    std::lock_guard<std::mutex> lk(st.mu);
    st.workspace.clear();
    Py_RETURN_NONE;
  });
}

PyObject* set_error(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    want_args(n, 1);
    Py_INCREF(a[0]);
    Py_XDECREF(g_error);
    g_error = a[0];
    Py_RETURN_NONE;
  });
}

#define DGL_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {DGL_METHOD(add_rms_norm),
                           DGL_METHOD(add_rms_norm_backward),
                           DGL_METHOD(grouped_matmul),
                           DGL_METHOD(grouped_matmul_backward),
                           DGL_METHOD(quantize_mx4),
                           DGL_METHOD(dequantize_mx4),
                           DGL_METHOD(mx4_matmul),
                           DGL_METHOD(check),
                           DGL_METHOD(clear_workspaces),
                           DGL_METHOD(set_error),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "dg_layer_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_dg_layer_torch() { return PyModule_Create(&g_module); }
