// Argument marshalling of the many-adapter calls and of the gradient norm in C++: the same
// checks that _binding.py makes for the other calls, and one call of the C ABI. A decode step
// makes many calls of a few microseconds of device time each, and a norm takes hundreds of
// tensors; marshalled in Python, the host set the time (lora_fwd of 32 tokens 23 us against
// 9 us on the device, clip_grad_norm of 64 tensors 121 us against 12 us). Each function
// returns the C ABI's code first; _binding.py turns it into an RdfftError.
#include <ATen/ATen.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <pybind11/pybind11.h>
#include <pybind11/stl.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <initializer_list>
#include <optional>
#include <string>
#include <vector>

#include "adapter_plan.h"
#include "rdfft.h"

namespace py = pybind11;
using at::Tensor;
using MaybeTensor = std::optional<Tensor>;

namespace {

rdfft_stream_t stream_of(const Tensor& t) {
  return reinterpret_cast<rdfft_stream_t>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream());
}

void dense(const Tensor& t, const char* name) {
  if (!t.is_cuda()) throw py::type_error(std::string(name) + " must be a CUDA tensor");
  if (!t.is_contiguous()) throw py::value_error(std::string(name) + " must be contiguous");
}

int dtype_code(const Tensor& t) {
  if (t.scalar_type() == at::kFloat) return RDFFT_F32;
  if (t.scalar_type() == at::kBFloat16) return RDFFT_BF16;
  throw py::type_error("rdfft supports float32 and bfloat16 tensors, got " + std::string(t.dtype().name()));
}

std::string shape_text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

void like(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType dtype, const Tensor& ref) {
  dense(t, name);
  if (t.sizes() != shape || t.scalar_type() != dtype || t.device() != ref.device())
    throw py::value_error(std::string(name) + " must have shape " + shape_text(shape) + ", dtype " +
                          at::toString(dtype) + " and be on " + ref.device().str());
}
void like(const MaybeTensor& t, const char* name, at::IntArrayRef shape, at::ScalarType dtype, const Tensor& ref) {
  if (t) like(*t, name, shape, dtype, ref);
}

// The given tensor, checked, or a new one of that shape.
Tensor out_of(const MaybeTensor& t, const char* name, at::IntArrayRef shape, at::ScalarType dtype, const Tensor& ref) {
  if (!t) return at::empty(shape, ref.options().dtype(dtype));
  like(*t, name, shape, dtype, ref);
  return *t;
}

void* ptr(const Tensor& t) { return t.data_ptr(); }
void* ptr(const MaybeTensor& t) { return t ? t->data_ptr() : nullptr; }
float* fptr(const MaybeTensor& t) { return static_cast<float*>(ptr(t)); }

// The call behind `code` wrote into tensors that the caller gave: a graph that saved one of them must
// not go on with the new values unnoticed. (An inference tensor counts no versions.)
void written(int code, const Tensor& t) {
  if (code == RDFFT_OK && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void written(int code, std::initializer_list<const MaybeTensor*> given) {
  for (const MaybeTensor* t : given)
    if (*t) written(code, **t);
}

py::object maybe(const MaybeTensor& t) { return t ? py::cast(*t) : py::object(py::none()); }

// ------------------------------------------------------------------------------- plan
// The buffer of a plan of T tokens and n adapters: the kernels index it by those sizes.
void plan_buffer(const Tensor& buf, int64_t T, int n, const Tensor& ref) {
  int64_t words = 0;
  const bool sizes = adapter_plan_size(T, n, &words) == RDFFT_OK;
  if (!sizes || !buf.is_cuda() || !buf.is_contiguous() || buf.scalar_type() != at::kInt || buf.numel() < words ||
      buf.device() != ref.device())
    throw py::value_error("the plan's buffer must be adapter_plan's int32 tensor for its " + std::to_string(T) +
                          " tokens and " + std::to_string(n) + " adapters, on " + ref.device().str());
}

py::tuple adapter_plan_(const Tensor& ids, int n, const MaybeTensor& buf) {
  dense(ids, "ids");
  if (ids.scalar_type() != at::kInt || ids.dim() != 1)
    throw py::type_error("ids must be a one-dimensional int32 tensor");
  const int64_t T = ids.numel();
  int64_t words = 0;
  const int rc = adapter_plan_size(T, n, &words);
  if (rc != RDFFT_OK) return py::make_tuple(rc, py::none());
  if (buf) plan_buffer(*buf, T, n, ids);
  const c10::cuda::OptionalCUDAGuard guard(ids.device());
  Tensor plan = buf ? *buf : at::empty({words}, ids.options());
  const int code = adapter_plan(ids.const_data_ptr<int>(), T, n, plan.mutable_data_ptr<int>(), stream_of(ids));
  written(code, {&buf});
  return py::make_tuple(code, plan);
}

// Words [at, at + len) of a plan.
Tensor plan_words(const Tensor& buf, int64_t at, int64_t len) { return buf.narrow(0, at, len); }
Tensor plan_offsets(const Tensor& buf, int64_t T, int n) { return plan_words(buf, rdfft::plan_layout(T, n).offsets, n + 2); }
Tensor plan_order(const Tensor& buf, int64_t T, int n) { return plan_words(buf, rdfft::plan_layout(T, n).order, T); }

void plan_for(const Tensor& plan, int64_t T, int n, const Tensor& rows, int64_t adapters, const char* of) {
  const int64_t width = rows.size(-1);
  if (T != (width ? rows.numel() / width : 0) || n != adapters || plan.device() != rows.device())
    throw py::value_error("the plan is for " + std::to_string(T) + " tokens and " + std::to_string(n) +
                          " adapters on " + plan.device().str() + ", not for " + of);
  plan_buffer(plan, T, n, rows);
}

// --------------------------------------------------------------------------- low rank
struct LoraSizes {
  int K, N, r;
  at::DimVector out;                            // x's leading dimensions and N
};

LoraSizes lora_sizes(const Tensor& x, const Tensor& a, const Tensor& b, const Tensor& plan, int64_t T, int n,
                     const MaybeTensor& scale) {
  dense(x, "x"), dense(a, "a"), dense(b, "b");
  if (a.dim() != 3 || b.dim() != 3 || a.size(0) != b.size(0) || a.size(1) != b.size(2) || x.dim() < 1 ||
      x.size(-1) != a.size(2))
    throw py::value_error("x must have shape (..., K), a (n, r, K) and b (n, N, r)");
  dtype_code(x);
  if (a.scalar_type() != x.scalar_type() || b.scalar_type() != x.scalar_type() || a.device() != x.device() ||
      b.device() != x.device())
    throw py::value_error("a and b must match x in dtype and device");
  plan_for(plan, T, n, x, a.size(0), "x and a");
  like(scale, "scale", {n}, at::kFloat, x);
  const int64_t most = 1 << 30;                 // the C ABI refuses far smaller sizes
  LoraSizes s{(int)std::min(a.size(2), most), (int)std::min(b.size(1), most), (int)std::min(a.size(1), most), {}};
  s.out.append(x.sizes().begin(), x.sizes().end());
  s.out.back() = b.size(1);
  return s;
}

py::tuple lora_fwd_(const Tensor& x, const Tensor& a, const Tensor& b, const Tensor& plan, int64_t T, int n,
                    const MaybeTensor& scale, const MaybeTensor& base, const MaybeTensor& y_, const MaybeTensor& u) {
  const LoraSizes s = lora_sizes(x, a, b, plan, T, n, scale);
  like(base, "base", s.out, x.scalar_type(), x);
  like(u, "u", {T, s.r}, at::kFloat, x);
  const c10::cuda::OptionalCUDAGuard guard(x.device());
  Tensor y = out_of(y_, "y", s.out, x.scalar_type(), x);
  const int code = lora_fwd(ptr(x), ptr(a), ptr(b), fptr(scale), ptr(base), ptr(y), fptr(u),
                            plan.const_data_ptr<int>(), T, s.K, s.N, s.r, n, dtype_code(x), stream_of(x));
  written(code, {&y_, &u});
  return py::make_tuple(code, y);
}

py::tuple lora_bwd_(const Tensor& g, const Tensor& x, const Tensor& a, const Tensor& b, const Tensor& plan, int64_t T,
                    int n, const MaybeTensor& u, const MaybeTensor& scale, bool need_x, bool need_a, bool need_b,
                    const MaybeTensor& grad_x_, const MaybeTensor& grad_a_, const MaybeTensor& grad_b_,
                    const MaybeTensor& workspace) {
  const LoraSizes s = lora_sizes(x, a, b, plan, T, n, scale);
  like(g, "g", s.out, x.scalar_type(), x);
  like(u, "u", {T, s.r}, at::kFloat, x);
  if (need_b && !u) throw py::value_error("grad_b needs the u that lora_fwd writes");
  const c10::cuda::OptionalCUDAGuard guard(x.device());
  MaybeTensor gx, ga, gb, v = workspace;
  if (need_x) gx = out_of(grad_x_, "grad_x", x.sizes(), x.scalar_type(), x);
  if (need_a) ga = out_of(grad_a_, "grad_a", a.sizes(), at::kFloat, x);
  if (need_b) gb = out_of(grad_b_, "grad_b", b.sizes(), at::kFloat, x);
  if (need_a) v = out_of(workspace, "workspace", {T, s.r}, at::kFloat, x);
  like(v, "workspace", {T, s.r}, at::kFloat, x);
  const int code = lora_bwd(ptr(g), ptr(x), ptr(a), ptr(b), fptr(scale), fptr(u), fptr(v), ptr(gx), fptr(ga), fptr(gb),
                            plan.const_data_ptr<int>(), T, s.K, s.N, s.r, n, dtype_code(x), stream_of(x));
  if (need_x) written(code, {&grad_x_});
  if (need_a) written(code, {&grad_a_});
  if (need_b) written(code, {&grad_b_});
  if (need_x || need_a) written(code, {&workspace});
  return py::make_tuple(code, maybe(gx), maybe(ga), maybe(gb));
}

// -------------------------------------------------------------------- block circulant
int circ_D(const Tensor& x, const Tensor& c_hat, int64_t p, const Tensor& plan, int64_t T, int n) {
  dense(x, "x"), dense(c_hat, "c_hat");
  if (c_hat.scalar_type() != at::kFloat || c_hat.device() != x.device())
    throw py::type_error("c_hat must be float32 on x's device");
  if (c_hat.dim() != 4 || c_hat.size(1) != c_hat.size(2) || c_hat.size(3) != p || x.dim() < 1 ||
      x.size(-1) != c_hat.size(1) * p)
    throw py::value_error("x must have shape (..., q * p) and c_hat (n, q, q, p)");
  plan_for(plan, T, n, x, c_hat.size(0), "x and c_hat");
  return (int)std::min<int64_t>(x.size(-1), 1 << 30);
}

py::tuple circ_fwd_many_(const Tensor& x, const Tensor& c_hat, int p, const Tensor& plan, int64_t T, int n,
                         const MaybeTensor& base, const MaybeTensor& y_) {
  const int D = circ_D(x, c_hat, p, plan, T, n);
  const int code_of_type = dtype_code(x);
  like(base, "base", x.sizes(), x.scalar_type(), x);
  const c10::cuda::OptionalCUDAGuard guard(x.device());
  Tensor y = out_of(y_, "y", x.sizes(), x.scalar_type(), x);
  const int code = circ_fwd_many(ptr(x), c_hat.const_data_ptr<float>(), ptr(base), ptr(y), plan.const_data_ptr<int>(),
                                 T, D, p, n, code_of_type, stream_of(x));
  written(code, {&y_});
  return py::make_tuple(code, y);
}

py::tuple circ_bwd_many_(const Tensor& g, const Tensor& x, const Tensor& c_hat, int p, const Tensor& plan, int64_t T,
                         int n, const MaybeTensor& grad_x_, const MaybeTensor& grad_c_, bool need_x, bool need_c,
                         const MaybeTensor& workspace_) {
  const int D = circ_D(x, c_hat, p, plan, T, n);
  const int type = dtype_code(x);
  like(g, "g", x.sizes(), x.scalar_type(), x);
  const c10::cuda::OptionalCUDAGuard guard(x.device());
  MaybeTensor gx, gc, ws = workspace_;
  if (need_x) gx = out_of(grad_x_, "grad_x", x.sizes(), x.scalar_type(), x);
  if (need_c) {
    gc = out_of(grad_c_, "grad_c", c_hat.sizes(), at::kFloat, x);
    size_t need = 0;
    const int rc = circ_bwd_many_workspace_size(T, D, p, n, type, need_x, &need);
    if (rc != RDFFT_OK) return py::make_tuple(rc, py::none(), py::none());
    if (!ws && need) ws = at::empty({(int64_t)need}, x.options().dtype(at::kByte));
  }
  if (ws) {
    dense(*ws, "workspace");
    if (ws->device() != x.device()) throw py::value_error("workspace must be on x's device");
  }
  const int code = circ_bwd_many(ptr(g), ptr(x), c_hat.const_data_ptr<float>(), ptr(gx), fptr(gc),
                                 plan.const_data_ptr<int>(), T, D, p, n, type, ptr(ws), ws ? ws->nbytes() : 0,
                                 stream_of(x));
  if (need_x) written(code, {&grad_x_});
  if (need_c) written(code, {&grad_c_, &workspace_});
  return py::make_tuple(code, maybe(gx), maybe(gc));
}

// ----------------------------------------------------------------------- gradient norm
struct List {
  std::vector<void*> ptrs;
  std::vector<int64_t> numels;
  std::vector<int> codes;
  Tensor first;
};

List list_of(const py::list& ts, const char* name) {
  const size_t m = ts.size();
  if (m == 0) throw py::value_error(std::string(name) + ": at least one tensor is needed");
  List l;
  l.ptrs.reserve(m), l.numels.reserve(m), l.codes.reserve(m);
  for (size_t i = 0; i < m; ++i) {
    PyObject* o = PyList_GET_ITEM(ts.ptr(), (Py_ssize_t)i);
    if (!THPVariable_Check(o)) throw py::type_error(std::string(name) + " must be tensors");
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || !t.is_contiguous() || (t.scalar_type() != at::kFloat && t.scalar_type() != at::kBFloat16))
      throw py::type_error(std::string(name) + " must be contiguous float32 or bfloat16 CUDA tensors");
    if (i == 0) l.first = t;
    if (t.get_device() != l.first.get_device()) throw py::value_error(std::string(name) + " must be on one device");
    l.ptrs.push_back(t.data_ptr());
    l.numels.push_back(t.numel());
    l.codes.push_back(t.scalar_type() == at::kBFloat16 ? RDFFT_BF16 : RDFFT_F32);
  }
  return l;
}

// (code, norm); out empty: the norm alone.
py::tuple norm_(const py::list& ts, bool clip, double max_norm, const std::optional<py::list>& out) {
  const List in = list_of(ts, "tensors");
  List o;
  if (out) {
    o = list_of(*out, "out");
    if (o.numels != in.numels || o.codes != in.codes || o.first.device() != in.first.device())
      throw py::value_error("out must match the tensors in number, element counts, dtypes and device");
  }
  const int count = (int)std::min<size_t>(ts.size(), 1 << 30);
  size_t need = 0;
  const int rc = grad_norm_workspace_size(count, &need);
  if (rc != RDFFT_OK) return py::make_tuple(rc, py::none());
  const c10::cuda::OptionalCUDAGuard guard(in.first.device());
  // memory of its own for the norm: a caller may keep it long after the workspace, which needs no
  // tensor around it (0.5 us of the 11 that 64 tensors take)
  const c10::DataPtr ws = c10::cuda::CUDACachingAllocator::get()->allocate(need);
  const Tensor norm = at::empty({}, in.first.options().dtype(at::kFloat));
  float* const n = norm.mutable_data_ptr<float>();
  const void* const* grads = const_cast<const void* const*>(in.ptrs.data());
  const int code =
      clip ? clip_grad_norm(grads, out ? o.ptrs.data() : in.ptrs.data(), in.numels.data(), in.codes.data(), count,
                            (float)max_norm, n, ws.get(), need, stream_of(norm))
           : grad_norm(grads, in.numels.data(), in.codes.data(), count, n, ws.get(), need, stream_of(norm));
  if (clip)
    for (py::handle t : out ? *out : ts) written(code, THPVariable_Unpack(t.ptr()));
  return py::make_tuple(code, norm);
}

}  // namespace

PYBIND11_MODULE(_native, m) {
  m.def("adapter_plan", &adapter_plan_);
  m.def("plan_offsets", &plan_offsets);
  m.def("plan_order", &plan_order);
  m.def("lora_fwd", &lora_fwd_);
  m.def("lora_bwd", &lora_bwd_);
  m.def("circ_fwd_many", &circ_fwd_many_);
  m.def("circ_bwd_many", &circ_bwd_many_);
  m.def("norm", &norm_);
}
