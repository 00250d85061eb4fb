// Python binding of the LM-head and log-probability entry points of libdspark.so, over torch tensors.
//
// What it does is what the ctypes wrappers of the other entry points do -- check dtype, shape, device and
// strides, allocate the outputs that were not passed, hand raw pointers and the current stream to the C
// ABI of include/dspark.h -- in compiled code, because these calls are also made for one token at a time:
// through ctypes a token_logprobs call took 18 us of host time for 16 us of kernel.

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <string>
#include <vector>

#include "../../include/dspark.h"

namespace {

using at::Tensor;
using OptTensor = std::optional<Tensor>;

void need(bool ok, const char* name, const char* what) {
  if (!ok) throw py::value_error(std::string(name) + " " + what);
}

// Raise the package's DsparkError for a status other than OK.
void check(const char* fn, int status) {
  if (status == DSPARK_OK) return;
  const std::string msg = dspark_last_error();
  const py::object cls = py::module_::import("speculative_decoding_04_b200.dspark").attr("DsparkError");
  PyErr_SetObject(cls.ptr(), cls(fn, status, msg).ptr());
  throw py::error_already_set();
}

int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return DSPARK_F32;
    case at::kBFloat16: return DSPARK_BF16;
    case at::kHalf: return DSPARK_F16;
    default: return -1;
  }
}

// A tensor as rows without a copy: the last dimension dense, the rows a constant stride apart.
struct Rows {
  char* p;
  int64_t rows, cols, ld;
};

Rows rows_of(const Tensor& t, const char* name) {
  need(t.is_cuda(), name, "must be a CUDA tensor");
  const int64_t nd = t.dim();
  need(nd >= 2, name, "must have at least 2 dimensions");
  Rows r{static_cast<char*>(t.data_ptr()), 1, t.size(nd - 1), 0};
  for (int64_t d = 0; d < nd - 1; ++d) r.rows *= t.size(d);
  r.ld = std::max<int64_t>(1, r.cols);
  if (r.rows <= 1 && (r.cols <= 1 || t.stride(nd - 1) == 1)) return r;
  if (t.is_contiguous()) return r;
  need(r.cols <= 1 || t.stride(nd - 1) == 1, name, "must have a dense last dimension");
  int64_t step = -1, span = 0;  // stride of a row, and what the next outer dimension's has to be
  for (int64_t d = nd - 2; d >= 0; --d) {
    if (t.size(d) == 1) continue;
    if (step < 0) step = t.stride(d);
    else need(t.stride(d) == span, name, "must have rows a constant stride apart");
    span = t.stride(d) * t.size(d);
  }
  need(step >= r.cols, name, "must have rows that do not overlap");
  r.ld = step;
  return r;
}

Rows floats(const Tensor& t, const char* name) {
  need(dtype_code(t.scalar_type()) >= 0, name, "must be fp32, bf16 or fp16");
  return rows_of(t, name);
}

Rows like(const Tensor& t, const char* name, const Tensor& ref, at::ScalarType dtype) {
  need(t.scalar_type() == dtype, name, "has the wrong dtype");
  need(t.device() == ref.device(), name, "is on another device");
  need(t.sizes() == ref.sizes(), name, "has the wrong shape");
  return rows_of(t, name);
}

// The address of a contiguous argument of n values on ref's device (nullptr if it was not given).
template <typename T>
T* arg(const Tensor& t, const char* name, at::ScalarType dtype, int64_t n, const Tensor& ref) {
  need(t.scalar_type() == dtype, name, "has the wrong dtype");
  need(t.device() == ref.device(), name, "is on another device");
  need(t.numel() == n && t.is_contiguous(), name, "must be contiguous with one value per entry");
  return static_cast<T*>(t.data_ptr());
}
template <typename T>
T* arg(const OptTensor& t, const char* name, at::ScalarType dtype, int64_t n, const Tensor& ref) {
  return t ? arg<T>(*t, name, dtype, n, ref) : nullptr;
}

std::vector<int64_t> shape(at::IntArrayRef lead, std::initializer_list<int64_t> tail) {
  std::vector<int64_t> s(lead.begin(), lead.end());
  s.insert(s.end(), tail);
  return s;
}

// A new tensor on ref's device, from the allocator directly: through the dispatcher an output costs 1 us
// of host time, and token_logprobs has five.
Tensor fresh(at::IntArrayRef sizes, at::ScalarType dtype, const Tensor& ref) {
  return at::detail::empty_cuda(sizes, dtype, ref.device(), std::nullopt);
}

Tensor given_or_new(const OptTensor& t, at::IntArrayRef sizes, at::ScalarType dtype, const Tensor& ref) {
  return t ? *t : fresh(sizes, dtype, ref);
}

int size32(int64_t n, const char* name) {
  need(n <= INT32_MAX, name, "is too large");
  return static_cast<int>(n);
}

void* current_stream(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

py::tuple token_logprobs(const Tensor& logits, const Tensor& tokens, double T, int64_t top, const OptTensor& rows,
                         const OptTensor& logp_, const OptTensor& entropy_, const OptTensor& top_idx_,
                         const OptTensor& top_logp_, const OptTensor& stats_, const OptTensor& flags) {
  const Rows l = floats(logits, "logits");
  const c10::cuda::CUDAGuard guard(logits.device());
  const int N = size32(tokens.numel(), "tokens"), V = size32(l.cols, "V");
  const int32_t* tok = arg<int32_t>(tokens, "tokens", at::kInt, N, logits);
  const int64_t* row = arg<int64_t>(rows, "rows", at::kLong, N, logits);
  const auto lead = tokens.sizes();
  const Tensor logp = given_or_new(logp_, shape(lead, {}), at::kFloat, logits);
  const Tensor entropy = given_or_new(entropy_, shape(lead, {}), at::kFloat, logits);
  const Tensor stats = given_or_new(stats_, shape(lead, {2}), at::kFloat, logits);
  py::object idx_out = py::none(), lp_out = py::none();
  int32_t* ti = nullptr;
  float* tl = nullptr;
  const bool some = top > 0 && top <= DSPARK_TOP_MAX;  // (anything else is refused below)
  if (some) {
    const Tensor a = given_or_new(top_idx_, shape(lead, {top}), at::kInt, logits);
    const Tensor b = given_or_new(top_logp_, shape(lead, {top}), at::kFloat, logits);
    ti = arg<int32_t>(a, "top_idx", at::kInt, N * top, logits);
    tl = arg<float>(b, "top_logp", at::kFloat, N * top, logits);
    idx_out = py::cast(a);
    lp_out = py::cast(b);
  }
  check("dspark_token_logprobs",
        dspark_token_logprobs(l.p, dtype_code(logits.scalar_type()), l.ld, l.rows, row, tok, N, V, static_cast<float>(T),
                              static_cast<int>(std::max<int64_t>(-1, std::min<int64_t>(top, DSPARK_TOP_MAX + 1))),
                              arg<float>(logp, "logp", at::kFloat, N, logits),
                              arg<float>(entropy, "entropy", at::kFloat, N, logits), ti, tl,
                              arg<float>(stats, "stats", at::kFloat, 2ll * N, logits),
                              reinterpret_cast<uint32_t*>(arg<int32_t>(flags, "flags", at::kInt, N, logits)),
                              current_stream(logits)));
  return py::make_tuple(logp, entropy, idx_out, lp_out, stats);
}

Tensor token_logprobs_backward(const Tensor& logits, const Tensor& tokens, double T, const Tensor& stats,
                               const OptTensor& entropy, const OptTensor& g_logp, const OptTensor& g_entropy,
                               const OptTensor& top_idx, const OptTensor& g_top, const OptTensor& grad_) {
  const Rows l = floats(logits, "logits");
  const c10::cuda::CUDAGuard guard(logits.device());
  const int N = size32(l.rows, "logits"), V = size32(l.cols, "V");
  const int32_t* tok = arg<int32_t>(tokens, "tokens", at::kInt, N, logits);
  need(top_idx.has_value() == g_top.has_value(), "top_idx", "and g_top come together");
  int64_t top = 0;
  if (top_idx && N > 0) {
    need(top_idx->numel() % N == 0, "top_idx", "must have the same number of alternatives for every row");
    top = top_idx->numel() / N;
  }
  Tensor grad;
  Rows g;
  if (grad_) {
    grad = *grad_;
    g = like(grad, "grad", logits, logits.scalar_type());
  } else {
    // Rows as far apart as the logits', so that both start at the same offset within 16 bytes; where a lot
    // lies between the logits' rows (one position of each request), the nearest such distance.
    const int64_t vec = 16 / logits.element_size(), most = l.cols + std::max<int64_t>(l.cols, 1024);
    const int64_t ldg = l.ld <= most ? l.ld : l.cols + (l.ld - l.cols) % vec;
    grad = at::detail::empty_strided_cuda({l.rows, l.cols}, {ldg, 1}, logits.scalar_type(), logits.device());
    g = Rows{static_cast<char*>(grad.data_ptr()), l.rows, l.cols, ldg};
    if (logits.dim() != 2) grad = grad.view(logits.sizes());
  }
  check("dspark_token_logprobs_backward",
        dspark_token_logprobs_backward(
            l.p, dtype_code(logits.scalar_type()), l.ld, tok, N, V, static_cast<float>(T),
            arg<float>(stats, "stats", at::kFloat, 2ll * N, logits), arg<float>(entropy, "entropy", at::kFloat, N, logits),
            arg<float>(g_logp, "g_logp", at::kFloat, N, logits), arg<float>(g_entropy, "g_entropy", at::kFloat, N, logits),
            static_cast<int>(std::min<int64_t>(top, DSPARK_TOP_MAX + 1)),
            arg<int32_t>(top_idx, "top_idx", at::kInt, N * top, logits),
            arg<float>(g_top, "g_top", at::kFloat, N * top, logits), g.p, g.ld, current_stream(logits)));
  return grad;
}

// The int8 rows and scales of x's rows, given or new.  New rows start on 16 bytes (what the product reads),
// long ones on 128: a row's 128-byte pieces then lie in one line each (664 x 118128 x 4271: 250 us, 305 with
// rows 4272 bytes apart).
struct Q8 {
  Tensor q, scale;
  int8_t* p;
  float* sp;
  int64_t ld;
};

Q8 q8_out(const Tensor& x, const Rows& r, const OptTensor& q_, const OptTensor& scale_) {
  Q8 o;
  const auto lead = x.sizes().slice(0, x.dim() - 1);
  if (q_) {
    const Rows t = like(*q_, "q", x, at::kChar);
    o.q = *q_;
    o.p = reinterpret_cast<int8_t*>(t.p);
    o.ld = t.ld;
  } else {
    const int64_t step = r.cols >= 512 ? 128 : 16;
    o.ld = (r.cols + step - 1) / step * step;
    o.q = fresh(shape(lead, {o.ld}), at::kChar, x);
    o.p = static_cast<int8_t*>(o.q.data_ptr());
    if (o.ld != r.cols) o.q = o.q.narrow(-1, 0, r.cols);
  }
  o.scale = given_or_new(scale_, shape(lead, {}), at::kFloat, x);
  o.sp = arg<float>(o.scale, "scale", at::kFloat, r.rows, x);
  return o;
}

py::tuple rmsnorm_q8(const Tensor& x, const OptTensor& gain, double eps, const OptTensor& residual,
                     const OptTensor& h_out, const OptTensor& q_, const OptTensor& scale_) {
  const Rows r = floats(x, "x");
  const c10::cuda::CUDAGuard guard(x.device());
  const int M = size32(r.rows, "x"), d = size32(r.cols, "x");
  const auto dt = x.scalar_type();
  const auto gdt = gain && gain->scalar_type() != dt ? at::kFloat : dt;
  const void* gp = gain ? arg<void>(*gain, "gain", gdt, d, x) : nullptr;
  Rows res{nullptr, 0, 0, 0}, h{nullptr, 0, 0, 0};
  py::object hout = py::none();
  if (residual) {
    res = like(*residual, "residual", x, dt);
    if (h_out) {
      h = like(*h_out, "h_out", x, dt);
      hout = py::cast(*h_out);
    } else {
      const Tensor t = fresh(x.sizes(), dt, x);
      h = Rows{static_cast<char*>(t.data_ptr()), r.rows, r.cols, std::max<int64_t>(1, r.cols)};
      hout = py::cast(t);
    }
  }
  const Q8 o = q8_out(x, r, q_, scale_);
  check("dspark_rmsnorm_q8",
        dspark_rmsnorm_q8(r.p, dtype_code(dt), r.ld, res.p, res.ld, gp, dtype_code(gdt), M, d, static_cast<float>(eps), h.p,
                          h.ld, o.p, o.ld, o.sp, current_stream(x)));
  return py::make_tuple(o.q, o.scale, hout);
}

py::tuple quantize_q8(const Tensor& x, const OptTensor& q_, const OptTensor& scale_) {
  const Rows r = floats(x, "x");
  const c10::cuda::CUDAGuard guard(x.device());
  const Q8 o = q8_out(x, r, q_, scale_);
  check("dspark_quantize_q8",
        dspark_quantize_q8(r.p, dtype_code(x.scalar_type()), r.ld, size32(r.rows, "x"), size32(r.cols, "x"), o.p, o.ld, o.sp,
                           current_stream(x)));
  return py::make_tuple(o.q, o.scale);
}

Tensor matmul_q8(const Tensor& q, const Tensor& q_scale, const Tensor& w, const Tensor& w_scale, const py::object& dtype,
                 const OptTensor& out_, const OptTensor& flags) {
  need(q.scalar_type() == at::kChar, "q", "must be int8");
  need(w.scalar_type() == at::kChar, "w", "must be int8");
  Rows a = rows_of(q, "q"), b = rows_of(w, "w");
  const c10::cuda::CUDAGuard guard(q.device());
  need(w.dim() == 2 && w.device() == q.device(), "w", "must be [N, K] on q's device");
  need(a.cols == b.cols, "w", "must have rows as long as q's");
  const int M = size32(a.rows, "q"), N = size32(b.rows, "w"), K = size32(a.cols, "K");
  if (M <= 1) a.ld = (a.cols + 15) / 16 * 16;  // one row's stride says nothing
  if (N <= 1) b.ld = (b.cols + 15) / 16 * 16;
  Tensor out;
  int64_t ldo = std::max(1, N);
  const auto want = shape(q.sizes().slice(0, q.dim() - 1), {N});
  if (out_) {
    out = *out_;
    need(out.device() == q.device() && out.sizes() == at::IntArrayRef(want), "out", "must be [..., N] on q's device");
    ldo = floats(out, "out").ld;
  } else {
    if (!THPDtype_Check(dtype.ptr())) throw py::type_error("out_dtype must be a torch.dtype");
    const auto dt = reinterpret_cast<THPDtype*>(dtype.ptr())->scalar_type;
    need(dtype_code(dt) >= 0, "out_dtype", "must be fp32, bf16 or fp16");
    out = fresh(want, dt, q);
  }
  check("dspark_matmul_q8",
        dspark_matmul_q8(reinterpret_cast<const int8_t*>(a.p), a.ld, arg<float>(q_scale, "q_scale", at::kFloat, M, q),
                         reinterpret_cast<const int8_t*>(b.p), b.ld, arg<float>(w_scale, "w_scale", at::kFloat, N, q), M, N, K,
                         out.data_ptr(), dtype_code(out.scalar_type()), ldo,
                         reinterpret_cast<uint32_t*>(arg<int32_t>(flags, "flags", at::kInt, M, q)), current_stream(q)));
  return out;
}

}  // namespace

PYBIND11_MODULE(_binding, m) {
  m.def("token_logprobs", &token_logprobs);
  m.def("token_logprobs_backward", &token_logprobs_backward);
  m.def("rmsnorm_q8", &rmsnorm_q8);
  m.def("quantize_q8", &quantize_q8);
  m.def("matmul_q8", &matmul_q8);
}
