// binding.cpp -- the block norm and the gated delta rule as functions on torch tensors
// (module gated_norm_b200._marshal): checks, output allocation and descriptors for the C entry
// points of include/gnorm.h.  In C++ because the calls of a decoding step or a small batch take
// the GPU a few microseconds, and the same checks in Python take three times the launch.
//
// Every function returns the C entry point's status first; the Python side raises on it.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <initializer_list>
#include <optional>
#include <string>
#include <tuple>

#include "gnorm.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

std::string shape_of(const Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

[[noreturn]] void bad_type(const char* name, const char* want, const Tensor& t) {
  throw py::type_error(std::string(name) + " must be " + want + ", got " +
                       c10::toString(t.scalar_type()));
}
[[noreturn]] void bad_value(const std::string& what) { throw py::value_error(what); }

constexpr int kBf16 = 1, kFp32 = 2;  // accepted types

void check_type(const Tensor& t, const char* name, int types) {
  const auto s = t.scalar_type();
  if ((s == at::kBFloat16 && (types & kBf16)) || (s == at::kFloat && (types & kFp32))) return;
  bad_type(name, types == kBf16 ? "bfloat16" : types == kFp32 ? "float32" : "bfloat16 or float32", t);
}
int type_of(const Tensor& t) { return t.scalar_type() == at::kFloat ? kFp32 : kBf16; }

// A stride of more than one row, token or slot, as a descriptor takes it.  There 0 means "packed",
// while a tensor's 0 (`expand`) means one row in the place of all: never passed on.
int64_t distance(int64_t stride, const char* name, const char* what) {
  if (stride == 0)
    bad_value(std::string(name) + ": its " + what + " share memory (an expanded tensor); pass " + name +
              ".contiguous()");
  return stride;
}

void* ptr(const Tensor& t) { return t.numel() ? t.data_ptr() : nullptr; }
void* ptr(const OptTensor& t) { return t ? ptr(*t) : nullptr; }

// The stream a call runs on: the caller's handle, or torch's current one of the device; and the
// allocations of the call follow it.
struct Here {
  c10::cuda::CUDAGuard device;
  std::optional<c10::cuda::CUDAStreamGuard> own;
  void* stream;
  Here(const at::Device& d, std::optional<uintptr_t> handle) : device(d) {
    if (handle) {
      const auto s = c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(*handle), d.index());
      own.emplace(s);
      stream = reinterpret_cast<void*>(*handle);
    } else {
      stream = c10::cuda::getCurrentCUDAStream(d.index()).stream();
    }
  }
};

Tensor scratch(const OptTensor& given, size_t need, const at::Device& dev) {
  if (!given) {
    // from torch's allocator for every call: ordered on the stream that uses it, and owned by
    // the graph when the call is captured
    return at::empty({static_cast<int64_t>(need)}, at::TensorOptions().dtype(at::kByte).device(dev));
  }
  if (given->device() != dev || !given->is_contiguous())
    bad_value("workspace_buf must be a contiguous tensor on " + dev.str());
  return *given;
}

// ------------------------------------------------------------------------- block norm

// Row stride of rows of the last dimension: contiguous of any rank, or a 2-D view with unit
// column stride.
int64_t rows(const Tensor& t, const char* name, int types, const Tensor* like) {
  check_type(t, name, types);
  if (like != nullptr) {
    if (t.sizes() != like->sizes())
      bad_value("a " + shape_of(*like) + " and " + name + " " + shape_of(t) + " differ");
    if (t.device() != like->device()) bad_value(std::string("a and ") + name + " are on different devices");
  } else if (t.dim() < 1) {
    bad_value(std::string(name) + " must have a last dimension N");
  }
  int64_t ld = t.size(-1);
  if (!t.is_contiguous()) {
    if (t.dim() != 2 || t.stride(1) != 1)
      bad_value(std::string(name) + ": rows need unit column stride (2-D row-strided views or contiguous tensors)");
    if (t.size(0) > 1) ld = distance(t.stride(0), name, "rows");
  }
  if (!t.is_cuda()) bad_value(std::string(name) + " must be a CUDA tensor");
  return ld;
}

void vec(const Tensor& t, int64_t n, int types, const char* name, const at::Device& dev) {
  check_type(t, name, types);
  if (t.numel() != n || !t.is_contiguous() || t.device() != dev)
    bad_value(std::string(name) + " must be a contiguous [" + std::to_string(n) + "] tensor on " + dev.str());
}

// What both directions share, into the descriptor.
template <typename Desc>
void block_common(Desc& d, const Tensor& a, const Tensor& r, const OptTensor& g, const Tensor& w1,
                  const Tensor& w2, const OptTensor& alpha) {
  d.lda = rows(a, "a", kBf16, nullptr);
  d.N = a.size(-1);
  d.M = d.N ? a.numel() / d.N : 0;
  d.ldr = rows(r, "r", kBf16 | kFp32, &a);
  if (g) d.ldg = rows(*g, "g", kBf16, &a);
  vec(w1, d.N, kBf16 | kFp32, "w1", a.device());
  vec(w2, d.N, type_of(w1), "w2", a.device());
  if (alpha) vec(*alpha, 1, kFp32, "alpha", a.device());
  d.a = ptr(a);
  d.r = ptr(r);
  d.g = ptr(g);
  d.w1 = ptr(w1);
  d.w2 = ptr(w2);
  d.w_fp32 = type_of(w1) == kFp32;
  d.res_fp32 = type_of(r) == kFp32;
  d.alpha = static_cast<const float*>(ptr(alpha));
}

// Tells autograd that a call has written tensors of the caller's: one that a graph has saved before
// must not go into its backward as if it were the old one.  (An inference tensor is in no graph.)
void wrote(int status, std::initializer_list<const OptTensor*> given) {
  if (status != GNORM_OK) return;
  for (const OptTensor* t : given)
    if (*t && !(*t)->is_inference()) (*t)->unsafeGetTensorImpl()->bump_version();
}

Tensor out_like(const OptTensor& t, const Tensor& like, at::ScalarType type) {
  return t ? *t : at::empty(like.sizes(), like.options().dtype(type));
}

std::tuple<int, Tensor, Tensor, Tensor, Tensor> block_fwd(
    const Tensor& a, const Tensor& r, const Tensor& w1, const Tensor& w2, double eps1, double eps2,
    const OptTensor& g, const OptTensor& alpha, const OptTensor& h_, const OptTensor& z_,
    const OptTensor& rstd1_, const OptTensor& rstd2_, std::optional<uintptr_t> stream) {
  gnorm_block_fwd_desc d = {};
  block_common(d, a, r, g, w1, w2, alpha);
  const Here here(a.device(), stream);
  const Tensor h = out_like(h_, a, r.scalar_type()), z = out_like(z_, a, at::kBFloat16);
  d.ldh = rows(h, "h", type_of(r), &a);
  d.ldz = rows(z, "z", kBf16, &a);
  const auto f32 = a.options().dtype(at::kFloat);
  const Tensor rstd1 = rstd1_ ? *rstd1_ : at::empty({d.M}, f32);
  const Tensor rstd2 = rstd2_ ? *rstd2_ : at::empty({d.M}, f32);
  vec(rstd1, d.M, kFp32, "rstd1", a.device());
  vec(rstd2, d.M, kFp32, "rstd2", a.device());
  d.eps1 = static_cast<float>(eps1);
  d.eps2 = static_cast<float>(eps2);
  d.h = ptr(h);
  d.z = ptr(z);
  d.rstd1 = static_cast<float*>(ptr(rstd1));
  d.rstd2 = static_cast<float*>(ptr(rstd2));
  const int st = gnorm_block_fwd(&d, here.stream);
  wrote(st, {&h_, &z_, &rstd1_, &rstd2_});
  return {st, h, z, rstd1, rstd2};
}

std::tuple<int, Tensor, Tensor, OptTensor, Tensor, Tensor, OptTensor> block_bwd(
    const OptTensor& dh, const Tensor& dz, const Tensor& a, const Tensor& r, const Tensor& w1,
    const Tensor& w2, const Tensor& rstd1, const Tensor& rstd2, const OptTensor& g,
    const OptTensor& alpha, const OptTensor& da_, const OptTensor& dr_, const OptTensor& dg_,
    const OptTensor& dw1_, const OptTensor& dw2_, const OptTensor& dalpha_, bool dw_fp32,
    const OptTensor& workspace, std::optional<uintptr_t> stream) {
  gnorm_block_bwd_desc d = {};
  block_common(d, a, r, g, w1, w2, alpha);
  const at::Device dev = a.device();
  if (dh) d.lddh = rows(*dh, "dh", type_of(r), &a);
  d.lddz = rows(dz, "dz", kBf16, &a);
  vec(rstd1, d.M, kFp32, "rstd1", dev);
  vec(rstd2, d.M, kFp32, "rstd2", dev);
  if (dg_ && !g) bad_value("dg without a gate");
  if (dalpha_ && !alpha) bad_value("dalpha without an alpha");
  const Here here(dev, stream);
  const Tensor da = out_like(da_, a, at::kBFloat16), dr = out_like(dr_, a, r.scalar_type());
  d.ldda = rows(da, "da", kBf16, &a);
  d.lddr = rows(dr, "dr", type_of(r), &a);
  OptTensor dg, dalpha;
  if (g) {
    dg = out_like(dg_, a, at::kBFloat16);
    d.lddg = rows(*dg, "dg", kBf16, &a);
  }
  const auto wt = a.options().dtype(dw_fp32 ? at::kFloat : at::kBFloat16);
  const Tensor dw1 = dw1_ ? *dw1_ : at::empty({d.N}, wt), dw2 = dw2_ ? *dw2_ : at::empty({d.N}, wt);
  vec(dw1, d.N, dw_fp32 ? kFp32 : kBf16, "dw1", dev);
  vec(dw2, d.N, dw_fp32 ? kFp32 : kBf16, "dw2", dev);
  if (alpha) {
    dalpha = dalpha_ ? *dalpha_ : at::empty(alpha->sizes(), alpha->options());
    vec(*dalpha, 1, kFp32, "dalpha", dev);
  }
  const Tensor ws = scratch(workspace, workspace ? 0 : gnorm_block_bwd_workspace_bytes(d.M, d.N), dev);
  d.dh = ptr(dh);
  d.dz = ptr(dz);
  d.rstd1 = static_cast<const float*>(ptr(rstd1));
  d.rstd2 = static_cast<const float*>(ptr(rstd2));
  d.da = ptr(da);
  d.dr = ptr(dr);
  d.dg = ptr(dg);
  d.dw1 = ptr(dw1);
  d.dw2 = ptr(dw2);
  d.dw_fp32 = dw_fp32;
  d.dalpha = static_cast<float*>(ptr(dalpha));
  d.workspace = ptr(ws);
  d.workspace_bytes = ws.nbytes();
  const int st = gnorm_block_bwd(&d, here.stream);
  wrote(st, {&da_, &dr_, &dg_, &dw1_, &dw2_, &dalpha_});
  return {st, da, dr, dg, dw1, dw2, dalpha};
}

// ------------------------------------------------------------------------- delta rule

// Token stride of a [*lead, *tail] tensor ([T, ...] or [B, L, ...]) whose heads are packed
// within a token (tokens may be any distance apart, e.g. a slice of a wider projection).
int64_t tokens(const Tensor& t, const char* name, at::IntArrayRef lead, at::IntArrayRef tail, int types,
               const at::Device& dev) {
  check_type(t, name, types);
  const int64_t n = static_cast<int64_t>(lead.size()), m = static_cast<int64_t>(tail.size());
  bool same = t.dim() == n + m;
  for (int64_t i = 0; same && i < n + m; ++i) same = t.size(i) == (i < n ? lead[i] : tail[i - n]);
  if (!same) {
    std::string want;
    for (int64_t i = 0; i < n + m; ++i)
      want += (i ? ", " : "") + std::to_string(i < n ? lead[i] : tail[i - n]);
    bad_value(std::string(name) + " must be (" + want + "), got " + shape_of(t));
  }
  int64_t ld = 1;  // packed: the values of a token
  for (int64_t x : tail) ld *= x;
  if (!t.is_contiguous() && t.numel() != 0) {
    int64_t want = 1;
    for (int64_t i = n + m - 1; i >= n; --i) {
      if (t.size(i) > 1 && t.stride(i) != want)
        bad_value(std::string(name) + ": the heads of a token must be packed");
      want *= t.size(i);
    }
    const int64_t inner = n == 2 && lead[1] > 1 ? 1 : 0;  // the dimension of neighbouring tokens
    if (lead[inner] > 1) ld = distance(t.stride(inner), name, "tokens");
    if (n == 2 && lead[0] > 1 && t.stride(0) != ld * lead[1])
      bad_value(std::string(name) + ": tokens must be evenly spaced over the batch");
  }
  if (!t.is_cuda()) bad_value(std::string(name) + " must be a CUDA tensor");
  if (t.device() != dev)
    bad_value(std::string(name) + " is on " + t.device().str() + ", the other tensors on " + dev.str());
  return ld;
}

void state_check(const OptTensor& t, const char* name, at::IntArrayRef shape, const at::Device& dev) {
  if (!t) return;
  check_type(*t, name, kFp32);
  if (t->device() != dev || !t->is_contiguous() || t->sizes() != shape) {
    std::string want;
    for (size_t i = 0; i < shape.size(); ++i) want += (i ? ", " : "") + std::to_string(shape[i]);
    bad_value(std::string(name) + " must be a contiguous (" + want + ") tensor on " + dev.str() + ", got " +
              shape_of(*t) + " on " + t->device().str());
  }
}

struct DeltaShape {
  at::IntArrayRef lead, qk, vv, gb;
  int64_t state[4];
  at::IntArrayRef state_shape() const { return {state, 4}; }
};

// What both directions share, into the descriptor.
DeltaShape delta_common(gnorm_delta_in& d, const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& g,
                        const Tensor& beta, std::optional<double> scale, const OptTensor& cu,
                        const OptTensor& initial) {
  if ((q.dim() != 3 && q.dim() != 4) || v.dim() != q.dim())
    bad_value("q, k and v must be [T, heads, dim] or [B, L, heads, dim]");
  DeltaShape s;
  const int64_t n = q.dim() - 2;
  s.lead = q.sizes().slice(0, n);
  s.qk = q.sizes().slice(n, 2);
  s.vv = v.sizes().slice(n, 2);
  s.gb = s.vv.slice(0, 1);
  const at::Device dev = q.device();
  d.ldq = tokens(q, "q", s.lead, s.qk, kBf16, dev);
  d.ldk = tokens(k, "k", s.lead, s.qk, kBf16, dev);
  d.ldv = tokens(v, "v", s.lead, s.vv, kBf16, dev);
  d.ldg = tokens(g, "g", s.lead, s.gb, kFp32, dev);
  d.ldbeta = tokens(beta, "beta", s.lead, s.gb, kBf16 | kFp32, dev);
  d.q = ptr(q);
  d.k = ptr(k);
  d.v = ptr(v);
  d.g = static_cast<const float*>(ptr(g));
  d.beta = ptr(beta);
  d.beta_fp32 = type_of(beta) == kFp32;
  d.Hk = s.qk[0];
  d.K = s.qk[1];
  d.Hv = s.vv[0];
  d.V = s.vv[1];
  d.scale = static_cast<float>(scale ? *scale : 1.0 / std::sqrt(static_cast<double>(d.K)));
  if (cu) {
    if (n != 1) bad_value("cu_seqlens goes with [T, heads, dim] tensors");
    if (cu->scalar_type() != at::kInt) bad_type("cu_seqlens", "int32", *cu);
    if (cu->dim() != 1 || cu->numel() < 1 || !cu->is_contiguous() || cu->device() != dev)
      bad_value("cu_seqlens must be a contiguous [B + 1] tensor on " + dev.str());
    d.cu_seqlens = static_cast<const int*>(cu->data_ptr());
    d.B = cu->numel() - 1;
    d.T = s.lead[0];
  } else {
    d.B = n == 2 ? s.lead[0] : 1;
    d.T = n == 2 ? s.lead[0] * s.lead[1] : s.lead[0];
  }
  s.state[0] = d.B;
  s.state[1] = d.Hv;
  s.state[2] = d.K;
  s.state[3] = d.V;
  state_check(initial, "initial_state", s.state_shape(), dev);
  d.initial_state = static_cast<const float*>(ptr(initial));
  return s;
}

std::tuple<int, Tensor, OptTensor> delta_fwd(
    const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& g, const Tensor& beta,
    std::optional<double> scale, const OptTensor& cu, const OptTensor& initial, bool output_final,
    const OptTensor& o_, const OptTensor& final_, const OptTensor& workspace,
    std::optional<uintptr_t> stream) {
  gnorm_delta_fwd_desc f = {};
  gnorm_delta_in& d = f.in;
  const DeltaShape s = delta_common(d, q, k, v, g, beta, scale, cu, initial);
  const at::Device dev = q.device();
  const Here here(dev, stream);
  const Tensor o = out_like(o_, v, at::kBFloat16);
  f.ldo = tokens(o, "o", s.lead, s.vv, kBf16, dev);
  OptTensor final_state = final_;
  if (!final_state && output_final) final_state = at::empty(s.state_shape(), q.options().dtype(at::kFloat));
  state_check(final_state, "final_state", s.state_shape(), dev);
  const Tensor ws =
      scratch(workspace, workspace ? 0 : gnorm_delta_workspace_bytes(d.T, d.B, d.Hv, d.K, d.V, 0), dev);
  f.o = ptr(o);
  f.final_state = static_cast<float*>(ptr(final_state));
  f.zero_tail = !o_ && cu;
  f.workspace = ptr(ws);
  f.workspace_bytes = ws.nbytes();
  const int st = gnorm_delta_fwd(&f, here.stream);
  wrote(st, {&o_, &final_});
  return {st, o, final_state};
}

std::tuple<int, Tensor, Tensor, Tensor, Tensor, Tensor, OptTensor> delta_bwd(
    const Tensor& d_o, const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& g,
    const Tensor& beta, std::optional<double> scale, const OptTensor& cu, const OptTensor& initial,
    const OptTensor& dfinal, const OptTensor& dq_, const OptTensor& dk_, const OptTensor& dv_,
    const OptTensor& dg_, const OptTensor& dbeta_, const OptTensor& dinitial_, const OptTensor& workspace,
    std::optional<uintptr_t> stream) {
  gnorm_delta_bwd_desc b = {};
  gnorm_delta_in& d = b.in;
  const DeltaShape s = delta_common(d, q, k, v, g, beta, scale, cu, initial);
  const at::Device dev = q.device();
  b.lddo = tokens(d_o, "do", s.lead, s.vv, kBf16, dev);
  state_check(dfinal, "dfinal_state", s.state_shape(), dev);
  const int given = !!dq_ + !!dk_ + !!dv_ + !!dg_ + !!dbeta_;
  if (cu && given != 0 && given != 5)
    bad_value("with cu_seqlens pass all of dq, dk, dv, dg and dbeta, or none");
  const Here here(dev, stream);
  const Tensor dq = out_like(dq_, q, at::kBFloat16), dk = out_like(dk_, k, at::kBFloat16),
               dv = out_like(dv_, v, at::kBFloat16), dg = out_like(dg_, g, at::kFloat),
               dbeta = out_like(dbeta_, beta, beta.scalar_type());
  b.lddq = tokens(dq, "dq", s.lead, s.qk, kBf16, dev);
  b.lddk = tokens(dk, "dk", s.lead, s.qk, kBf16, dev);
  b.lddv = tokens(dv, "dv", s.lead, s.vv, kBf16, dev);
  b.lddg = tokens(dg, "dg", s.lead, s.gb, kFp32, dev);
  b.lddbeta = tokens(dbeta, "dbeta", s.lead, s.gb, type_of(beta), dev);
  OptTensor dinitial = dinitial_;
  if (!dinitial && initial) dinitial = at::empty(s.state_shape(), q.options().dtype(at::kFloat));
  state_check(dinitial, "dinitial_state", s.state_shape(), dev);
  const Tensor ws =
      scratch(workspace, workspace ? 0 : gnorm_delta_workspace_bytes(d.T, d.B, d.Hv, d.K, d.V, 1), dev);
  b.d_o = ptr(d_o);
  b.dfinal_state = static_cast<const float*>(ptr(dfinal));
  b.dq = ptr(dq);
  b.dk = ptr(dk);
  b.dv = ptr(dv);
  b.dg = static_cast<float*>(ptr(dg));
  b.dbeta = ptr(dbeta);
  b.dinitial_state = static_cast<float*>(ptr(dinitial));
  b.zero_tail = cu && given == 0;
  b.workspace = ptr(ws);
  b.workspace_bytes = ws.nbytes();
  const int st = gnorm_delta_bwd(&b, here.stream);
  wrote(st, {&dq_, &dk_, &dv_, &dg_, &dbeta_, &dinitial_});
  return {st, dq, dk, dv, dg, dbeta, dinitial};
}

std::tuple<int, Tensor> delta_step(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& g,
                                   const Tensor& beta, const Tensor& state, const OptTensor& slots,
                                   std::optional<double> scale, const OptTensor& o_,
                                   std::optional<uintptr_t> stream) {
  if (q.dim() != 3 || v.dim() != 3) bad_value("q, k and v must be [B, heads, dim]");
  gnorm_delta_step_desc d = {};
  const at::IntArrayRef lead = q.sizes().slice(0, 1), qk = q.sizes().slice(1, 2), vv = v.sizes().slice(1, 2);
  const at::IntArrayRef gb = vv.slice(0, 1);
  const at::Device dev = q.device();
  d.B = lead[0];
  d.Hk = qk[0];
  d.K = qk[1];
  d.Hv = vv[0];
  d.V = vv[1];
  d.ldq = tokens(q, "q", lead, qk, kBf16, dev);
  d.ldk = tokens(k, "k", lead, qk, kBf16, dev);
  d.ldv = tokens(v, "v", lead, vv, kBf16, dev);
  d.ldg = tokens(g, "g", lead, gb, kFp32, dev);
  d.ldbeta = tokens(beta, "beta", lead, gb, kBf16 | kFp32, dev);
  check_type(state, "state", kFp32);
  bool packed = state.dim() == 4 && state.size(1) == d.Hv && state.size(2) == d.K && state.size(3) == d.V &&
                state.device() == dev;
  int64_t want = 1;
  for (int64_t i = 3; packed && i >= 1; --i) {
    packed = state.size(i) <= 1 || state.stride(i) == want;
    want *= state.size(i);
  }
  if (!packed)
    bad_value("state must be [pool, " + std::to_string(d.Hv) + ", " + std::to_string(d.K) + ", " +
              std::to_string(d.V) + "] on " + dev.str() + " with packed slots, got " + shape_of(state) +
              " on " + state.device().str());
  d.pool = state.size(0);
  d.ldstate = d.pool > 1 ? distance(state.stride(0), "state", "slots") : want;
  if (slots) {
    if (slots->scalar_type() != at::kInt) bad_type("slots", "int32", *slots);
    if (slots->sizes() != lead || !slots->is_contiguous() || slots->device() != dev)
      bad_value("slots must be a contiguous [" + std::to_string(d.B) + "] tensor on " + dev.str());
  }
  const Here here(dev, stream);
  const Tensor o = out_like(o_, v, at::kBFloat16);
  d.ldo = tokens(o, "o", lead, vv, kBf16, dev);
  d.q = ptr(q);
  d.k = ptr(k);
  d.v = ptr(v);
  d.g = static_cast<const float*>(ptr(g));
  d.beta = ptr(beta);
  d.beta_fp32 = type_of(beta) == kFp32;
  d.scale = static_cast<float>(scale ? *scale : 1.0 / std::sqrt(static_cast<double>(d.K)));
  d.state = static_cast<float*>(ptr(state));
  d.slots = static_cast<const int*>(ptr(slots));
  d.o = ptr(o);
  const int st = gnorm_delta_step(&d, here.stream);
  const OptTensor pool = state;
  wrote(st, {&pool, &o_});
  return {st, o};
}

}  // namespace

PYBIND11_MODULE(_marshal, m) {
  m.doc() = "Argument checks and descriptors of the block norm and the gated delta rule.";
  const py::call_guard<py::gil_scoped_release> free;
  m.def("block_fwd", &block_fwd, free);
  m.def("block_bwd", &block_bwd, free);
  m.def("delta_fwd", &delta_fwd, free);
  m.def("delta_bwd", &delta_bwd, free);
  m.def("delta_step", &delta_step, free);
}
