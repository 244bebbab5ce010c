// delta.cu -- launchers and extern "C" entry points of the gated delta rule.
#include "delta_cols.cuh"
#include "delta_grad.cuh"
#include "delta_head.cuh"
#include "delta_prep.cuh"
#include "delta_scan.cuh"
#include "delta_step.cuh"

#include <cmath>

#include "checks.h"
#include "launch.h"

namespace gnorm {
namespace {

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 1;  // cu_seqlens are 32-bit

template <typename Kernel, typename... Args>
cudaError_t launch_grid(Kernel kernel, dim3 grid, int block, int smem, cudaStream_t stream,
                        const Args&... args) {
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = use_pdl() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// cuTensorMapEncodeTiled, fetched from the driver through the runtime (no libcuda link).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver call below needs a context, and a thread that has made no runtime call yet (an
// autograd worker) has none: setting the current device binds its primary context.
bool bind_context() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess;
}

// Boxes of 64 tokens and `box` columns of a [T, cols] tensor with row stride ld; 64 columns are
// swizzled (tile_off).  Without tokens there is nothing to map and nothing is copied.
bool token_map(CUtensorMap* map, const void* base, int64_t T, int64_t cols, int64_t ld, int box) {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  if (T == 0) return true;
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t boxes[2] = {static_cast<cuuint32_t>(box), kChunk};
  const cuuint32_t steps[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, boxes,
            steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
            box == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KD>
cudaError_t launch_prep(const DeltaArgs& a, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(delta_slots(a.seq.T, a.seq.B)), static_cast<unsigned>(a.Hk));
  return launch_grid(delta_prep_kernel<KD>, grid, kPrepThreads, prep_smem<KD>(), s, a);
}

// Strips of 16 columns a CTA.  One while they all fit on the SMs side by side, so that every
// strip has an SM's four schedulers to itself; otherwise two, which share the right operands
// (where the forward has no better way: run_fwd).
int scan_groups(const DeltaArgs& a, int num_sms) {
  return static_cast<long long>(a.V / 16) * a.Hv * a.seq.B <= num_sms ? 1 : 2;
}

template <int KD, int G, bool kOut, bool kSave>
cudaError_t launch_scan_fwd(const DeltaArgs& a, const DeltaMaps& m, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.V / (16 * G)), static_cast<unsigned>(a.Hv),
                  static_cast<unsigned>(a.seq.B));
  return launch_grid(delta_scan_fwd_kernel<KD, G, kOut, kSave>, grid, G * kStripThreads,
                     scan_smem<KD, G, false>(), s, a, m);
}

template <int KD>
cudaError_t launch_scan_bwd(const DeltaArgs& a, const DeltaMaps& m, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.V / 16), static_cast<unsigned>(a.Hv),
                  static_cast<unsigned>(a.seq.B));
  return launch_grid(delta_scan_bwd_kernel<KD>, grid, kStripThreads, scan_smem<KD, 1, true>(), s, a,
                     m);
}

template <int KD, int VD>
cudaError_t launch_grad(const DeltaArgs& a, const DeltaMaps& m, int num_sms, cudaStream_t s) {
  const long long units = a.slots * a.Hk;
  const dim3 grid(static_cast<unsigned>(units < num_sms ? units : num_sms));
  return launch_grid(delta_grad_kernel<KD, VD>, grid, kGradThreads, GradSmem<KD, VD>::kBytes, s, a, m);
}

// A whole head per CTA instead of strips or columns?  An SM takes about 4.1 us a chunk for a
// whole head, 2.6 for a quarter (delta_cols.cuh).  Sequences of one length (the host knows): once
// quarters do not fit the SMs side by side (one of 4096 tokens: 40 heads 310 us against
// 395, 64 heads 336 against 416; 32 heads, before the last steps, 354 against 212; 8 x 1024
// tokens x 16 heads 114 against 222).
// Packed sequences, of which the longest decides and is often twice the mean: with more heads
// than SMs (5 of 4096 tokens in all x 32 heads 150 against 237; 5 of 2048 x 16, of nearly equal
// lengths, 71 against 75; 8 of 8192 x 16, less even, 274 against 252).  Heads of
// 64 columns waste half of an instruction's rows (8 of 8192 x 32, K = V = 64: 275 against 246).
bool whole_heads(const DeltaArgs& a, int num_sms) {
  const long long heads = static_cast<long long>(a.seq.B) * a.Hv;
  if (a.V != 128) return false;
  return a.seq.cu != nullptr && a.seq.B > 1 ? heads > num_sms : 4 * heads > num_sms;
}

template <int KD>
cudaError_t launch_head_fwd(const DeltaArgs& a, const DeltaMaps& m, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.Hv), static_cast<unsigned>(a.seq.B));
  return launch_grid(delta_head_fwd_kernel<KD, 128>, grid, kHeadThreads, head_smem<KD, 128>(), s, a, m);
}

cudaError_t launch_cols_fwd(const DeltaArgs& a, const DeltaMaps& m, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.V / ColsSmem::VT), static_cast<unsigned>(a.Hv),
                  static_cast<unsigned>(a.seq.B));
  return launch_grid(delta_cols_fwd_kernel, grid, ColsSmem::kThreads, ColsSmem::kBytes, s, a, m);
}

// The kernels behind prep read the call's inputs, and cu_seqlens, before they wait for the kernel
// before.  That is sound because prep, the first of the call, waits for everything older before it
// lets the next kernel start, and because no kernel of a call writes an input of the call (the
// entry points refuse outputs that overlap one).  A kernel put before prep, or a prep that does not
// run, would have to do the same.
template <int KD>
cudaError_t run_fwd(const DeltaArgs& a, const DeltaMaps& m, bool whole, int groups, cudaStream_t s) {
  const cudaError_t e = launch_prep<KD>(a, s);
  if (e != cudaSuccess) return e;
  if (whole) return launch_head_fwd<KD>(a, m, s);
  if (groups == 1) return launch_scan_fwd<KD, 1, true, false>(a, m, s);
  // two strips of K = 64 on an SM beat their columns on tcgen05 (4096 tokens x 32 heads of K = 64,
  // V = 128: 186 us against 202), of K = 128 they do not (235 against 210)
  if constexpr (KD == 128)
    return launch_cols_fwd(a, m, s);
  else
    return launch_scan_fwd<KD, 2, true, false>(a, m, s);
}

template <int KD>
cudaError_t run_bwd(const DeltaArgs& a, const DeltaMaps& m, int groups, int num_sms, cudaStream_t s) {
  cudaError_t e = launch_prep<KD>(a, s);
  if (e != cudaSuccess) return e;
  e = groups == 1 ? launch_scan_fwd<KD, 1, false, true>(a, m, s)
                  : launch_scan_fwd<KD, 2, false, true>(a, m, s);
  if (e == cudaSuccess) e = launch_scan_bwd<KD>(a, m, s);
  if (e == cudaSuccess)
    e = a.V == 64 ? launch_grad<KD, 64>(a, m, num_sms, s) : launch_grad<KD, 128>(a, m, num_sms, s);
  return e;
}

size_t round_up(size_t v) { return (v + GNORM_WORKSPACE_ALIGN - 1) / GNORM_WORKSPACE_ALIGN * GNORM_WORKSPACE_ALIGN; }

struct DeltaLayout {
  size_t prep = 0, s = 0, d = 0, w = 0, x = 0, dots = 0, total = 0;
};

DeltaLayout delta_layout(int64_t T, int64_t B, int64_t Hv, int64_t K, int64_t V, bool backward) {
  const size_t n = static_cast<size_t>(delta_slots(T, B)) * static_cast<size_t>(Hv);
  DeltaLayout l;
  size_t at = 0;
  auto take = [&](size_t each) {
    const size_t p = at;
    at = round_up(at + n * each);
    return p;
  };
  l.prep = take(kPrepBytes);
  if (backward) {
    l.s = take(static_cast<size_t>(K * V) * 4);
    l.d = take(static_cast<size_t>(K * V) * 4);
    l.w = take(static_cast<size_t>(3 * V / 64) * kTileBytes);
    l.x = take(static_cast<size_t>(2 * V / 64) * kTileBytes);
    l.dots = take(static_cast<size_t>(V / 16) * 128 * 4);
  }
  l.total = at;
  return l;
}

int check_heads(int64_t Hk, int64_t Hv, int64_t K, int64_t V) {
  if (Hk < 1 || Hv < Hk || Hv > 65535 || Hv % Hk != 0) return GNORM_ERR_SHAPE;
  if ((K != 64 && K != 128) || (V != 64 && V != 128)) return GNORM_ERR_SHAPE;
  return GNORM_OK;
}

// Row stride of a [T, heads, D] tensor: 0 means packed.
int check_token_ld(int64_t* ld, int64_t cols, int64_t align) {
  if (*ld == 0) *ld = cols;
  if (*ld < cols) return GNORM_ERR_SHAPE;
  return *ld % align != 0 ? GNORM_ERR_ALIGN : GNORM_OK;
}

// Validates the shared inputs in place and fills the kernels' argument block.
int check_delta(gnorm_delta_in* d, DeltaArgs* a) {
  int st = check_heads(d->Hk, d->Hv, d->K, d->V);
  if (st != GNORM_OK) return st;
  if (d->T < 0 || d->T > kMaxTokens || d->B < 0 || d->B > 65535) return GNORM_ERR_SHAPE;
  if (d->B == 0 && d->T != 0) return GNORM_ERR_SHAPE;
  if (d->cu_seqlens == nullptr && d->B > 0 && d->T % d->B != 0) return GNORM_ERR_SHAPE;
  if (!std::isfinite(d->scale)) return GNORM_ERR_ARG;
  const int64_t kc = d->Hk * d->K, vc = d->Hv * d->V;
  if ((st = check_token_ld(&d->ldq, kc, 8)) != GNORM_OK) return st;
  if ((st = check_token_ld(&d->ldk, kc, 8)) != GNORM_OK) return st;
  if ((st = check_token_ld(&d->ldv, vc, 8)) != GNORM_OK) return st;
  if ((st = check_token_ld(&d->ldg, d->Hv, 1)) != GNORM_OK) return st;
  if ((st = check_token_ld(&d->ldbeta, d->Hv, 1)) != GNORM_OK) return st;
  if (d->T > 0 && (!d->q || !d->k || !d->v || !d->g || !d->beta)) return GNORM_ERR_NULL;
  if (!aligned(d->q, 16) || !aligned(d->k, 16) || !aligned(d->v, 16) || !aligned(d->g, 4) ||
      !aligned(d->beta, d->beta_fp32 ? 4 : 2) || !aligned(d->cu_seqlens, 4) ||
      !aligned(d->initial_state, 16))
    return GNORM_ERR_ALIGN;
  a->seq.cu = d->cu_seqlens;
  a->seq.B = static_cast<int>(d->B);
  a->seq.T = d->T;
  a->seq.seqlen = d->B > 0 ? d->T / d->B : 0;
  a->q = static_cast<const uint16_t*>(d->q);
  a->k = static_cast<const uint16_t*>(d->k);
  a->v = static_cast<const uint16_t*>(d->v);
  a->g = d->g;
  a->beta = d->beta;
  a->beta_fp32 = d->beta_fp32 ? 1 : 0;
  a->ldq = d->ldq;
  a->ldk = d->ldk;
  a->ldv = d->ldv;
  a->ldg = d->ldg;
  a->ldbeta = d->ldbeta;
  a->Hk = static_cast<int>(d->Hk);
  a->Hv = static_cast<int>(d->Hv);
  a->V = static_cast<int>(d->V);
  a->scale = d->scale;
  a->state_in = d->initial_state;
  return GNORM_OK;
}

size_t state_bytes(const gnorm_delta_in& d) {
  return static_cast<size_t>(d.B) * d.Hv * d.K * d.V * 4;
}

constexpr int kDeltaInputs = 7;
void delta_regions(const gnorm_delta_in& d, Region* in) {
  in[0] = mat(d.q, d.T, d.Hk * d.K, d.ldq);
  in[1] = mat(d.k, d.T, d.Hk * d.K, d.ldk);
  in[2] = mat(d.v, d.T, d.Hv * d.V, d.ldv);
  in[3] = mat(d.g, d.T, d.Hv, d.ldg, 4);
  in[4] = mat(d.beta, d.T, d.Hv, d.ldbeta, d.beta_fp32 ? 4 : 2);
  in[5] = span(d.cu_seqlens, d.cu_seqlens ? static_cast<size_t>(d.B + 1) * 4 : 0);
  in[6] = span(d.initial_state, state_bytes(d));
}

int check_ws(void* ws, size_t have, size_t need) {
  if (need == 0) return GNORM_OK;
  return ws == nullptr || !aligned(ws, GNORM_WORKSPACE_ALIGN) || have < need ? GNORM_ERR_WORKSPACE
                                                                            : GNORM_OK;
}

void add_zero(DeltaArgs* a, void* p, int64_t ld, int64_t cols, int elem) {
  a->zero_p[a->n_zero] = static_cast<uint8_t*>(p);
  a->zero_ld[a->n_zero] = ld * elem;
  a->zero_row[a->n_zero] = static_cast<int>(cols * elem);
  ++a->n_zero;
}

template <int KD, int VD>
cudaError_t launch_step(const StepArgs& a, int num_sms, cudaStream_t s) {
  // 32 columns a CTA (4 CTAs per 128-column head) while whole heads would not give every SM
  // a CTA; whole heads otherwise, whose rows are read in full 512-byte lines.
  const bool narrow = static_cast<long long>(a.B) * a.Hv < num_sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(narrow ? VD / 32 : 1), static_cast<unsigned>(a.Hv),
                     static_cast<unsigned>(a.B));
  cfg.blockDim = dim3(kStepThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = use_pdl() ? 1 : 0;
  return narrow ? cudaLaunchKernelEx(&cfg, delta_step_kernel<KD, VD, 32>, a)
                : cudaLaunchKernelEx(&cfg, delta_step_kernel<KD, VD, VD>, a);
}

}  // namespace
}  // namespace gnorm

using namespace gnorm;

extern "C" {

int gnorm_delta_fwd(const gnorm_delta_fwd_desc* desc, void* stream) {
  if (desc == nullptr) return GNORM_ERR_NULL;
  gnorm_delta_fwd_desc f = *desc;
  DeltaArgs a;
  int st = check_delta(&f.in, &a);
  if (st != GNORM_OK) return st;
  const gnorm_delta_in& d = f.in;
  if ((st = check_token_ld(&f.ldo, d.Hv * d.V, 8)) != GNORM_OK) return st;
  if (d.B == 0) return GNORM_OK;
  if (d.T > 0 && !f.o) return GNORM_ERR_NULL;
  if (!aligned(f.o, 16) || !aligned(f.final_state, 16)) return GNORM_ERR_ALIGN;
  Region in[kDeltaInputs];
  delta_regions(d, in);
  const Region out[] = {mat(f.o, d.T, d.Hv * d.V, f.ldo), span(f.final_state, state_bytes(d)),
                        span(f.workspace, f.workspace_bytes)};
  if (any_alias(in, kDeltaInputs, out, 3)) return GNORM_ERR_ALIAS;
  const DeltaLayout l = delta_layout(d.T, d.B, d.Hv, d.K, d.V, false);
  if ((st = check_ws(f.workspace, f.workspace_bytes, l.total)) != GNORM_OK) return st;
  a.o = static_cast<uint16_t*>(f.o);
  a.ldo = f.ldo;
  a.state_out = f.final_state;
  a.prep = static_cast<uint8_t*>(f.workspace) + l.prep;
  if (f.zero_tail && f.o) add_zero(&a, f.o, f.ldo, d.Hv * d.V, 2);
  DeviceInfo info;
  if ((st = device_info(&info)) != GNORM_OK) return st;
  a.err = info.err_word;
  a.sms = info.num_sms;
  const cudaStream_t s = as_stream(stream);
  const bool whole = whole_heads(a, info.num_sms);
  const int groups = scan_groups(a, info.num_sms);
  DeltaMaps m{};
  if (!bind_context() || !token_map(&m.q, d.q, d.T, d.Hk * d.K, d.ldq, 64) ||
      !token_map(&m.k, d.k, d.T, d.Hk * d.K, d.ldk, 64) ||
      !token_map(&m.v, d.v, d.T, d.Hv * d.V, d.ldv, whole ? 64 : 16 * groups))
    return GNORM_ERR_CUDA;
  const cudaError_t e =
      d.K == 64 ? run_fwd<64>(a, m, whole, groups, s) : run_fwd<128>(a, m, whole, groups, s);
  return e == cudaSuccess ? GNORM_OK : GNORM_ERR_CUDA;
}

int gnorm_delta_bwd(const gnorm_delta_bwd_desc* desc, void* stream) {
  if (desc == nullptr) return GNORM_ERR_NULL;
  gnorm_delta_bwd_desc f = *desc;
  DeltaArgs a;
  int st = check_delta(&f.in, &a);
  if (st != GNORM_OK) return st;
  const gnorm_delta_in& d = f.in;
  const int64_t kc = d.Hk * d.K, vc = d.Hv * d.V;
  if ((st = check_token_ld(&f.lddo, vc, 8)) != GNORM_OK) return st;
  if ((st = check_token_ld(&f.lddq, kc, 8)) != GNORM_OK) return st;
  if ((st = check_token_ld(&f.lddk, kc, 8)) != GNORM_OK) return st;
  if ((st = check_token_ld(&f.lddv, vc, 8)) != GNORM_OK) return st;
  if ((st = check_token_ld(&f.lddg, d.Hv, 1)) != GNORM_OK) return st;
  if ((st = check_token_ld(&f.lddbeta, d.Hv, 1)) != GNORM_OK) return st;
  if (d.B == 0) return GNORM_OK;
  if (d.T > 0 && (!f.d_o || !f.dq || !f.dk || !f.dv || !f.dg || !f.dbeta)) return GNORM_ERR_NULL;
  if (!aligned(f.d_o, 16) || !aligned(f.dq, 16) || !aligned(f.dk, 16) || !aligned(f.dv, 16) ||
      !aligned(f.dg, 4) || !aligned(f.dbeta, d.beta_fp32 ? 4 : 2) ||
      !aligned(f.dfinal_state, 16) || !aligned(f.dinitial_state, 16))
    return GNORM_ERR_ALIGN;
  Region in[kDeltaInputs + 2];
  delta_regions(d, in);
  in[kDeltaInputs] = mat(f.d_o, d.T, vc, f.lddo);
  in[kDeltaInputs + 1] = span(f.dfinal_state, state_bytes(d));
  const Region out[] = {mat(f.dq, d.T, kc, f.lddq),
                        mat(f.dk, d.T, kc, f.lddk),
                        mat(f.dv, d.T, vc, f.lddv),
                        mat(f.dg, d.T, d.Hv, f.lddg, 4),
                        mat(f.dbeta, d.T, d.Hv, f.lddbeta, d.beta_fp32 ? 4 : 2),
                        span(f.dinitial_state, state_bytes(d)),
                        span(f.workspace, f.workspace_bytes)};
  if (any_alias(in, kDeltaInputs + 2, out, 7)) return GNORM_ERR_ALIAS;
  const DeltaLayout l = delta_layout(d.T, d.B, d.Hv, d.K, d.V, true);
  if ((st = check_ws(f.workspace, f.workspace_bytes, l.total)) != GNORM_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(f.workspace);
  a.prep = ws + l.prep;
  a.s_ws = ws + l.s;
  a.d_ws = ws + l.d;
  a.w_ws = ws + l.w;
  a.x_ws = ws + l.x;
  a.dots = reinterpret_cast<float*>(ws + l.dots);
  a.dout = static_cast<const uint16_t*>(f.d_o);
  a.lddo = f.lddo;
  a.dstate_out = f.dfinal_state;
  a.dstate_in = f.dinitial_state;
  a.dq = static_cast<uint16_t*>(f.dq);
  a.dk = static_cast<uint16_t*>(f.dk);
  a.dv = static_cast<uint16_t*>(f.dv);
  a.dg = f.dg;
  a.dbeta = f.dbeta;
  a.lddq = f.lddq;
  a.lddk = f.lddk;
  a.lddv = f.lddv;
  a.lddg = f.lddg;
  a.lddbeta = f.lddbeta;
  if (f.zero_tail && d.T > 0) {
    add_zero(&a, f.dq, f.lddq, kc, 2);
    add_zero(&a, f.dk, f.lddk, kc, 2);
    add_zero(&a, f.dv, f.lddv, vc, 2);
    add_zero(&a, f.dg, f.lddg, d.Hv, 4);
    add_zero(&a, f.dbeta, f.lddbeta, d.Hv, d.beta_fp32 ? 4 : 2);
  }
  DeviceInfo info;
  if ((st = device_info(&info)) != GNORM_OK) return st;
  a.err = info.err_word;
  a.sms = info.num_sms;
  a.slots = delta_slots(d.T, d.B);
  const cudaStream_t s = as_stream(stream);
  const int groups = scan_groups(a, info.num_sms);
  DeltaMaps m{};
  if (!bind_context() || !token_map(&m.q, d.q, d.T, kc, d.ldq, 64) ||
      !token_map(&m.k, d.k, d.T, kc, d.ldk, 64) ||
      !token_map(&m.v, d.v, d.T, vc, d.ldv, 16 * groups) ||
      !token_map(&m.do_strip, f.d_o, d.T, vc, f.lddo, 16) ||
      !token_map(&m.do_tile, f.d_o, d.T, vc, f.lddo, 64) ||
      !token_map(&m.dv, f.dv, d.T, vc, f.lddv, 64))
    return GNORM_ERR_CUDA;
  const cudaError_t e = d.K == 64 ? run_bwd<64>(a, m, groups, info.num_sms, s)
                                  : run_bwd<128>(a, m, groups, info.num_sms, s);
  return e == cudaSuccess ? GNORM_OK : GNORM_ERR_CUDA;
}

size_t gnorm_delta_workspace_bytes(int64_t T, int64_t B, int64_t Hv, int64_t K, int64_t V,
                                   int backward) {
  if (T < 0 || T > kMaxTokens || B < 0 || B > 65535 || check_heads(1, Hv, K, V) != GNORM_OK)
    return 0;
  return delta_layout(T, B, Hv, K, V, backward != 0).total;
}

int gnorm_delta_step(const gnorm_delta_step_desc* desc, void* stream) {
  if (desc == nullptr) return GNORM_ERR_NULL;
  gnorm_delta_step_desc f = *desc;
  int st = check_heads(f.Hk, f.Hv, f.K, f.V);
  if (st != GNORM_OK) return st;
  if (f.B < 0 || f.B > 65535 || f.pool < 0 || f.pool > kMaxTokens) return GNORM_ERR_SHAPE;
  if (f.slots == nullptr && f.pool < f.B) return GNORM_ERR_SHAPE;
  if (!std::isfinite(f.scale)) return GNORM_ERR_ARG;
  const int64_t kc = f.Hk * f.K, vc = f.Hv * f.V;
  if ((st = check_token_ld(&f.ldq, kc, 1)) != GNORM_OK) return st;
  if ((st = check_token_ld(&f.ldk, kc, 1)) != GNORM_OK) return st;
  if ((st = check_token_ld(&f.ldv, vc, 4)) != GNORM_OK) return st;
  if ((st = check_token_ld(&f.ldg, f.Hv, 1)) != GNORM_OK) return st;
  if ((st = check_token_ld(&f.ldbeta, f.Hv, 1)) != GNORM_OK) return st;
  if ((st = check_token_ld(&f.ldo, vc, 4)) != GNORM_OK) return st;
  if ((st = check_token_ld(&f.ldstate, vc * f.K, 4)) != GNORM_OK) return st;
  if (f.B == 0) return GNORM_OK;
  if (!f.q || !f.k || !f.v || !f.g || !f.beta || !f.o || (!f.state && f.pool > 0))
    return GNORM_ERR_NULL;
  if (!aligned(f.q, 2) || !aligned(f.k, 2) || !aligned(f.v, 8) || !aligned(f.o, 8) ||
      !aligned(f.g, 4) || !aligned(f.beta, f.beta_fp32 ? 4 : 2) || !aligned(f.state, 16) ||
      !aligned(f.slots, 4))
    return GNORM_ERR_ALIGN;
  const Region in[] = {mat(f.q, f.B, kc, f.ldq),
                       mat(f.k, f.B, kc, f.ldk),
                       mat(f.v, f.B, vc, f.ldv),
                       mat(f.g, f.B, f.Hv, f.ldg, 4),
                       mat(f.beta, f.B, f.Hv, f.ldbeta, f.beta_fp32 ? 4 : 2),
                       span(f.slots, f.slots ? static_cast<size_t>(f.B) * 4 : 0)};
  const Region out[] = {mat(f.o, f.B, vc, f.ldo), mat(f.state, f.pool, vc * f.K, f.ldstate, 4)};
  if (any_alias(in, 6, out, 2)) return GNORM_ERR_ALIAS;
  DeviceInfo info;
  if ((st = device_info(&info)) != GNORM_OK) return st;
  StepArgs a;
  a.q = static_cast<const uint16_t*>(f.q);
  a.k = static_cast<const uint16_t*>(f.k);
  a.v = static_cast<const uint16_t*>(f.v);
  a.g = f.g;
  a.beta = f.beta;
  a.beta_fp32 = f.beta_fp32 ? 1 : 0;
  a.ldq = f.ldq;
  a.ldk = f.ldk;
  a.ldv = f.ldv;
  a.ldg = f.ldg;
  a.ldbeta = f.ldbeta;
  a.ldo = f.ldo;
  a.Hk = static_cast<int>(f.Hk);
  a.Hv = static_cast<int>(f.Hv);
  a.B = static_cast<int>(f.B);
  a.scale = f.scale;
  a.slots = f.slots;
  a.pool = static_cast<int>(f.pool);
  a.state = f.state;
  a.lds = f.ldstate;
  a.o = static_cast<uint16_t*>(f.o);
  const cudaStream_t s = as_stream(stream);
  cudaError_t e;
  if (f.K == 64)
    e = f.V == 64 ? launch_step<64, 64>(a, info.num_sms, s) : launch_step<64, 128>(a, info.num_sms, s);
  else
    e = f.V == 64 ? launch_step<128, 64>(a, info.num_sms, s) : launch_step<128, 128>(a, info.num_sms, s);
  return e == cudaSuccess ? GNORM_OK : GNORM_ERR_CUDA;
}

}  // extern "C"
