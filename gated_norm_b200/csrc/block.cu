// block.cu -- launch plan, launchers and extern "C" entry points of the block norm
// (block_kernel.cuh).
#include "block_kernel.cuh"

#include <algorithm>
#include <cmath>

#include "checks.h"
#include "launch.h"

namespace gnorm {
namespace {

struct BlockPlan {
  int tpr = 0, cpt = 0, threads = 0, ctas_per_sm = 0;
  int rows_per_stage = 0, stages = 0, grid = 0, smem = 0;
  int64_t num_blocks = 0;
  uint32_t stage_bytes = 0;
};

// Rows of up to 256 values are one chunk per thread inside a warp; up to 4096 two chunks per
// thread; wider rows take one row group of 512 threads.
RowGeometry block_geometry(int64_t N) {
  const int64_t n8 = N / 8;
  if (n8 <= 8) return {8, 1};
  if (n8 <= 16) return {16, 1};
  if (n8 <= 32) return {32, 1};
  if (n8 <= 64) return {32, 2};
  if (n8 <= 128) return {64, 2};
  if (n8 <= 256) return {128, 2};
  if (n8 <= 512) return {256, 2};
  if (n8 <= 1024) return {512, 2};
  return {512, 4};
}

constexpr int64_t kBlockStageBytes[2] = {32768, 49152};

int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// kind 0 forward, 1 backward.  Fills the input offsets of `args` (row_bytes set by the caller).
int block_plan(int kind, int64_t M, int64_t N, const DeviceInfo& d, BlockArgs* args,
               BlockPlan* out) {
  const RowGeometry geo = block_geometry(N);
  BlockPlan p;
  p.tpr = geo.threads_per_row;
  p.cpt = geo.chunks_per_thread;
  p.threads = block_threads(p.tpr);
  p.ctas_per_sm = block_ctas_per_sm(kind, p.tpr, p.cpt);
  const int groups = p.threads / p.tpr;
  int64_t row_bytes = kind == 1 ? 8 : 0;
  for (const BlockIn& t : args->in) row_bytes += t.row_bytes;
  auto stage_size = [&](int64_t R, bool fill) {
    int64_t off = 0;
    for (BlockIn& t : args->in) {
      if (fill) t.off = static_cast<uint32_t>(off);
      off += up(R * t.row_bytes, 128);
    }
    if (fill) args->rstd_off = static_cast<uint32_t>(off);
    return off + (kind == 1 ? up(R * 8, 128) : 0);
  };
  int64_t smem_cta = d.smem_optin;
  if (p.ctas_per_sm > 1)
    smem_cta = std::min<int64_t>(smem_cta, kB200SmemPerSm / p.ctas_per_sm - kSmemPerCtaReserve);
  const int64_t budget = smem_cta - kHeaderBytes;
  int64_t target = std::max<int64_t>(groups, kBlockStageBytes[kind] / row_bytes);
  while (target > 1 && 2 * stage_size(target, false) > budget) --target;
  const int64_t grid_max = static_cast<int64_t>(d.num_sms) * p.ctas_per_sm;
  const int64_t per_cta = (M + grid_max - 1) / grid_max;
  // equal shares: k blocks per CTA of about `target` rows
  const int64_t k = (per_cta + target - 1) / target;
  const int64_t R = (per_cta + k - 1) / k;
  const int64_t stage = stage_size(R, true);
  // One stage is enough to run (rows of 16384 FP32 residuals leave room for no more).
  const int64_t stages = std::min<int64_t>(kMaxStages, budget / stage);
  if (stages < 1) return GNORM_ERR_UNSUPPORTED;
  int64_t body = stages * stage;
  if (kind == 1 && groups > 1) body = std::max<int64_t>(body, static_cast<int64_t>(groups) * N * 4);
  if (kHeaderBytes + body > smem_cta) return GNORM_ERR_UNSUPPORTED;
  p.rows_per_stage = static_cast<int>(R);
  p.stages = static_cast<int>(stages);
  p.stage_bytes = static_cast<uint32_t>(stage);
  p.num_blocks = (M + R - 1) / R;
  p.grid = static_cast<int>(std::min<int64_t>(p.num_blocks, grid_max));
  p.smem = static_cast<int>(kHeaderBytes + body);
  *out = p;
  return GNORM_OK;
}

template <int TPR, int CPT, bool kGate, bool kRes32>
cudaError_t launch_block_variant(int kind, const BlockPlan& p, const BlockArgs& a, cudaStream_t s,
                                 bool pdl) {
  auto* kernel = kind == 0 ? block_norm_fwd_kernel<TPR, CPT, kGate, kRes32>
                           : block_norm_bwd_kernel<TPR, CPT, kGate, kRes32>;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), p.smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kernel, p.grid, p.threads + 32, p.smem, s, pdl, a);
}

template <int TPR, int CPT>
cudaError_t launch_block_geometry(int kind, const BlockPlan& p, const BlockArgs& a, int res_fp32,
                                  cudaStream_t s, bool pdl) {
  if (a.in[2].p != nullptr)
    return res_fp32 ? launch_block_variant<TPR, CPT, true, true>(kind, p, a, s, pdl)
                    : launch_block_variant<TPR, CPT, true, false>(kind, p, a, s, pdl);
  return res_fp32 ? launch_block_variant<TPR, CPT, false, true>(kind, p, a, s, pdl)
                  : launch_block_variant<TPR, CPT, false, false>(kind, p, a, s, pdl);
}

cudaError_t launch_block(int kind, const BlockPlan& p, BlockArgs& a, int res_fp32, cudaStream_t s) {
  a.rows_per_stage = p.rows_per_stage;
  a.stages = p.stages;
  a.stage_bytes = p.stage_bytes;
  a.num_blocks = p.num_blocks;
  const bool pdl = use_pdl();
  switch (p.tpr * 8 + p.cpt) {
    case 8 * 8 + 1: return launch_block_geometry<8, 1>(kind, p, a, res_fp32, s, pdl);
    case 16 * 8 + 1: return launch_block_geometry<16, 1>(kind, p, a, res_fp32, s, pdl);
    case 32 * 8 + 1: return launch_block_geometry<32, 1>(kind, p, a, res_fp32, s, pdl);
    case 32 * 8 + 2: return launch_block_geometry<32, 2>(kind, p, a, res_fp32, s, pdl);
    case 64 * 8 + 2: return launch_block_geometry<64, 2>(kind, p, a, res_fp32, s, pdl);
    case 128 * 8 + 2: return launch_block_geometry<128, 2>(kind, p, a, res_fp32, s, pdl);
    case 256 * 8 + 2: return launch_block_geometry<256, 2>(kind, p, a, res_fp32, s, pdl);
    case 512 * 8 + 2: return launch_block_geometry<512, 2>(kind, p, a, res_fp32, s, pdl);
    case 512 * 8 + 4: return launch_block_geometry<512, 4>(kind, p, a, res_fp32, s, pdl);
    default: return cudaErrorInvalidConfiguration;
  }
}

constexpr int64_t kBlockMaxRows = int64_t(1) << 40;

int check_block_shape(int64_t M, int64_t N) {
  if (M < 0 || M > kBlockMaxRows) return GNORM_ERR_SHAPE;
  if (N < 8 || N > GNORM_N_MAX || (N % 8) != 0) return GNORM_ERR_SHAPE;
  return GNORM_OK;
}

BlockIn block_in(const void* p, int64_t ld, int64_t N, int elem) {
  BlockIn t;
  if (p == nullptr) return t;
  t.p = static_cast<const uint8_t*>(p);
  t.ld_bytes = ld * elem;
  t.row_bytes = static_cast<uint32_t>(N * elem);
  return t;
}

size_t w_span(int64_t N, int fp32) { return static_cast<size_t>(N) * (fp32 ? 4 : 2); }

// Partial rows a backward of this shape may use on a device (an upper bound over the types).
int64_t block_partials(int64_t M, int64_t N, int num_sms) {
  const RowGeometry geo = block_geometry(N);
  return std::min<int64_t>(
      M, static_cast<int64_t>(num_sms) *
             block_ctas_per_sm(1, geo.threads_per_row, geo.chunks_per_thread));
}

size_t block_workspace(int64_t M, int64_t N, int num_sms) {
  const size_t raw = static_cast<size_t>(block_partials(M, N, num_sms)) * (2 * N + 1) * 4;
  return (raw + GNORM_WORKSPACE_ALIGN - 1) / GNORM_WORKSPACE_ALIGN * GNORM_WORKSPACE_ALIGN +
         GNORM_WORKSPACE_ALIGN;
}

}  // namespace
}  // namespace gnorm

using namespace gnorm;

extern "C" {

int gnorm_block_fwd(const gnorm_block_fwd_desc* desc, void* stream) {
  if (desc == nullptr) return GNORM_ERR_NULL;
  gnorm_block_fwd_desc f = *desc;
  int st = check_block_shape(f.M, f.N);
  if (st != GNORM_OK) return st;
  if (!std::isfinite(f.eps1) || f.eps1 < 0.f || !std::isfinite(f.eps2) || f.eps2 < 0.f)
    return GNORM_ERR_ARG;
  for (int64_t* ld : {&f.lda, &f.ldr, &f.ldg, &f.ldh, &f.ldz})
    if ((st = check_ld(ld, f.N)) != GNORM_OK) return st;
  if (f.M == 0) return GNORM_OK;
  if (!f.a || !f.r || !f.w1 || !f.w2 || !f.h || !f.z || !f.rstd1 || !f.rstd2)
    return GNORM_ERR_NULL;
  for (const void* p : {f.a, f.r, f.g, f.w1, f.w2, static_cast<const void*>(f.h),
                        static_cast<const void*>(f.z)})
    if (!aligned(p, 16)) return GNORM_ERR_ALIGN;
  if (!aligned(f.rstd1, 4) || !aligned(f.rstd2, 4) || !aligned(f.alpha, 4)) return GNORM_ERR_ALIGN;
  const int e = f.res_fp32 ? 4 : 2;
  const size_t rstd_bytes = static_cast<size_t>(f.M) * 4;
  const Region in[] = {mat(f.a, f.M, f.N, f.lda), mat(f.r, f.M, f.N, f.ldr, e),
                       mat(f.g, f.M, f.N, f.ldg), span(f.w1, w_span(f.N, f.w_fp32)),
                       span(f.w2, w_span(f.N, f.w_fp32)), span(f.alpha, 4)};
  const Region out[] = {mat(f.h, f.M, f.N, f.ldh, e), mat(f.z, f.M, f.N, f.ldz),
                        span(f.rstd1, rstd_bytes), span(f.rstd2, rstd_bytes)};
  if (any_alias(in, 6, out, 4)) return GNORM_ERR_ALIAS;
  DeviceInfo d;
  if ((st = device_info(&d)) != GNORM_OK) return st;
  BlockArgs a;
  a.in[0] = block_in(f.a, f.lda, f.N, 2);
  a.in[1] = block_in(f.r, f.ldr, f.N, e);
  a.in[2] = block_in(f.g, f.ldg, f.N, 2);
  a.w1 = f.w1;
  a.w2 = f.w2;
  a.w_fp32 = f.w_fp32 ? 1 : 0;
  a.alpha = f.alpha;
  a.eps1 = f.eps1;
  a.eps2 = f.eps2;
  a.h = static_cast<uint8_t*>(f.h);
  a.z = static_cast<uint16_t*>(f.z);
  a.rstd1 = f.rstd1;
  a.rstd2 = f.rstd2;
  a.ldh = f.ldh;
  a.ldz = f.ldz;
  a.M = f.M;
  a.N = static_cast<int>(f.N);
  a.inv_n = static_cast<float>(1.0 / static_cast<double>(f.N));
  a.err = d.err_word;
  BlockPlan plan;
  if ((st = block_plan(0, f.M, f.N, d, &a, &plan)) != GNORM_OK) return st;
  return launch_block(0, plan, a, f.res_fp32 ? 1 : 0, as_stream(stream)) == cudaSuccess
             ? GNORM_OK
             : GNORM_ERR_CUDA;
}

int gnorm_block_bwd(const gnorm_block_bwd_desc* desc, void* stream) {
  if (desc == nullptr) return GNORM_ERR_NULL;
  gnorm_block_bwd_desc b = *desc;
  int st = check_block_shape(b.M, b.N);
  if (st != GNORM_OK) return st;
  for (int64_t* ld : {&b.lddh, &b.lddz, &b.lda, &b.ldr, &b.ldg, &b.ldda, &b.lddr, &b.lddg})
    if ((st = check_ld(ld, b.N)) != GNORM_OK) return st;
  if (!b.dw1 || !b.dw2) return GNORM_ERR_NULL;
  if (!aligned(b.dw1, 16) || !aligned(b.dw2, 16) || !aligned(b.dalpha, 4)) return GNORM_ERR_ALIGN;
  if (b.dalpha && !b.alpha) return GNORM_ERR_NULL;
  const size_t dw_bytes = w_span(b.N, b.dw_fp32);
  const cudaStream_t s = as_stream(stream);
  if (b.M == 0) {
    const Region out[] = {span(b.dw1, dw_bytes), span(b.dw2, dw_bytes), span(b.dalpha, 4)};
    if (any_alias(out, 0, out, 3)) return GNORM_ERR_ALIAS;
    if (cudaMemsetAsync(b.dw1, 0, dw_bytes, s) != cudaSuccess ||
        cudaMemsetAsync(b.dw2, 0, dw_bytes, s) != cudaSuccess ||
        (b.dalpha && cudaMemsetAsync(b.dalpha, 0, 4, s) != cudaSuccess))
      return GNORM_ERR_CUDA;
    return GNORM_OK;
  }
  if (!b.dz || !b.a || !b.r || !b.w1 || !b.w2 || !b.rstd1 || !b.rstd2 || !b.da || !b.dr)
    return GNORM_ERR_NULL;
  if ((b.g != nullptr) != (b.dg != nullptr)) return GNORM_ERR_NULL;
  for (const void* p : {b.dh, b.dz, b.a, b.r, b.g, b.w1, b.w2, static_cast<const void*>(b.da),
                        static_cast<const void*>(b.dr), static_cast<const void*>(b.dg)})
    if (!aligned(p, 16)) return GNORM_ERR_ALIGN;
  if (!aligned(b.rstd1, 4) || !aligned(b.rstd2, 4) || !aligned(b.alpha, 4)) return GNORM_ERR_ALIGN;
  const int e = b.res_fp32 ? 4 : 2;
  const size_t rstd_bytes = static_cast<size_t>(b.M) * 4;
  const Region in[] = {mat(b.dh, b.M, b.N, b.lddh, e), mat(b.dz, b.M, b.N, b.lddz),
                       mat(b.a, b.M, b.N, b.lda), mat(b.r, b.M, b.N, b.ldr, e),
                       mat(b.g, b.M, b.N, b.ldg), span(b.w1, w_span(b.N, b.w_fp32)),
                       span(b.w2, w_span(b.N, b.w_fp32)), span(b.alpha, 4),
                       span(b.rstd1, rstd_bytes), span(b.rstd2, rstd_bytes)};
  const Region out[] = {mat(b.da, b.M, b.N, b.ldda), mat(b.dr, b.M, b.N, b.lddr, e),
                        mat(b.dg, b.M, b.N, b.lddg), span(b.dw1, dw_bytes),
                        span(b.dw2, dw_bytes), span(b.dalpha, 4),
                        span(b.workspace, b.workspace_bytes)};
  if (any_alias(in, 10, out, 7)) return GNORM_ERR_ALIAS;
  DeviceInfo d;
  if ((st = device_info(&d)) != GNORM_OK) return st;
  BlockArgs a;
  a.in[0] = block_in(b.a, b.lda, b.N, 2);
  a.in[1] = block_in(b.r, b.ldr, b.N, e);
  a.in[2] = block_in(b.g, b.ldg, b.N, 2);
  a.in[3] = block_in(b.dz, b.lddz, b.N, 2);
  a.in[4] = block_in(b.dh, b.lddh, b.N, e);
  BlockPlan plan;
  if ((st = block_plan(1, b.M, b.N, d, &a, &plan)) != GNORM_OK) return st;
  if (b.workspace == nullptr || !aligned(b.workspace, GNORM_WORKSPACE_ALIGN) ||
      b.workspace_bytes < block_workspace(b.M, b.N, d.num_sms))
    return GNORM_ERR_WORKSPACE;
  a.w1 = b.w1;
  a.w2 = b.w2;
  a.w_fp32 = b.w_fp32 ? 1 : 0;
  a.alpha = b.alpha;
  a.rstd1 = const_cast<float*>(b.rstd1);
  a.rstd2 = const_cast<float*>(b.rstd2);
  a.da = static_cast<uint16_t*>(b.da);
  a.dr = static_cast<uint8_t*>(b.dr);
  a.dg = static_cast<uint16_t*>(b.dg);
  a.ldda = b.ldda;
  a.lddr = b.lddr;
  a.lddg = b.lddg;
  a.partial = static_cast<float*>(b.workspace);
  a.partial_alpha = a.partial + static_cast<size_t>(plan.grid) * 2 * b.N;
  a.M = b.M;
  a.N = static_cast<int>(b.N);
  a.inv_n = static_cast<float>(1.0 / static_cast<double>(b.N));
  a.err = d.err_word;
  if (launch_block(1, plan, a, b.res_fp32 ? 1 : 0, s) != cudaSuccess) return GNORM_ERR_CUDA;
  BlockReduceArgs r;
  r.partial = a.partial;
  r.partial_alpha = a.partial_alpha;
  r.P = plan.grid;
  r.N = a.N;
  r.alpha = b.alpha;
  r.dw1 = b.dw1;
  r.dw2 = b.dw2;
  r.dw_fp32 = b.dw_fp32 ? 1 : 0;
  r.dalpha = b.dalpha;
  const int quads = 2 * a.N / 4;
  const int grid = (quads + kReduceQuads - 1) / kReduceQuads + 1;
  return launch_kernel(block_dw_reduce_kernel, grid, kReduceThreads, 0, s, use_pdl(), r) ==
                 cudaSuccess
             ? GNORM_OK
             : GNORM_ERR_CUDA;
}

size_t gnorm_block_bwd_workspace_bytes(int64_t M, int64_t N) {
  DeviceInfo d;
  if (check_block_shape(M, N) != GNORM_OK || device_info(&d) != GNORM_OK) return 0;
  return block_workspace(M, N, d.num_sms);
}

}  // extern "C"
