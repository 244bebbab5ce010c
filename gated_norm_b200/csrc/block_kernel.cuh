// block_kernel.cuh -- the norm after a block, its gate, the residual scale and the norm
// before the next block in one pass, forward and backward (sm_100a).
//
// Per row (a: the block's output, r: the residual, g: the gate, alpha: the residual scale):
//
//   r1 = 1 / sqrt(mean(a^2) + eps1)    ahat = a r1    b = ahat w1    s = g sigmoid(g)
//   h  = r + alpha s b                 r2 = 1 / sqrt(mean(h^2) + eps2)    hhat = h r2
//   z  = hhat w2
//
// and, from the gradients dh (of h through the residual) and dz (of z):
//
//   u2 = dz w2    c2 = mean(u2 hhat)    d  = dh + r2 (u2 - hhat c2)   (= dr)
//   t  = d s      dg = alpha d b (sigmoid(g) + s (1 - sigmoid(g)))
//   u1 = alpha t w1    c1 = mean(u1 ahat)    da = r1 (u1 - ahat c1)
//   T1 = sum over rows of t ahat    dw1 = alpha T1    dalpha = sum_j w1_j T1_j
//   dw2 = sum over rows of dz hhat
//
// The backward computes h again from a, g and r instead of reading the stored h: the same
// number of input streams, no rounding of h in between (dw2 and dr stay FP32-exact), and h
// need not be kept.
//
// Bound by HBM: with BF16 residuals the forward moves 10 bytes per element (a, g, r in; h, z
// out) and the backward 16 (dh, dz, a, g, r in; da, dg, dr out).  Design: the pipeline of the
// gated norm's kernels -- a producer warp streams row blocks of every input into a ring of
// shared-memory stages with bulk copies, the consumer warps own TPR threads per row and CPT
// 16-byte chunks per thread, row blocks are assigned round-robin, so each input byte is read
// from HBM once and the row sums between the passes cost shared-memory reads only.
//
// 16384 x 4096, BF16: forward 108 us (96% of the measured copy's rate), forward and backward 313
// (the backward about 205, 81%): the backward's 45 instructions an element, two computing warps
// a scheduler and two sums across eight warps a row.  512 threads with the same two chunks each
// spill (486 us), with one chunk each wait on sixteen warps' barriers (364).
#pragma once

#include "device_common.cuh"

namespace gnorm {

constexpr int kBlockMaxIn = 5;

// One input of a row block: rows of `row_bytes` bytes, `ld_bytes` apart.
struct BlockIn {
  const uint8_t* p = nullptr;
  long long ld_bytes = 0;
  uint32_t row_bytes = 0;
  uint32_t off = 0;  // byte offset inside a stage
};

struct BlockArgs {
  // a, r, g, dz, dh; absent ones (dz and dh in the forward) have p == nullptr, row_bytes 0
  BlockIn in[kBlockMaxIn];
  const void* w1 = nullptr;
  const void* w2 = nullptr;
  int w_fp32 = 0;
  const float* alpha = nullptr;  // device, one value; nullptr = 1
  float eps1 = 0.f, eps2 = 0.f;
  uint8_t* h = nullptr;  // forward outputs
  uint16_t* z = nullptr;
  float* rstd1 = nullptr;  // written by the forward, read by the backward
  float* rstd2 = nullptr;
  uint16_t* da = nullptr;  // backward outputs
  uint8_t* dr = nullptr;
  uint16_t* dg = nullptr;
  float* partial = nullptr;        // [grid, 2 N]: T1, dw2 of the CTA's rows
  float* partial_alpha = nullptr;  // [grid]: sum_j w1_j T1_j of the CTA's rows
  long long ldh = 0, ldz = 0, ldda = 0, lddr = 0, lddg = 0;  // elements
  long long M = 0;
  int N = 0;
  float inv_n = 0.f;
  int rows_per_stage = 0;
  int stages = 0;
  uint32_t stage_bytes = 0;
  uint32_t rstd_off = 0;  // backward: byte offset of the rows' rstd1 and rstd2 in a stage
  long long num_blocks = 0;
  unsigned* err = nullptr;
};

// Computing threads and resident CTAs per SM of a row geometry (kind 0 forward, 1 backward).
// 256 threads; one row group of 512 for the widest rows.  The registers that hold a row's
// intermediates decide the residency.  The producer's warp, the ninth, takes a further warp's share
// of one scheduler's registers: 3 CTAs of 288 threads leave 68 registers per thread, 2 leave 96,
// one leaves 168 (at 544 threads: 96).  The gated backwards spill 28 to 48 bytes a thread with one
// chunk, 20 to 36 with two and at most 128 threads a row, 0 to 8 with 256 threads a row; with 512
// threads a row 312 to 336 (two chunks) and 440 to 564 (four), the ungated ones 44 to 84 and 328 to
// 360: 8192 x 8192 with a gate takes 316 us backward (53% of the measured copy's rate), 4096 x
// 16384 434 (38%), forward 105 (99%) and 162 (64%).
GNORM_HD constexpr int block_threads(int tpr) { return tpr > 256 ? tpr : 256; }
GNORM_HD constexpr int block_ctas_per_sm(int kind, int tpr, int cpt) {
  return tpr > 256 ? 1 : kind == 0 ? (cpt == 1 ? 3 : 2) : (cpt == 1 ? 2 : 1);
}

// Eight residual values of chunk c (BF16 or FP32) as pairs.
template <bool kF32>
__device__ __forceinline__ void load_res_pairs(const uint8_t* row, int c, float2 p[4]) {
  if constexpr (kF32) {
    const float4* q = reinterpret_cast<const float4*>(row) + 2 * c;
    const float4 lo = q[0], hi = q[1];
    p[0] = make_float2(lo.x, lo.y);
    p[1] = make_float2(lo.z, lo.w);
    p[2] = make_float2(hi.x, hi.y);
    p[3] = make_float2(hi.z, hi.w);
  } else {
    bf16x8_to_pairs(reinterpret_cast<const uint4*>(row)[c], p);
  }
}

template <bool kF32>
__device__ __forceinline__ void store_res_pairs(uint8_t* row, int c, const float2 p[4]) {
  if constexpr (kF32) {
    float4* q = reinterpret_cast<float4*>(row) + 2 * c;
    q[0] = make_float4(p[0].x, p[0].y, p[1].x, p[1].y);
    q[1] = make_float4(p[2].x, p[2].y, p[3].x, p[3].y);
  } else {
    reinterpret_cast<uint4*>(row)[c] = pairs_to_bf16x8(p);
  }
}

__device__ __forceinline__ void load_w_pairs(const void* w, int w_fp32, int c, float2 p[4]) {
  if (w_fp32)
    load_weight_pairs<true>(w, c, p);
  else
    load_weight_pairs<false>(w, c, p);
}

// Ring header in shared memory: full and empty barriers, the stages' block ids and the row
// sums' slots, as in the gated norm's kernels.
struct BlockRing {
  uint64_t* full;
  uint64_t* empty;
  long long* blk_id;
  float* red_slots;
  uint8_t* stage0;
};

__device__ __forceinline__ BlockRing block_ring(uint8_t* smem) {
  BlockRing r;
  r.full = reinterpret_cast<uint64_t*>(smem);
  r.empty = r.full + kMaxStages;
  r.blk_id = reinterpret_cast<long long*>(smem + 256);
  r.red_slots = reinterpret_cast<float*>(smem + kRedSlotOffset);
  r.stage0 = smem + kHeaderBytes;
  return r;
}

// The producer warp: streams the CTA's row blocks through the ring.  Lane 0 waits for a free
// stage and posts the byte count; packed tensors are one bulk copy per block, strided ones a
// copy per row spread over the lanes.  kRstd: the rows' rstd values come along with 4-byte
// asynchronous copies counted on the same barrier.
template <bool kRstd>
__device__ __forceinline__ void block_producer(const BlockArgs& a, const BlockRing& ring,
                                               int lane) {
  const int S = a.stages;
  const int R = a.rows_per_stage;
  uint32_t row_total = 0;
  for (int i = 0; i < kBlockMaxIn; ++i) row_total += a.in[i].row_bytes;
  int s = 0;
  uint32_t phase = 0;
  for (long long blk = blockIdx.x;; blk += gridDim.x) {
    bool ok = true;
    if (lane == 0) ok = mbar_wait(&ring.empty[s], phase ^ 1u, a.err, kErrWaitEmpty);
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (!ok) break;
    const bool end = blk >= a.num_blocks;
    if (!end) {
      const long long r0 = blk * R;
      const long long left = a.M - r0;
      const int rows = static_cast<int>(left < R ? left : R);
      uint8_t* st = ring.stage0 + static_cast<size_t>(s) * a.stage_bytes;
      if (lane == 0) mbar_expect_tx(&ring.full[s], static_cast<uint32_t>(rows) * row_total);
      __syncwarp();
      for (int i = 0; i < kBlockMaxIn; ++i) {
        const BlockIn& t = a.in[i];
        if (t.p == nullptr) continue;
        uint8_t* dst = st + t.off;
        if (t.ld_bytes == t.row_bytes) {
          if (lane == 0)
            bulk_copy_g2s(dst, t.p + r0 * t.ld_bytes, static_cast<uint32_t>(rows) * t.row_bytes,
                          &ring.full[s]);
        } else {
          for (int j = lane; j < rows; j += 32)
            bulk_copy_g2s(dst + static_cast<size_t>(j) * t.row_bytes, t.p + (r0 + j) * t.ld_bytes,
                          t.row_bytes, &ring.full[s]);
        }
      }
      if constexpr (kRstd) {
        float* sr = reinterpret_cast<float*>(st + a.rstd_off);
        for (int j = lane; j < rows; j += 32) {
          async_copy_4(sr + j, a.rstd1 + r0 + j);
          async_copy_4(sr + R + j, a.rstd2 + r0 + j);
        }
      }
    }
    if constexpr (kRstd) async_copies_arrive(&ring.full[s]);
    if (lane == 0) {
      ring.blk_id[s] = end ? -1 : blk;
      mbar_arrive(&ring.full[s]);
    }
    if (end) break;
    if (++s == S) {
      s = 0;
      phase ^= 1u;
    }
  }
}

template <int TPR, int CPT, bool kGate, bool kRes32>
__global__ void __launch_bounds__(block_threads(TPR) + 32, block_ctas_per_sm(0, TPR, CPT))
    block_norm_fwd_kernel(const __grid_constant__ BlockArgs a) {
  constexpr int kNCT = block_threads(TPR);
  constexpr int kGroups = kNCT / TPR;
  // Weights stay in registers with one or two chunks per thread; wider rows reload them
  // (L1-resident; some spill up to 24 bytes a thread all the same).
  constexpr bool kKeepW = CPT <= 2;
  extern __shared__ __align__(128) uint8_t smem[];
  const BlockRing ring = block_ring(smem);
  const int S = a.stages, R = a.rows_per_stage, N = a.N;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&ring.full[s], 1);
      mbar_init(&ring.empty[s], kNCT / 32);
    }
    fence_barrier_init();
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  allow_dependent_launch();
  if (warp == 0) {
    block_producer<false>(a, ring, lane);
    return;
  }

  const int ctid = threadIdx.x - 32;
  const int group = ctid / TPR;
  const int lr = ctid - group * TPR;
  const int warp_group0 = (ctid & ~31) / TPR;
  const int n8 = N >> 3;
  const float2 alpha2 = splat2(a.alpha != nullptr ? *a.alpha : 1.f);
  float2 w1[kKeepW ? CPT : 1][4], w2[kKeepW ? CPT : 1][4];
  bool cval[CPT];
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    const int c = k * TPR + lr;
    cval[k] = c < n8;
    if constexpr (kKeepW) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w1[k][i] = w2[k][i] = splat2(0.f);
      if (cval[k]) {
        load_w_pairs(a.w1, a.w_fp32, c, w1[k]);
        load_w_pairs(a.w2, a.w_fp32, c, w2[k]);
      }
    }
  }

  int s = 0, slot = 0;
  uint32_t phase = 0;
  while (true) {
    if (!mbar_wait(&ring.full[s], phase, a.err, kErrWaitFull)) break;
    const long long blk = ring.blk_id[s];
    if (blk < 0) break;
    const long long r0 = blk * R;
    const long long left = a.M - r0;
    const int rows = static_cast<int>(left < R ? left : R);
    const uint8_t* st = ring.stage0 + static_cast<size_t>(s) * a.stage_bytes;
    for (int rb = 0; rb < rows; rb += kGroups) {
      if (rb + warp_group0 >= rows) break;
      const int row = rb + group;
      const bool valid = row < rows;
      const size_t srow = valid ? row : 0;
      const long long grow = r0 + row;
      const uint8_t* sa = st + a.in[0].off + srow * a.in[0].row_bytes;
      const uint8_t* sr = st + a.in[1].off + srow * a.in[1].row_bytes;
      const uint8_t* sg = st + a.in[2].off + srow * a.in[2].row_bytes;
      // the norm after the block
      uint4 av[CPT];
      float part[CPT];
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        part[k] = 0.f;
        if (cval[k]) {
          av[k] = reinterpret_cast<const uint4*>(sa)[k * TPR + lr];
          float2 ap[4];
          bf16x8_to_pairs(av[k], ap);
          part[k] = chunk_dot(ap, ap);
        }
      }
      float ss = row_sum<TPR>(combine_chunks<CPT>(part), ring.red_slots, group, lr, slot);
      slot ^= 1;
      const float r1 = rsqrtf(fmaf(ss, a.inv_n, a.eps1));
      const float2 r12 = splat2(r1);
      // gate, residual scale and sum; h stays in FP32 registers for the second norm
      float2 h[CPT][4];
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        part[k] = 0.f;
        if (cval[k]) {
          const int c = k * TPR + lr;
          float2 ap[4], gp[4], wl[4];
          bf16x8_to_pairs(av[k], ap);
          load_res_pairs<kRes32>(sr, c, h[k]);
          if constexpr (kGate) bf16x8_to_pairs(reinterpret_cast<const uint4*>(sg)[c], gp);
          if constexpr (!kKeepW) load_w_pairs(a.w1, a.w_fp32, c, wl);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float2 b = mul2(mul2(ap[i], r12), kKeepW ? w1[k][i] : wl[i]);
            if constexpr (kGate) b = mul2(b, mul2(gp[i], sigmoid2(gp[i])));
            h[k][i] = fma2(alpha2, b, h[k][i]);
          }
          part[k] = chunk_dot(h[k], h[k]);
          if (valid)
            store_res_pairs<kRes32>(a.h + grow * a.ldh * (kRes32 ? 4 : 2), c, h[k]);
        }
      }
      ss = row_sum<TPR>(combine_chunks<CPT>(part), ring.red_slots, group, lr, slot);
      slot ^= 1;
      const float r2 = rsqrtf(fmaf(ss, a.inv_n, a.eps2));
      const float2 r22 = splat2(r2);
      if (valid && lr == 0) {
        a.rstd1[grow] = r1;
        a.rstd2[grow] = r2;
      }
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        if (cval[k]) {
          const int c = k * TPR + lr;
          float2 zp[4], wl[4];
          if constexpr (!kKeepW) load_w_pairs(a.w2, a.w_fp32, c, wl);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            zp[i] = mul2(mul2(h[k][i], r22), kKeepW ? w2[k][i] : wl[i]);
          if (valid) reinterpret_cast<uint4*>(a.z + grow * a.ldz)[c] = pairs_to_bf16x8(zp);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ring.empty[s]);
    if (++s == S) {
      s = 0;
      phase ^= 1u;
    }
  }
}

// Sums `v` over the CTA's consumer threads in a fixed order (warp butterfly, then the warps
// one after another); every thread returns the sum.  `slots`: one float per warp.
template <int kNCT>
__device__ __forceinline__ float cta_sum(float v, float* slots, int ctid) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((ctid & 31) == 0) slots[ctid >> 5] = v;
  named_barrier_sync(15, kNCT);
  v = slots[0];
#pragma unroll
  for (int i = 1; i < kNCT / 32; ++i) v += slots[i];
  return v;
}

template <int TPR, int CPT, bool kGate, bool kRes32>
__global__ void __launch_bounds__(block_threads(TPR) + 32, block_ctas_per_sm(1, TPR, CPT))
    block_norm_bwd_kernel(const __grid_constant__ BlockArgs a) {
  constexpr int kNCT = block_threads(TPR);
  constexpr int kGroups = kNCT / TPR;
  // Registers: with 256 threads per CTA the weights and a row's intermediates (hhat, u2,
  // sigmoid) stay in registers between the passes; with 512 the weights are reloaded
  // (L1-resident), and rows of four chunks per thread also recompute the intermediates from
  // the staged inputs (both still spill: block_ctas_per_sm).
  constexpr bool kKeepW = CPT <= 2 && TPR <= 256;
  constexpr bool kKeep = CPT <= 2;
  extern __shared__ __align__(128) uint8_t smem[];
  const BlockRing ring = block_ring(smem);
  const int S = a.stages, R = a.rows_per_stage, N = a.N;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&ring.full[s], 33);  // 32 producer lanes' rstd copies + lane 0's arrival
      mbar_init(&ring.empty[s], kNCT / 32);
    }
    fence_barrier_init();
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  allow_dependent_launch();
  if (warp == 0) {
    block_producer<true>(a, ring, lane);
    return;
  }

  const int ctid = threadIdx.x - 32;
  const int group = ctid / TPR;
  const int lr = ctid - group * TPR;
  const int warp_group0 = (ctid & ~31) / TPR;
  const int n8 = N >> 3;
  const float alpha = a.alpha != nullptr ? *a.alpha : 1.f;
  const float2 alpha2 = splat2(alpha);
  const bool has_dh = a.in[4].p != nullptr;
  float2 w1[kKeepW ? CPT : 1][4], w2[kKeepW ? CPT : 1][4];
  float2 t1[CPT][4], dw2[CPT][4];  // this thread's columns of T1 and dw2
  bool cval[CPT];
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    const int c = k * TPR + lr;
    cval[k] = c < n8;
#pragma unroll
    for (int i = 0; i < 4; ++i) t1[k][i] = dw2[k][i] = splat2(0.f);
    if constexpr (kKeepW) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w1[k][i] = w2[k][i] = splat2(0.f);
      if (cval[k]) {
        load_w_pairs(a.w1, a.w_fp32, c, w1[k]);
        load_w_pairs(a.w2, a.w_fp32, c, w2[k]);
      }
    }
  }

  int s = 0, slot = 0;
  uint32_t phase = 0;
  while (true) {
    if (!mbar_wait(&ring.full[s], phase, a.err, kErrWaitFull)) break;
    const long long blk = ring.blk_id[s];
    if (blk < 0) break;
    const long long r0 = blk * R;
    const long long left = a.M - r0;
    const int rows = static_cast<int>(left < R ? left : R);
    const uint8_t* st = ring.stage0 + static_cast<size_t>(s) * a.stage_bytes;
    const float* srs = reinterpret_cast<const float*>(st + a.rstd_off);
    for (int rb = 0; rb < rows; rb += kGroups) {
      if (rb + warp_group0 >= rows) break;
      const int row = rb + group;
      const bool valid = row < rows;
      const size_t srow = valid ? row : 0;
      const long long grow = r0 + row;
      const uint8_t* sa = st + a.in[0].off + srow * a.in[0].row_bytes;
      const uint8_t* sr = st + a.in[1].off + srow * a.in[1].row_bytes;
      const uint8_t* sg = st + a.in[2].off + srow * a.in[2].row_bytes;
      const uint8_t* sdz = st + a.in[3].off + srow * a.in[3].row_bytes;
      const uint8_t* sdh = st + a.in[4].off + srow * a.in[4].row_bytes;
      const float r1 = srs[srow], r2 = srs[R + srow];
      const float2 r12 = splat2(r1), r22 = splat2(r2);

      // hhat and u2 of chunk k from the staged rows; ah, b, the sigmoid and s as well
      auto forward_chunk = [&](int k, float2 ah[4], float2 b[4], float2 sg4[4], float2 hh[4]) {
        const int c = k * TPR + lr;
        float2 ap[4], gp[4], rp[4], wl[4];
        bf16x8_to_pairs(reinterpret_cast<const uint4*>(sa)[c], ap);
        load_res_pairs<kRes32>(sr, c, rp);
        if constexpr (kGate) bf16x8_to_pairs(reinterpret_cast<const uint4*>(sg)[c], gp);
        if constexpr (!kKeepW) load_w_pairs(a.w1, a.w_fp32, c, wl);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ah[i] = mul2(ap[i], r12);
          b[i] = mul2(ah[i], kKeepW ? w1[k][i] : wl[i]);
          float2 sb = b[i];
          if constexpr (kGate) {
            sg4[i] = sigmoid2(gp[i]);
            sb = mul2(b[i], mul2(gp[i], sg4[i]));
          }
          hh[i] = mul2(fma2(alpha2, sb, rp[i]), r22);
        }
      };

      // pass 1: the sum of u2 hhat; dw2
      float2 hh[kKeep ? CPT : 1][4], u2[kKeep ? CPT : 1][4], sgm[kKeep ? CPT : 1][4];
      float part[CPT];
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        part[k] = 0.f;
        if (cval[k]) {
          const int c = k * TPR + lr;
          float2 ah[4], b[4], sl[4], hl[4], dzp[4], ul[4], wl[4];
          forward_chunk(k, ah, b, sl, hl);
          bf16x8_to_pairs(reinterpret_cast<const uint4*>(sdz)[c], dzp);
          if constexpr (!kKeepW) load_w_pairs(a.w2, a.w_fp32, c, wl);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ul[i] = mul2(dzp[i], kKeepW ? w2[k][i] : wl[i]);
            if (valid) dw2[k][i] = fma2(dzp[i], hl[i], dw2[k][i]);
          }
          part[k] = chunk_dot(ul, hl);
          if constexpr (kKeep) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              hh[k][i] = hl[i];
              u2[k][i] = ul[i];
              if constexpr (kGate) sgm[k][i] = sl[i];
            }
          }
        }
      }
      float dot = row_sum<TPR>(combine_chunks<CPT>(part), ring.red_slots, group, lr, slot);
      slot ^= 1;
      const float2 nc2 = splat2(-(dot * a.inv_n));

      // pass 2: dr, dg, the sum of u1 ahat; T1.  u1 takes u2's registers.
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        part[k] = 0.f;
        if (cval[k]) {
          const int c = k * TPR + lr;
          float2 ah[4], b[4], sl[4], hl[4], ul[4], d[4], gp[4], wl1[4];
          if constexpr (!kKeepW) load_w_pairs(a.w1, a.w_fp32, c, wl1);
          if constexpr (kKeep) {
            float2 ap[4];
            bf16x8_to_pairs(reinterpret_cast<const uint4*>(sa)[c], ap);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              ah[i] = mul2(ap[i], r12);
              b[i] = mul2(ah[i], kKeepW ? w1[k][i] : wl1[i]);
              hl[i] = hh[k][i];
              ul[i] = u2[k][i];
              if constexpr (kGate) sl[i] = sgm[k][i];
            }
          } else {
            float2 dzp[4], wl2[4];
            forward_chunk(k, ah, b, sl, hl);
            bf16x8_to_pairs(reinterpret_cast<const uint4*>(sdz)[c], dzp);
            load_w_pairs(a.w2, a.w_fp32, c, wl2);
#pragma unroll
            for (int i = 0; i < 4; ++i) ul[i] = mul2(dzp[i], wl2[i]);
          }
          if (has_dh)
            load_res_pairs<kRes32>(sdh, c, d);
          else
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = splat2(0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] = fma2(r22, fma2(hl[i], nc2, ul[i]), d[i]);
          if (valid) store_res_pairs<kRes32>(a.dr + grow * a.lddr * (kRes32 ? 4 : 2), c, d);
          if constexpr (kGate) {
            float2 dgp[4];
            bf16x8_to_pairs(reinterpret_cast<const uint4*>(sg)[c], gp);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // sigmoid' as in the gated norm: sigmoid (1 + g (1 - sigmoid))
              const float2 ds = mul2(sl[i], gate_grad_bracket(gp[i], sl[i]));
              dgp[i] = mul2(mul2(alpha2, mul2(d[i], b[i])), ds);
              d[i] = mul2(d[i], mul2(gp[i], sl[i]));  // t = d s
            }
            if (valid) reinterpret_cast<uint4*>(a.dg + grow * a.lddg)[c] = pairs_to_bf16x8(dgp);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (valid) t1[k][i] = fma2(d[i], ah[i], t1[k][i]);
            ul[i] = mul2(mul2(alpha2, d[i]), kKeepW ? w1[k][i] : wl1[i]);  // u1
            if constexpr (kKeep) u2[k][i] = ul[i];
          }
          part[k] = chunk_dot(ul, ah);
        }
      }
      const float nc2f = nc2.x;
      dot = row_sum<TPR>(combine_chunks<CPT>(part), ring.red_slots, group, lr, slot);
      slot ^= 1;
      const float2 nc1 = splat2(-(dot * a.inv_n));

      // pass 3: da = r1 (u1 - ahat c1)
#pragma unroll
      for (int k = 0; k < CPT; ++k) {
        if (cval[k]) {
          const int c = k * TPR + lr;
          float2 ah[4], ul[4], dap[4];
          if constexpr (kKeep) {
            float2 ap[4];
            bf16x8_to_pairs(reinterpret_cast<const uint4*>(sa)[c], ap);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              ah[i] = mul2(ap[i], r12);
              ul[i] = u2[k][i];
            }
          } else {
            float2 b[4], sl[4], hl[4], dzp[4], d[4], gp[4], wl[4];
            forward_chunk(k, ah, b, sl, hl);
            bf16x8_to_pairs(reinterpret_cast<const uint4*>(sdz)[c], dzp);
            load_w_pairs(a.w2, a.w_fp32, c, wl);
            if (has_dh)
              load_res_pairs<kRes32>(sdh, c, d);
            else
#pragma unroll
              for (int i = 0; i < 4; ++i) d[i] = splat2(0.f);
            if constexpr (kGate) bf16x8_to_pairs(reinterpret_cast<const uint4*>(sg)[c], gp);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              d[i] = fma2(r22, fma2(hl[i], splat2(nc2f), mul2(dzp[i], wl[i])), d[i]);
            load_w_pairs(a.w1, a.w_fp32, c, wl);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if constexpr (kGate) d[i] = mul2(d[i], mul2(gp[i], sl[i]));
              ul[i] = mul2(mul2(alpha2, d[i]), wl[i]);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) dap[i] = mul2(r12, fma2(ah[i], nc1, ul[i]));
          if (valid) reinterpret_cast<uint4*>(a.da + grow * a.ldda)[c] = pairs_to_bf16x8(dap);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ring.empty[s]);
    if (++s == S) {
      s = 0;
      phase ^= 1u;
    }
  }

  // This CTA's partial rows: its row groups' accumulators added in a fixed order, T1 then dw2.
  named_barrier_sync(15, kNCT);  // every consumer is done with the stage buffers
  float* prow = a.partial + static_cast<size_t>(blockIdx.x) * 2 * N;
  float wsum = 0.f;  // this thread's share of sum_j w1_j T1_j
  float* red = reinterpret_cast<float*>(ring.stage0);  // [kGroups, N]
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float2(*acc)[4] = which == 0 ? t1 : dw2;
    if constexpr (kGroups > 1) {
      if (which == 1) named_barrier_sync(15, kNCT);  // the first sum has been read
    }
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      if (cval[k]) {
        const int c = k * TPR + lr;
        float* dst = kGroups > 1 ? red + group * N + c * 8 : prow + which * N + c * 8;
        reinterpret_cast<float4*>(dst)[0] =
            make_float4(acc[k][0].x, acc[k][0].y, acc[k][1].x, acc[k][1].y);
        reinterpret_cast<float4*>(dst)[1] =
            make_float4(acc[k][2].x, acc[k][2].y, acc[k][3].x, acc[k][3].y);
        if (which == 0) {
          float2 wl[4];
          load_w_pairs(a.w1, a.w_fp32, c, wl);
          wsum += chunk_dot(acc[k], wl);
        }
      }
    }
    if constexpr (kGroups > 1) {
      named_barrier_sync(15, kNCT);
      const int n4 = N >> 2;
      const float4* red4 = reinterpret_cast<const float4*>(red);
      for (int j4 = ctid; j4 < n4; j4 += kNCT) {
        float4 v = red4[j4];
#pragma unroll
        for (int gi = 1; gi < kGroups; ++gi) {
          const float4 o = red4[gi * n4 + j4];
          v.x += o.x;
          v.y += o.y;
          v.z += o.z;
          v.w += o.w;
        }
        reinterpret_cast<float4*>(prow + which * N)[j4] = v;
      }
    }
  }
  named_barrier_sync(15, kNCT);
  wsum = cta_sum<kNCT>(wsum, ring.red_slots, ctid);
  if (ctid == 0) a.partial_alpha[blockIdx.x] = wsum;
}

struct BlockReduceArgs {
  const float* partial = nullptr;
  const float* partial_alpha = nullptr;
  int P = 0;
  int N = 0;
  const float* alpha = nullptr;
  void* dw1 = nullptr;
  void* dw2 = nullptr;
  int dw_fp32 = 0;
  float* dalpha = nullptr;
};

// Second pass over the partial rows [P, 2 N], in the fixed order of dw_reduce_kernel: a CTA
// owns kReduceQuads column quads with kReduceLanes row lanes each; a lane adds its rows in
// increasing order, the lanes of a quad are combined by shuffles and then pairwise through
// shared memory.  The last CTA sums the P shares of dalpha instead.
__global__ void __launch_bounds__(kReduceThreads)
    block_dw_reduce_kernel(const __grid_constant__ BlockReduceArgs a) {
  constexpr int kWarps = kReduceThreads / 32;
  constexpr int kBatch = 8;
  __shared__ float4 red[kWarps][kReduceQuads];
  __shared__ float slots[kWarps];
  grid_dependency_wait();
  allow_dependent_launch();
  if (blockIdx.x == gridDim.x - 1) {
    float v = 0.f;
    for (int i = threadIdx.x; i < a.P; i += kReduceThreads) v += __ldcg(a.partial_alpha + i);
    v = cta_sum<kReduceThreads>(v, slots, threadIdx.x);
    if (threadIdx.x == 0 && a.dalpha != nullptr) *a.dalpha = v;
    return;
  }
  const int q = threadIdx.x % kReduceQuads;
  const int rl = threadIdx.x / kReduceQuads;
  const int warp = threadIdx.x >> 5;
  const int n4 = a.N >> 2;  // column quads of one weight
  const int j4 = blockIdx.x * kReduceQuads + q;
  const bool valid = j4 < 2 * n4;
  const float4* p4 = reinterpret_cast<const float4*>(a.partial);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int b0 = rl; b0 < a.P; b0 += kReduceLanes * kBatch) {
    float4 v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int b = b0 + kReduceLanes * i;
      v[i] = (valid && b < a.P) ? __ldcg(p4 + static_cast<size_t>(b) * 2 * n4 + j4)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (b0 + kReduceLanes * i < a.P) {
        acc.x += v[i].x;
        acc.y += v[i].y;
        acc.z += v[i].z;
        acc.w += v[i].w;
      }
    }
  }
#pragma unroll
  for (int off = kReduceQuads; off < 32; off <<= 1) {
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, off);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, off);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, off);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, off);
  }
  if ((threadIdx.x & 31) < kReduceQuads) red[warp][q] = acc;
  __syncthreads();
#pragma unroll
  for (int st = kWarps / 2; st > 0; st >>= 1) {
    if (threadIdx.x < st * kReduceQuads) {
      const int w = threadIdx.x / kReduceQuads;
      float4 m = red[w][q];
      const float4 o = red[w + st][q];
      m.x += o.x;
      m.y += o.y;
      m.z += o.z;
      m.w += o.w;
      red[w][q] = m;
    }
    __syncthreads();
  }
  if (threadIdx.x < kReduceQuads && valid) {
    float4 m = red[0][q];
    const bool first = j4 < n4;
    if (first) {
      const float al = a.alpha != nullptr ? *a.alpha : 1.f;
      m = make_float4(al * m.x, al * m.y, al * m.z, al * m.w);
    }
    void* dw = first ? a.dw1 : a.dw2;
    const int jj = first ? j4 : j4 - n4;
    if (a.dw_fp32) {
      reinterpret_cast<float4*>(dw)[jj] = m;
    } else {
      uint2 v;
      v.x = pack_bf16x2(m.x, m.y);
      v.y = pack_bf16x2(m.z, m.w);
      reinterpret_cast<uint2*>(dw)[jj] = v;
    }
  }
}

}  // namespace gnorm
