// delta_head.cuh -- the gated delta rule's forward with a whole head per CTA, on tcgen05
// (formulas and notation: delta_common.cuh).
//
// The strips of delta_scan.cuh spread one head over eight SMs, which is right while there are
// SMs to spare.  With more strips than SMs what counts is the work per SM, and shared memory
// binds the strips: each instruction reads its right operand for sixteen columns.  Here the
// right operands are read for the head's 128 columns at once: lane v of the accumulators is
// column v of V, transposed as there (S^T: 128 x K), and each intermediate goes back into
// tensor memory as the next product's left operand.
//
//   1  X = S K^T  (then Q: O = S Q^T)     2  D = -(beta X) N^T, W = X + D
//   3  U = (lambda Y) K                   4  O = gamma O + Y P^T,  S' = e^{G_C} S + U
//
// Eight warps own the rows (a thread one column of V: half of S's row in FP32 registers for the
// whole sequence, half of the chunk's tokens), one warp issues the products, one the copies.  A
// chunk takes about 4.1 us (40 heads of 4096 tokens 310 us; 367 while one thread issued the
// products from a branch of its own), half of it in the products' latency, which another head
// on the SM could fill if tensor memory (480 of 512 columns here) had the room.
#pragma once

#include "delta_common.cuh"
#include "tcgen05.cuh"

namespace gnorm {

constexpr int kHeadWarps = 8;
constexpr int kHeadThreads = (kHeadWarps + 2) * 32;

template <int KD, int VD>
struct HeadStage {
  static constexpr int kQ = 0;
  static constexpr int kK = KD / 64 * kTileBytes;
  static constexpr int kV = 2 * kK;
  static constexpr int kTri = kV + VD / 64 * kTileBytes;  // N (three parts), P (two)
  static constexpr int kScal = kTri + 5 * kTriGrid;
  static constexpr int kBytes = kScal + 1024;
};
template <int KD, int VD>
GNORM_HD constexpr int head_smem() {
  return 2 * HeadStage<KD, VD>::kBytes + 256 + 1024;  // barriers; 1024: alignment
}

// Sixteen pairs of FP32 values as three parts of packed BF16 pairs.
__device__ __forceinline__ void split3_16(const float* x, uint32_t p0[16], uint32_t p1[16], uint32_t p2[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    uint32_t p[3];
    split3(x[2 * i], x[2 * i + 1], p);
    p0[i] = p[0];
    p1[i] = p[1];
    p2[i] = p[2];
  }
}

template <int KD, int VD>
__global__ void __launch_bounds__(kHeadThreads, 1)
    delta_head_fwd_kernel(const __grid_constant__ DeltaArgs a, const __grid_constant__ DeltaMaps maps) {
  using St = HeadStage<KD, VD>;
  constexpr int kHalf = KD / 2;        // columns of K per thread
  constexpr int kRows = VD / 32 * 2;   // warps that own rows
  // tensor memory columns
  constexpr uint32_t kS = 0;           // S, three parts of KD / 2; then lambda Y, three of 32
  constexpr uint32_t kX = 192;         // X, D; then U (KD columns)
  constexpr uint32_t kO = 320;
  constexpr uint32_t kA = 384;         // -beta X, three parts of 32; then Y, two
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + 2 * St::kBytes);
  uint64_t *full = bars, *empty = bars + 2, *cleared = bars + 4, *s_in = bars + 5, *x_out = bars + 6,
           *a_in = bars + 7, *d_out = bars + 8, *y_in = bars + 9, *o_in = bars + 10, *u_out = bars + 11,
           *o_out = bars + 12, *o_free = bars + 13;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 14);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x;
  const int hk = h / (a.Hv / a.Hk);
  if (warp == kHeadWarps) tmem_alloc(tslot, 512);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1 + kRows);
    }
    mbar_init(cleared, 1);
    for (uint64_t* b : {x_out, d_out, u_out, o_out}) mbar_init(b, 1);
    for (uint64_t* b : {s_in, a_in, y_in, o_in, o_free}) mbar_init(b, kRows);
    fence_barrier_init();
  }
  // N and P above the diagonal, where no copy arrives
  for (int i = tid; i < 2 * 5 * kTriGrid / 16; i += kHeadThreads) {
    uint8_t* p = smem + (i >= 5 * kTriGrid / 16 ? St::kBytes - 5 * kTriGrid : 0) + St::kTri + i * 16;
    *reinterpret_cast<uint4*>(p) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_smem_to_async();
  const int b = seq_by_length(a.seq, blockIdx.y, lane);
  const long long start = seq_start(a.seq, b), end = seq_end(a.seq, b);
  const long long base = seq_base(a.seq, b);
  const int chunks = static_cast<int>((end - start + kChunk - 1) / kChunk);
  const int last_live = static_cast<int>(end - start - static_cast<long long>(chunks - 1) * kChunk);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();  // (the kernel before is this call's own: see delta_scan.cuh)
  allow_dependent_launch();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tslot, 0);
  bool alive = true;
  auto wait = [&](uint64_t* bar, uint32_t parity, unsigned bit) {
    if (alive) alive = mbar_spin(bar, parity & 1u, a.err, bit);
  };
  auto wait_stage = [&](int c) {
    wait(&full[c & 1], static_cast<uint32_t>(c >> 1), kErrWaitFull);
    if (c + 1 == chunks && last_live < kChunk) wait(cleared, 0, kErrWaitFull);
  };

  if (warp == kHeadWarps + 1) {
    // ---- copies
    for (int c = 0; c < chunks; ++c) {
      uint8_t* st = smem + (c & 1) * St::kBytes;
      uint64_t* bar = &full[c & 1];
      if (c >= 2) wait(&empty[c & 1], static_cast<uint32_t>((c >> 1) - 1), kErrWaitEmpty);
      const int t0 = static_cast<int>(start + static_cast<long long>(c) * kChunk);
      const uint8_t* prep = a.prep + ((base + c) * a.Hv + h) * kPrepBytes;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, 2 * St::kK + VD / 64 * kTileBytes + 5 * kTriBytes + 784);
#pragma unroll
        for (int kt = 0; kt < KD / 64; ++kt)
          tma_load_2d(st + St::kK + kt * kTileBytes, &maps.k, hk * KD + kt * 64, t0, bar);
#pragma unroll
        for (int vt = 0; vt < VD / 64; ++vt)
          tma_load_2d(st + St::kV + vt * kTileBytes, &maps.v, h * VD + vt * 64, t0, bar);
        bulk_copy_g2s(st + St::kScal, prep + kPrepTri, 784, bar);
#pragma unroll
        for (int kt = 0; kt < KD / 64; ++kt)
          tma_load_2d(st + St::kQ + kt * kTileBytes, &maps.q, hk * KD + kt * 64, t0, bar);
      }
      __syncwarp();
      // a row of matrices each: five parts of eight rows
      for (int i = lane; i < 40; i += 32) {
        const int part = i >> 3, t = i & 7;
        bulk_copy_g2s(st + St::kTri + part * kTriGrid + t * 1024,
                      prep + part * kTriBytes + tri_row(t) * 128, (t / 2 + 1) * 256, bar);
      }
      if (c + 1 == chunks && last_live < kChunk) {
        wait(bar, static_cast<uint32_t>(c >> 1), kErrWaitFull);
        clear_rows<32>(st + St::kQ, 128, 2 * (KD / 64) + VD / 64, kTileBytes, last_live, lane);
        fence_smem_to_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(cleared);
      }
    }
    // the last arrivals from the tensor cores come before the CTA leaves
    for (int c = chunks; c < chunks + 2; ++c)
      if (c >= 2) wait(&empty[c & 1], static_cast<uint32_t>((c >> 1) - 1), kErrWaitEmpty);
  } else if (warp == kHeadWarps) {
    // ---- products
    {
      const bool lead = elect_one();
      constexpr uint32_t idK = mma_desc<false, false, 64>(), idU = mma_desc<false, true, KD>();
      for (int c = 0; c < chunks; ++c) {
        const uint32_t sg = sbase + (c & 1) * St::kBytes;
        wait_stage(c);
        wait(s_in, c, kErrWaitMma);
        tc_fence_after();
        const uint64_t kd = smem_desc(sg + St::kK, 16, 1024), qd = smem_desc(sg + St::kQ, 16, 1024);
        const uint64_t kt = smem_desc(sg + St::kK, kTileBytes, 1024);  // transposed
        const uint64_t td = smem_desc_plain(sg + St::kTri, 128, 1024);
        auto rows_at = [](int ks) { return static_cast<uint32_t>((ks >> 2) * kTileBytes + (ks & 3) * 32); };
        auto tri_at = [](int part, int kb) { return static_cast<uint32_t>(part * kTriGrid + 2 * kb * 128); };
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
          for (int ks = 0; ks < KD / 16; ++ks)
            tc_mma_tw(lead, tmem + kX, tmem + kS + part * kHalf + ks * 8, desc_at(kd, rows_at(ks)), idK, part + ks > 0);
        if (lead) tc_commit(x_out);
        if (c > 0) wait(o_free, c - 1, kErrWaitMma);
        tc_fence_after();
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int ks = 0; ks < KD / 16; ++ks)
            tc_mma_tw(lead, tmem + kO, tmem + kS + part * kHalf + ks * 8, desc_at(qd, rows_at(ks)), idK, part + ks > 0);
        wait(a_in, c, kErrWaitMma);
        tc_fence_after();
#pragma unroll
        for (int kb = 0; kb < 4; ++kb)
#pragma unroll
          for (int x = 0; x < 3; ++x)
#pragma unroll
            for (int n = 0; n + x < 3; ++n)
              tc_mma_tw(lead, tmem + kX, tmem + kA + x * 32 + kb * 8, desc_at(td, tri_at(n, kb)), idK, kb + x + n > 0);
        if (lead) tc_commit(d_out);
        wait(y_in, c, kErrWaitMma);
        tc_fence_after();
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc_mma_tw(lead, tmem + kX, tmem + kS + part * 32 + ks * 8,
                     desc_at(kt, ks * 2048), idU, part + ks > 0);
        if (lead) tc_commit(u_out);
        wait(o_in, c, kErrWaitMma);
        tc_fence_after();
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) {
          tc_mma_tw(lead, tmem + kO, tmem + kA + kb * 8, desc_at(td, tri_at(3, kb)), idK, true);
          tc_mma_tw(lead, tmem + kO, tmem + kA + 32 + kb * 8, desc_at(td, tri_at(3, kb)), idK, true);
          tc_mma_tw(lead, tmem + kO, tmem + kA + kb * 8, desc_at(td, tri_at(4, kb)), idK, true);
        }
        if (lead) tc_commit(o_out);
        if (lead) tc_commit(&empty[c & 1]);
      }
      // the last chunk's products end before tensor memory is freed: o_out is waited for below
    }
  } else if ((warp & 3) * 32 < VD) {
    // ---- rows
    const int v = (warp & 3) * 32 + lane, hf = warp >> 2;
    const uint32_t mine = tmem + (static_cast<uint32_t>(warp & 3) << 21);
    auto arrive = [&](uint64_t* bar) {  // tensor-memory writes (or reads) before it are done
      tc_store_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    float st[kHalf];
    const long long head_state = (static_cast<long long>(b) * a.Hv + h) * KD * VD + v;
    if (a.state_in != nullptr) {
#pragma unroll
      for (int i = 0; i < kHalf; ++i)
        st[i] = a.state_in[head_state + static_cast<long long>(hf * kHalf + i) * VD];
    } else {
#pragma unroll
      for (int i = 0; i < kHalf; ++i) st[i] = 0.f;
    }
    auto put_s = [&]() {
#pragma unroll
      for (int n = 0; n < kHalf / 32; ++n) {
        uint32_t p0[16], p1[16], p2[16];
        split3_16(st + n * 32, p0, p1, p2);
        const uint32_t at = mine + kS + hf * (kHalf / 2) + n * 16;
        tc_store16(at, p0);
        tc_store16(at + kHalf, p1);
        tc_store16(at + 2 * kHalf, p2);
      }
    };
    auto put_o = [&](int c) {  // the output of chunk c
      wait(o_out, c, kErrWaitMma);
      tc_fence_after();
      float o[32];
      tc_load16(mine + kO + hf * 32, o);
      tc_load16(mine + kO + hf * 32 + 16, o + 16);
      arrive(o_free);
      const int live = (c + 1 == chunks ? last_live : kChunk) - hf * 32;
      const long long t0 = start + static_cast<long long>(c) * kChunk + hf * 32;
      uint16_t* dst = a.o + t0 * a.ldo + static_cast<long long>(h) * VD + v;
      if (live >= 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i, dst += a.ldo)
          *dst = __bfloat16_as_ushort(__float2bfloat16_rn(a.scale * o[i]));
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i, dst += a.ldo)
          if (i < live) *dst = __bfloat16_as_ushort(__float2bfloat16_rn(a.scale * o[i]));
      }
    };
    if (chunks > 0) {
      put_s();
      arrive(s_in);
    }
    for (int c = 0; c < chunks; ++c) {
      const uint8_t* stage = smem + (c & 1) * St::kBytes;
      const float* scal = reinterpret_cast<const float*>(stage + St::kScal);
      const float4* beta = reinterpret_cast<const float4*>(scal + hf * 32);
      const float4* gamma = reinterpret_cast<const float4*>(scal + 64 + hf * 32);
      const float4* lambda = reinterpret_cast<const float4*>(scal + 128 + hf * 32);
      if (c > 0) put_o(c - 1);
      wait_stage(c);
      wait(x_out, c, kErrWaitMma);
      tc_fence_after();
      // X = V - gamma K S
      float x[32];
      tc_load16(mine + kX + hf * 32, x);
      tc_load16(mine + kX + hf * 32 + 16, x + 16);
      {
        const uint8_t* vt = stage + St::kV + (v >> 6) * kTileBytes + (v & 7) * 2;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 gm = gamma[i];
          const float gs[4] = {gm.x, gm.y, gm.z, gm.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint16_t w = *reinterpret_cast<const uint16_t*>(vt + tile_off(hf * 32 + i * 4 + e, (v & 63) >> 3));
            x[i * 4 + e] = fmaf(-gs[e], x[i * 4 + e], __uint_as_float(static_cast<uint32_t>(w) << 16));
          }
        }
        float t[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 be = beta[i];
          t[4 * i] = -be.x * x[4 * i];
          t[4 * i + 1] = -be.y * x[4 * i + 1];
          t[4 * i + 2] = -be.z * x[4 * i + 2];
          t[4 * i + 3] = -be.w * x[4 * i + 3];
        }
        uint32_t p0[16], p1[16], p2[16];
        split3_16(t, p0, p1, p2);
        tc_store16(mine + kA + hf * 16, p0);
        tc_store16(mine + kA + 32 + hf * 16, p1);
        tc_store16(mine + kA + 64 + hf * 16, p2);
      }
      arrive(a_in);
      wait(d_out, c, kErrWaitMma);
      tc_fence_after();
      {
        float t[32];
        tc_load16(mine + kX + hf * 32, t);
        tc_load16(mine + kX + hf * 32 + 16, t + 16);
        // Y = beta W, and lambda Y
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 be = beta[i];
          x[4 * i] = be.x * (x[4 * i] + t[4 * i]);
          x[4 * i + 1] = be.y * (x[4 * i + 1] + t[4 * i + 1]);
          x[4 * i + 2] = be.z * (x[4 * i + 2] + t[4 * i + 2]);
          x[4 * i + 3] = be.w * (x[4 * i + 3] + t[4 * i + 3]);
        }
        uint32_t p0[16], p1[16], p2[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) split2(x[2 * i], x[2 * i + 1], p0[i], p1[i]);
        tc_store16(mine + kA + hf * 16, p0);
        tc_store16(mine + kA + 32 + hf * 16, p1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 lm = lambda[i];
          x[4 * i] *= lm.x;
          x[4 * i + 1] *= lm.y;
          x[4 * i + 2] *= lm.z;
          x[4 * i + 3] *= lm.w;
        }
        split3_16(x, p0, p1, p2);
        tc_store16(mine + kS + hf * 16, p0);
        tc_store16(mine + kS + 32 + hf * 16, p1);
        tc_store16(mine + kS + 64 + hf * 16, p2);
      }
      arrive(y_in);
      {
        // gamma Q S (its product came before D's)
        float o[32];
        tc_load16(mine + kO + hf * 32, o);
        tc_load16(mine + kO + hf * 32 + 16, o + 16);
        uint32_t r[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 gm = gamma[i];
          r[4 * i] = __float_as_uint(gm.x * o[4 * i]);
          r[4 * i + 1] = __float_as_uint(gm.y * o[4 * i + 1]);
          r[4 * i + 2] = __float_as_uint(gm.z * o[4 * i + 2]);
          r[4 * i + 3] = __float_as_uint(gm.w * o[4 * i + 3]);
        }
        tc_store16(mine + kO + hf * 32, r);
        tc_store16(mine + kO + hf * 32 + 16, r + 16);
      }
      arrive(o_in);
      const float whole = scal[192];
      wait(u_out, c, kErrWaitMma);
      tc_fence_after();
#pragma unroll
      for (int n = 0; n < kHalf / 16; ++n) {
        float t[16];
        tc_load16(mine + kX + hf * kHalf + n * 16, t);
#pragma unroll
        for (int i = 0; i < 16; ++i) st[n * 16 + i] = fmaf(whole, st[n * 16 + i], t[i]);
      }
      if (c + 1 < chunks) {
        put_s();
        arrive(s_in);
      }
      if (lane == 0) mbar_arrive(&empty[c & 1]);
    }
    if (chunks > 0) put_o(chunks - 1);
    if (a.state_out != nullptr) {
#pragma unroll
      for (int i = 0; i < kHalf; ++i)
        a.state_out[head_state + static_cast<long long>(hf * kHalf + i) * VD] = st[i];
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kHeadWarps) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

}  // namespace gnorm
