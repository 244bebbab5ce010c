// delta_cols.cuh -- the gated delta rule's forward, 32 columns of a head of K = 128 per CTA, on
// tcgen05 (formulas and notation: delta_common.cuh).
//
// Between the strips of delta_scan.cuh, of which one has an SM to itself, and a whole head per CTA
// (delta_head.cuh): as many CTAs as fit the SMs side by side when heads are fewer.  Tokens, or rows
// of the state, are an instruction's rows, and its columns the 32 of V once for every BF16 part of
// the right operand, which lies in shared memory with its parts side by side:
//
//   1  [K; Q] S           X = V - gamma K S                  S: 128 x (3 x 32)
//   2  N (beta X)         Y = beta (X - N beta X)            each part of N into sums of its own
//   3  K^T (lambda Y)     S' = e^{G_C} S + K^T lambda Y
//   4  P Y                O = scale (gamma Q S + P Y)        while the next chunk's X is made
//
// A thread has a row and eight columns: of the state, in FP32 registers for the whole sequence,
// and of a token, k's in half of the warps and q's in the others.  One warp issues what is on the
// way from state to state, one the smaller parts of N and P, one copies.
//
// A chunk takes about 4900 cycles, two strips on an SM 5700 (32 heads of 16384 tokens 661 us
// against 785, without prep): the instructions 1500, the rest the rows' steps between them, whose
// stores share shared memory's bandwidth (320 KB a chunk, 2500 cycles) with the instructions and
// the copies.  Eight columns a thread or sixteen take the same time; of 16 columns a CTA, 3900
// cycles against 3400 of a strip.
#pragma once

#include <type_traits>

#include "delta_common.cuh"
#include "tcgen05.cuh"

namespace gnorm {

struct ColsSmem {
  static constexpr int KD = 128, VT = 32;
  // a stage: [k][q] of each 64 columns of K, N (three parts) and P (two), v, scalars
  static constexpr int kTri = KD / 64 * 2 * kTileBytes;
  static constexpr int kV = kTri + 5 * kTriGrid;
  static constexpr int kScal = kV + kChunk * VT * 2;
  static constexpr int kStage = kScal + 1024;
  // right operands, tiles of 64 columns: two hold three parts
  static constexpr int kS = 2 * kStage;                         // the state
  static constexpr int kX = kS + 2 * (KD / 64) * kTileBytes;    // beta X, then lambda Y
  static constexpr int kY = kX + 2 * kTileBytes;                // Y, two parts
  static constexpr int kBars = kY + kTileBytes;
  static constexpr int kBytes = kBars + 128 + 1024;             // 1024: alignment
  static constexpr int kRowWarps = VT / 2;
  // beside them the copies, a warp that only fills up (so that the next two are on schedulers
  // without token rows), two that issue products
  static constexpr int kThreads = (kRowWarps + 4) * 32;
};

__global__ void __launch_bounds__(ColsSmem::kThreads, 1)
    delta_cols_fwd_kernel(const __grid_constant__ DeltaArgs a, const __grid_constant__ DeltaMaps maps) {
  using L = ColsSmem;
  constexpr int KD = L::KD, VT = L::VT, kRowWarps = L::kRowWarps, kStateTile = KD / 64 * kTileBytes;
  // tensor memory columns
  constexpr uint32_t kKS = 0;                                        // [K; Q] S, by part of S
  constexpr uint32_t kD0 = kKS + 3 * VT, kD1 = kD0 + 3 * VT, kD2 = kD1 + 2 * VT;  // N0, N1, N2 beta X
  constexpr uint32_t kU = kD2 + VT;                                  // K^T lambda Y
  constexpr uint32_t kO0 = kU + 3 * VT, kO1 = kO0 + 2 * VT;          // P0, P1 Y
  static_assert(kO1 + VT <= 512, "tensor memory");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t *full = bars, *empty = bars + 2, *cleared = bars + 4, *s_in = bars + 5, *x_out = bars + 6,
           *a_in = bars + 7, *d_out = bars + 8, *y_in = bars + 9, *o_in = bars + 10, *u_out = bars + 11,
           *o_out = bars + 12;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 13);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int v0 = blockIdx.x * VT, h = blockIdx.y;
  const int hk = h / (a.Hv / a.Hk);
  if (warp == kRowWarps + 2) tmem_alloc(tslot, 512);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 2);
      mbar_init(&empty[i], 2 + kRowWarps);
    }
    for (uint64_t* b : {cleared, x_out, u_out, o_out}) mbar_init(b, 1);
    mbar_init(d_out, 2);
    for (uint64_t* b : {s_in, o_in}) mbar_init(b, kRowWarps);
    for (uint64_t* b : {a_in, y_in}) mbar_init(b, kRowWarps / 2);
    fence_barrier_init();
  }
  // N and P above the diagonal, where no copy arrives
  for (int i = tid; i < 2 * 5 * kTriGrid / 16; i += L::kThreads) {
    uint8_t* p = smem + (i >= 5 * kTriGrid / 16 ? L::kStage - 5 * kTriGrid : 0) + L::kTri + i * 16;
    *reinterpret_cast<uint4*>(p) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_smem_to_async();
  const int b = seq_by_length(a.seq, blockIdx.z, lane);
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

  if (warp == kRowWarps) {
    // ---- copies
    // a lane's pieces of a part: rows of matrices 2 p and 2 p + 1 are one run in the workspace
    uint32_t to[10];
    {
      int n = 0;
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int u = 0; u <= p; ++u) {
          const int i = u * 32 + lane, second = i >= 16 * (p + 1) ? 1 : 0;
          to[n++] = static_cast<uint32_t>((2 * p + second) * 1024 + (i - second * 16 * (p + 1)) * 16);
        }
    }
    for (int c = 0; c < chunks; ++c) {
      uint8_t* st = smem + (c & 1) * L::kStage;
      uint64_t* bar = &full[c & 1];
      if (c >= 2) wait(&empty[c & 1], static_cast<uint32_t>((c >> 1) - 1), kErrWaitEmpty);
      const int t0 = static_cast<int>(start + static_cast<long long>(c) * kChunk);
      const uint8_t* prep = a.prep + ((base + c) * a.Hv + h) * kPrepBytes;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, L::kTri + kChunk * VT * 2 + 784);
#pragma unroll
        for (int kt = 0; kt < KD / 64; ++kt) {
          tma_load_2d(st + kt * 2 * kTileBytes, &maps.k, hk * KD + kt * 64, t0, bar);
          tma_load_2d(st + (kt * 2 + 1) * kTileBytes, &maps.q, hk * KD + kt * 64, t0, bar);
        }
        tma_load_2d(st + L::kV, &maps.v, h * a.V + v0, t0, bar);
        bulk_copy_g2s(st + L::kScal, prep + kPrepTri, 784, bar);
      }
      __syncwarp();
      const uint32_t tri = smem_u32(st) + L::kTri;
#pragma unroll
      for (int part = 0; part < 5; ++part)
#pragma unroll
        for (int i = 0; i < 10; ++i) cp16(tri + part * kTriGrid + to[i], prep + part * kTriBytes + (i * 32 + lane) * 16, true);
      cp_commit();
      cp_wait<0>();
      fence_smem_to_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
      if (c + 1 == chunks && last_live < kChunk) {
        wait(bar, static_cast<uint32_t>(c >> 1), kErrWaitFull);
        clear_rows<32>(st, 128, KD / 64 * 2, kTileBytes, last_live, lane);
        clear_rows<32>(st + L::kV, VT * 2, 1, 0, last_live, lane);
        fence_smem_to_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(cleared);
      }
    }
    // the last arrivals from the tensor cores come before the CTA leaves
    for (int c = chunks; c < chunks + 2; ++c)
      if (c >= 2) wait(&empty[c & 1], static_cast<uint32_t>((c >> 1) - 1), kErrWaitEmpty);
  } else if (warp == kRowWarps + 2) {
    // ---- products on the way from state to state
    constexpr uint32_t id3 = mma_desc<false, true, 3 * VT>(), idU = mma_desc<true, true, 3 * VT>();
    const bool lead = elect_one();
    const uint64_t sd = smem_desc(sbase + L::kS, kStateTile, 1024);
    const uint64_t xd = smem_desc(sbase + L::kX, kTileBytes, 1024);
    for (int c = 0; c < chunks; ++c) {
      const uint32_t sg = sbase + (c & 1) * L::kStage;
      const uint64_t kq = smem_desc(sg, 16, 1024), kt = smem_desc(sg, 2 * kTileBytes, 1024);
      const uint64_t td = smem_desc_plain(sg + L::kTri, 128, 1024);
      wait_stage(c);
      wait(s_in, c, kErrWaitMma);
      tc_fence_after();
#pragma unroll
      for (int ks = 0; ks < KD / 16; ++ks)
        tc_mma_w(lead, tmem + kKS, desc_at(kq, (ks >> 2) * 2 * kTileBytes + (ks & 3) * 32),
                 desc_at(sd, (ks >> 2) * kTileBytes + (ks & 3) * 2048), id3, ks > 0);
      if (lead) tc_commit(x_out);
      wait(a_in, c, kErrWaitMma);
      tc_fence_after();
#pragma unroll
      for (int kb = 0; kb < 4; ++kb)
        tc_mma_w(lead, tmem + kD0, desc_at(td, kb * 256), desc_at(xd, kb * 2048), id3, kb > 0);
      if (lead) tc_commit(d_out);
      wait(y_in, c, kErrWaitMma);
      tc_fence_after();
#pragma unroll
      for (int kb = 0; kb < 4; ++kb)
        tc_mma_w(lead, tmem + kU, desc_at(kt, kb * 2048), desc_at(xd, kb * 2048), idU, kb > 0);
      if (lead) {
        tc_commit(u_out);
        tc_commit(&empty[c & 1]);
      }
    }
  } else if (warp == kRowWarps + 3) {
    // ---- the smaller parts of N, and P
    constexpr uint32_t id2 = mma_desc<false, true, 2 * VT>(), id1 = mma_desc<false, true, VT>();
    const bool lead = elect_one();
    const uint64_t xd = smem_desc(sbase + L::kX, kTileBytes, 1024), yd = smem_desc(sbase + L::kY, kTileBytes, 1024);
    for (int c = 0; c < chunks; ++c) {
      const uint64_t td = smem_desc_plain(sbase + (c & 1) * L::kStage + L::kTri, 128, 1024);
      wait_stage(c);
      wait(a_in, c, kErrWaitMma);
      tc_fence_after();
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        const uint64_t x = desc_at(xd, kb * 2048);
        tc_mma_w(lead, tmem + kD1, desc_at(td, kTriGrid + kb * 256), x, id2, kb > 0);
        tc_mma_w(lead, tmem + kD2, desc_at(td, 2 * kTriGrid + kb * 256), x, id1, kb > 0);
      }
      if (lead) tc_commit(d_out);
      wait(o_in, c, kErrWaitMma);
      // while the rows of the next chunk's first product are at work, which use shared memory least
      if (c + 1 < chunks) wait(x_out, c + 1, kErrWaitMma);
      tc_fence_after();
      // rows 64..127, where Q S is; rows 0..63, not read, are the part before's
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        const uint64_t y = desc_at(yd, kb * 2048);
        tc_mma_w(lead, tmem + kO0, desc_at(td, 2 * kTriGrid + kb * 256), y, id2, kb > 0);
        tc_mma_w(lead, tmem + kO1, desc_at(td, 3 * kTriGrid + kb * 256), y, id1, kb > 0);
      }
      if (lead) {
        tc_commit(o_out);
        tc_commit(&empty[c & 1]);
      }
    }
  } else if (warp < kRowWarps) {
    // ---- rows: of tokens (0..63 k's, 64..127 q's), and of the state
    const int row = (warp & 3) * 32 + lane, tok = row & 63, hf = warp >> 2;
    const bool q_side = (warp & 2) != 0;
    const uint32_t mine = tmem + (static_cast<uint32_t>(warp & 3) << 21) + hf * 8;
    auto arrive = [&](uint64_t* bar) {  // shared-memory writes and tensor-memory reads before it are done
      fence_smem_to_async();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    // eight values of row r of a right operand, kParts parts side by side
    auto put = [&](auto parts, uint8_t* tiles, int wide, int r, const float2* x) {
      constexpr int kParts = decltype(parts)::value;
      uint32_t p[kParts][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (kParts == 3) {
          uint32_t t[3];
          split3(x[i].x, x[i].y, t);
          p[0][i] = t[0];
          p[1][i] = t[1];
          p[2][i] = t[2];
        } else {
          split2(x[i].x, x[i].y, p[0][i], p[1][i]);
        }
      }
#pragma unroll
      for (int m = 0; m < kParts; ++m) {
        const int col = m * VT + hf * 8;
        *reinterpret_cast<uint4*>(tiles + (col >> 6) * wide + tile_off(r, (col & 63) >> 3)) =
            make_uint4(p[m][0], p[m][1], p[m][2], p[m][3]);
      }
    };
    constexpr std::integral_constant<int, 3> three{};
    constexpr std::integral_constant<int, 2> two{};
    // pair i of a product's three column ranges, the smallest first
    auto pair = [](const float* t, int r, int i) { return make_float2(t[r * 8 + 2 * i], t[r * 8 + 2 * i + 1]); };
    auto sum3 = [&](const float* t, int i) { return add2(pair(t, 0, i), add2(pair(t, 1, i), pair(t, 2, i))); };
    float2 st[4];
    const long long state_at = ((static_cast<long long>(b) * a.Hv + h) * KD + row) * a.V + v0 + hf * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      st[i] = a.state_in != nullptr ? reinterpret_cast<const float2*>(a.state_in + state_at)[i]
                                                 : make_float2(0.f, 0.f);
    auto put_s = [&]() {
      put(three, smem + L::kS + (row >> 6) * kTileBytes, kStateTile, tok, st);
      arrive(s_in);
    };
    float2 out[4];  // gamma Q S
    auto put_o = [&](int c) {  // the output of chunk c
      float t[24];
      wait(o_out, c, kErrWaitMma);
      tc_fence_after();
      tc_load8x3(mine + kO0, mine + kO0 + VT, mine + kO1, t);
      const long long tk = static_cast<long long>(c) * kChunk + tok;
      if (tk < end - start) {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 o = mul2(splat2(a.scale), add2(out[i], sum3(t, i)));
          r[i] = pack_bf16x2(o.x, o.y);
        }
        *reinterpret_cast<uint4*>(a.o + (start + tk) * a.ldo + static_cast<long long>(h) * a.V + v0 + hf * 8) =
            make_uint4(r[0], r[1], r[2], r[3]);
      }
    };
    if (chunks > 0) put_s();
    for (int c = 0; c < chunks; ++c) {
      const uint8_t* stage = smem + (c & 1) * L::kStage;
      const float* scal = reinterpret_cast<const float*>(stage + L::kScal);
      wait_stage(c);
      const float beta = scal[tok], gamma = scal[64 + tok], lambda = scal[128 + tok], whole = scal[192];
      float2 x[4];
      float t[24];
      if (!q_side) bf16x8_to_pairs(*reinterpret_cast<const uint4*>(stage + L::kV + tok * (VT * 2) + hf * 16), x);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[c & 1]);
      wait(x_out, c, kErrWaitMma);
      tc_fence_after();
      tc_load8x3(mine + kKS, mine + kKS + VT, mine + kKS + 2 * VT, t);
      if (q_side) {
        if (c > 0) put_o(c - 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = mul2(splat2(gamma), sum3(t, i));
        arrive(o_in);
      } else {
        // X = V - gamma K S
        float2 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = fma2(splat2(-gamma), sum3(t, i), x[i]);
          y[i] = mul2(splat2(beta), x[i]);
        }
        put(three, smem + L::kX, kTileBytes, tok, y);
        arrive(a_in);
        wait(d_out, c, kErrWaitMma);
        tc_fence_after();
        // Y = beta (X - N beta X)
        float d[48];
        tc_load8x6(mine + kD0, mine + kD0 + VT, mine + kD0 + 2 * VT, mine + kD1, mine + kD1 + VT, mine + kD2, d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // the larger first part, then the others by their size
          const float2 lo = add2(add2(pair(d, 2, i), pair(d, 5, i)), pair(d, 4, i));
          const float2 n = add2(pair(d, 0, i), add2(add2(pair(d, 1, i), pair(d, 3, i)), lo));
          x[i] = mul2(splat2(beta), fma2(splat2(-1.f), n, x[i]));
          y[i] = mul2(splat2(lambda), x[i]);
        }
        put(three, smem + L::kX, kTileBytes, tok, y);
        arrive(y_in);
        put(two, smem + L::kY, kTileBytes, tok, x);
        arrive(o_in);
      }
      wait(u_out, c, kErrWaitMma);
      tc_fence_after();
      tc_load8x3(mine + kU, mine + kU + VT, mine + kU + 2 * VT, t);
#pragma unroll
      for (int i = 0; i < 4; ++i) st[i] = fma2(splat2(whole), st[i], sum3(t, i));
      if (c + 1 < chunks) put_s();
    }
    if (q_side && chunks > 0) put_o(chunks - 1);
    if (a.state_out != nullptr) {
#pragma unroll
      for (int i = 0; i < 4; ++i) reinterpret_cast<float2*>(a.state_out + state_at)[i] = st[i];
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kRowWarps + 2) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

}  // namespace gnorm
