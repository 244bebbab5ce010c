// delta_grad.cuh -- gradients of q, k, g and beta of the gated delta rule, all chunks at once
// (formulas and notation: delta_common.cuh).
//
// With the states S before and the gradients D after every chunk, W and dX from the scans:
//
//   F = dO W^T    E = dX W^T    Ph_ij = scale F_ij beta_j D_ij (j <= i)    Eh_ij = E_ij beta_j D_ij (j < i)
//   dQ = scale gamma dO S^T + Ph K
//   dK = -gamma dX S^T + lambda beta W D^T + Ph^T Q - (Eh + Eh^T) K
//
// dg_t collects every term whose decay spans t, and only those: no pair of large terms
// cancels, so heads that forget quickly keep their precision (the shorter form
// sum_{i>=t} (o_i.do_i - v_i.dv_i) + <S', D> loses it there: 2e-5 against 3e-6 in emulation):
//
//   dg_t = e^{G_C} <S, D> + sum_{i>=t} a_i + sum_{j<t} b_j + sum_{i>=t>j} (Ph_ij q_i.k_j - Eh_ij k_i.k_j)
//   a_i = scale gamma_i (q_i S).dO_i - gamma_i (k_i S).dX_i      b_j = lambda_j beta_j (k_j D).W_j
//
// One CTA per (chunk, key head) goes through the value heads of the group and adds their dQ
// and dK in registers, so the sum over shared heads has a fixed order.
//
// Everything here is products of 64-token tiles, done by tcgen05.  An instruction has 128
// rows; the 64 of a query-side product and the 64 of the key-side product with the same right
// operand are one: [dO; dX] S^T, [dO; dX] W^T, [Q; K] K^T, [Ph; -Eh] K.  Rows 0..63 of every
// accumulator belong to dQ, rows 64..127 to dK, and where only the key side has a product
// (W D^T, the transposed Ph and Eh, the second parts of dX and W) the upper rows multiply
// whatever tile lies before it and are not read.  A thread owns one row and half of the columns.
// Operands that are not exact in BF16 are in two parts here: dq and dk are BF16.
#pragma once

#include "delta_common.cuh"
#include "tcgen05.cuh"

namespace gnorm {

constexpr int kGradThreads = 256;
constexpr int kMLd = 65;
constexpr unsigned kErrWaitMma = 8u;  // a wait for the tensor cores ran out

template <int KD, int VD>
struct GradSmem {
  // [q][k] of each 64 columns of K, then [do][dX hi][dX lo][W hi][W lo] of each 64 columns of V
  static constexpr int kQK = 0;
  static constexpr int kA = kQK + KD / 64 * 2 * kTileBytes;
  // S, then D (hi and lo tiles); then Ph, -Eh (hi, then lo) and the pair terms' running sums
  static constexpr int kBig = kA + VD / 64 * 5 * kTileBytes;
  static constexpr int kState = 2 * (VD / 64) * (KD / 64) * kTileBytes;
  static constexpr int kPairs = 4 * kTileBytes + 128 * kMLd * 4;
  static constexpr int kScal = kBig + (kState > kPairs ? kState : kPairs);
  static constexpr int kBytes = kScal + 5120 + 1024;  // 1024: the tiles' alignment
};

template <int KD, int VD>
__global__ void __launch_bounds__(kGradThreads, 1) delta_grad_kernel(const __grid_constant__ DeltaArgs a) {
  using L = GradSmem<KD, VD>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  constexpr int kVT = VD / 64, kKT = KD / 64;
  constexpr int kHalf = KD / 2;                         // columns of K per thread
  constexpr int kF4 = KD * VD / 4 / kGradThreads;       // float4 of a state per thread
  // tensor memory columns (the second use of a range follows the reads of the first)
  constexpr uint32_t kD1 = 0, kD5 = 0;                  // [dO; dX] S^T     | [-; Ph^T] Q - [-; Eh^T] K
  constexpr uint32_t kD3 = 128, kD2b = 128;             // [-; dX lo] W^T   | [-; W] D^T
  constexpr uint32_t kD4 = 256, kD1b = 256;             // [-; dX lo] S^T   | [Ph; -Eh] K
  constexpr uint32_t kD2 = 384, kKK = 448;              // [dO; dX] W^T,  [Q; K] K^T
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = (warp & 3) * 32 + lane;               // 0..63 dQ, 64..127 dK
  const int half = warp >> 2;
  const bool key_side = (warp & 2) != 0;
  const int tok = row & 63;
  const long long slot = blockIdx.x;
  const int hk = blockIdx.y;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t s0 = smem_u32(smem);
  double* Gs = reinterpret_cast<double*>(smem + L::kScal);          // [64]
  float* scal = reinterpret_cast<float*>(smem + L::kScal + 512);    // beta, gamma, lambda, e^{G_C}
  float* adot = scal + 256;                                         // [4][64]
  float* bsum = adot + 256;                                         // [64]
  float* dbs = bsum + 64;                                           // [64]
  float* vpart = dbs + 64;                                          // [4][64]
  float* red = vpart + 256;                                         // [8]
  float* rowsum = red + 8;                                          // [128]
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kScal + 5096);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + L::kScal + 5104);

  grid_dependency_wait();
  allow_dependent_launch();
  const int b = seq_of_slot(a.seq, slot, lane);
  const long long chunk = slot - seq_base(a.seq, b);
  const long long t0 = seq_start(a.seq, b) + chunk * kChunk;
  const long long left = seq_end(a.seq, b) - t0;
  if (b == a.seq.B || chunk < 0 || left <= 0) return;
  const int live = static_cast<int>(left < kChunk ? left : kChunk);
  if (warp == 0) tmem_alloc(tslot, 512);
  if (tid == 32) {
    mbar_init(bar, 1);
    fence_barrier_init();
  }
#pragma unroll
  for (int kt = 0; kt < kKT; ++kt) {
    const long long col = static_cast<long long>(hk) * KD + kt * 64;
    load_rows<kGradThreads>(s0 + L::kQK + kt * 2 * kTileBytes, a.q + t0 * a.ldq + col, a.ldq, 64, live, tid);
    load_rows<kGradThreads>(s0 + L::kQK + (kt * 2 + 1) * kTileBytes, a.k + t0 * a.ldk + col, a.ldk, 64, live, tid);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t mine = tmem + (static_cast<uint32_t>(warp & 3) << 21);  // this warp's lanes
  const uint32_t aA = s0 + L::kA, big = s0 + L::kBig;
  uint32_t phase = 0;
  bool alive = true;
  auto wait_mma = [&]() {
    if (alive) alive = mbar_wait(bar, phase, a.err, kErrWaitMma);
    phase ^= 1u;
    tc_fence_after();
  };

  float acc[kHalf];  // dQ or dK of this row
#pragma unroll
  for (int i = 0; i < kHalf; ++i) acc[i] = 0.f;

  const int group = a.Hv / a.Hk;
  for (int r = 0; r < group; ++r) {
    const int h = hk * group + r;
    const long long hs = slot * a.Hv + h;
    const float4* S4 = reinterpret_cast<const float4*>(a.s_ws + hs * KD * VD * 4);
    const float4* D4 = reinterpret_cast<const float4*>(a.d_ws + hs * KD * VD * 4);
    float4 sv[kF4];
#pragma unroll
    for (int i = 0; i < kF4; ++i) sv[i] = S4[tid + i * kGradThreads];
#pragma unroll
    for (int vt = 0; vt < kVT; ++vt) {
      const uint32_t at = aA + vt * 5 * kTileBytes;
      const long long col = static_cast<long long>(h) * VD + vt * 64;
      load_rows<kGradThreads>(at, a.dout + t0 * a.lddo + col, a.lddo, 64, live, tid);
      load_rows<kGradThreads>(at + kTileBytes, a.dv + t0 * a.lddv + col, a.lddv, 64, live, tid);
      load_flat<kGradThreads>(at + 2 * kTileBytes, a.x_ws + (hs * kVT + vt) * kTileBytes, kTileBytes, tid);
      const uint8_t* w = a.w_ws + (hs * 3 * kVT + vt) * kTileBytes;
      load_flat<kGradThreads>(at + 3 * kTileBytes, w, kTileBytes, tid);
      load_flat<kGradThreads>(at + 4 * kTileBytes, w + kVT * kTileBytes, kTileBytes, tid);
    }
    cp_commit();
    if (warp == 0) {
      const int ta = 2 * lane, tb = ta + 1;
      const float ga = ta < live ? clamp_decay(a.g[(t0 + ta) * a.ldg + h]) : 0.f;
      const float gb = tb < live ? clamp_decay(a.g[(t0 + tb) * a.ldg + h]) : 0.f;
      double s = static_cast<double>(ga) + static_cast<double>(gb);
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += o;
      }
      Gs[ta] = s - static_cast<double>(gb);
      Gs[tb] = s;
    } else {
      const float* ps = reinterpret_cast<const float*>(a.prep + hs * kPrepBytes + kPrepTri);
      for (int i = tid - 32; i < 193; i += kGradThreads - 32) scal[i] = ps[i];
      // the strips' shares of b and dbeta, in strip order
      if (tid >= 128) {
        const int which = (tid - 128) >> 6, t = tid & 63;
        const float* p = a.dots + hs * (VD / 16) * 128 + which * 64 + t;
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < VD / 16; ++i) v += p[i * 128];
        (which == 0 ? bsum : dbs)[t] = v;
      }
    }
    // a state in fragment order -> hi and lo tiles [v][k]
    auto state_tiles = [&](const float4* x) {
#pragma unroll
      for (int i = 0; i < kF4; ++i) {
        const int f = tid + i * kGradThreads;
        const int ln = f & 31, n = (f >> 5) % (KD / 8), strip = (f >> 5) / (KD / 8);
        const int v = strip * 16 + (ln >> 2);
        uint8_t* dst = smem + L::kBig + ((v >> 6) * kKT + (n >> 3)) * kTileBytes + (ln & 3) * 4;
        uint32_t hi, lo;
        split2(x[i].x, x[i].y, hi, lo);
        *reinterpret_cast<uint32_t*>(dst + tile_off(v & 63, n & 7)) = hi;
        *reinterpret_cast<uint32_t*>(dst + L::kState / 2 + tile_off(v & 63, n & 7)) = lo;
        split2(x[i].z, x[i].w, hi, lo);
        *reinterpret_cast<uint32_t*>(dst + tile_off((v & 63) + 8, n & 7)) = hi;
        *reinterpret_cast<uint32_t*>(dst + L::kState / 2 + tile_off((v & 63) + 8, n & 7)) = lo;
      }
    };
    state_tiles(sv);
    cp_wait<0>();
    fence_smem_to_async();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      constexpr uint32_t idS = mma_desc<false, true, KD>(), idW = mma_desc<false, false, 64>();
#pragma unroll
      for (int ks = 0; ks < VD / 16; ++ks) {
        const uint32_t at = aA + (ks >> 2) * 5 * kTileBytes + (ks & 3) * 32;
        const uint64_t a0 = smem_desc(at, 16, 1024), a1 = smem_desc(at + kTileBytes, 16, 1024);
        const uint32_t st = big + (ks >> 2) * kKT * kTileBytes + (ks & 3) * 2048;
        const uint64_t sh = smem_desc(st, kTileBytes, 1024);
        const uint64_t sl = smem_desc(st + L::kState / 2, kTileBytes, 1024);
        const uint64_t wh = smem_desc(at + 3 * kTileBytes, 16, 1024);
        const uint64_t wl = smem_desc(at + 4 * kTileBytes, 16, 1024);
        tc_mma(tmem + kD1, a0, sh, idS, ks > 0);
        tc_mma(tmem + kD1, a0, sl, idS, true);
        tc_mma(tmem + kD1b, a1, sh, idS, ks > 0);
        tc_mma(tmem + kD2, a0, wh, idW, ks > 0);
        tc_mma(tmem + kD2, a0, wl, idW, true);
        tc_mma(tmem + kD2b, a1, wh, idW, ks > 0);
      }
      if (r == 0) {
#pragma unroll
        for (int ks = 0; ks < KD / 16; ++ks) {
          const uint32_t at = s0 + L::kQK + (ks >> 2) * 2 * kTileBytes + (ks & 3) * 32;
          tc_mma(tmem + kKK, smem_desc(at, 16, 1024), smem_desc(at + kTileBytes, 16, 1024), idW, ks > 0);
        }
      }
      tc_commit(bar);
    }
    // meanwhile D, and <S, D>
    float4 dv4[kF4];
#pragma unroll
    for (int i = 0; i < kF4; ++i) dv4[i] = D4[tid + i * kGradThreads];
    {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < kF4; ++i)
        v += sv[i].x * dv4[i].x + sv[i].y * dv4[i].y + sv[i].z * dv4[i].z + sv[i].w * dv4[i].w;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
      if (lane == 0) red[warp] = v;
    }
    wait_mma();
    // ---- D takes S's place
    state_tiles(dv4);
    // E (key side) or F, and the second part of E before its range is used again
    float ef[32];
    tc_load32(mine + kD2 + half * 32, ef);
    if (key_side) {
      float t[32];
      tc_load32(mine + kD2b + half * 32, t);
#pragma unroll
      for (int i = 0; i < 32; ++i) ef[i] += t[i];
    }
    fence_smem_to_async();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      constexpr uint32_t idS = mma_desc<false, true, KD>();
#pragma unroll
      for (int ks = 0; ks < VD / 16; ++ks) {
        const uint32_t at = aA + (ks >> 2) * 5 * kTileBytes + (ks & 3) * 32;
        const uint32_t st = big + (ks >> 2) * kKT * kTileBytes + (ks & 3) * 2048;
        const uint64_t wh = smem_desc(at + 2 * kTileBytes, 16, 1024);  // rows 64..127: W hi
        const uint64_t wl = smem_desc(at + 3 * kTileBytes, 16, 1024);
        const uint64_t dh = smem_desc(st, kTileBytes, 1024);
        const uint64_t dl = smem_desc(st + L::kState / 2, kTileBytes, 1024);
        tc_mma(tmem + kD3, wh, dh, idS, ks > 0);
        tc_mma(tmem + kD3, wh, dl, idS, true);
        tc_mma(tmem + kD3, wl, dh, idS, true);
      }
      tc_commit(bar);
    }
    // ---- meanwhile the products with S: scale the row, add, and its product with q or k (a_i)
    {
      const float f = key_side ? -scal[64 + tok] : a.scale * scal[64 + tok];
      float dot = 0.f;
#pragma unroll
      for (int c = 0; c < kHalf / 32; ++c) {
        float t[32];
        tc_load32(mine + kD1 + half * kHalf + c * 32, t);
        if (key_side) {
          float u[32];
          tc_load32(mine + kD1b + half * kHalf + c * 32, u);
#pragma unroll
          for (int i = 0; i < 32; ++i) t[i] += u[i];
        }
        const int col = half * kHalf + c * 32;
        const uint8_t* src = smem + L::kQK + ((col >> 6) * 2 + (key_side ? 1 : 0)) * kTileBytes;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint4 x = *reinterpret_cast<const uint4*>(src + tile_off(tok, ((col & 63) >> 3) + p));
          float xf[8];
          bf16x8_to_f32(x, xf);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float v = f * t[p * 8 + e];
            dot = fmaf(v, xf[e], dot);
            acc[c * 32 + p * 8 + e] += v;
          }
        }
      }
      adot[(half * 2 + (key_side ? 1 : 0)) * 64 + tok] = dot;
    }
    // ---- the pair terms: this row's 32 columns of Ph or -Eh, and of their products with q.k or k.k
    uint32_t hi[16], lo[16];
    {
      float kk[32];
      tc_load32(mine + kKK + half * 32, kk);
      const double G = Gs[tok];
      float run = 0.f;
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        float p[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = half * 32 + i + e;
          float v = 0.f;
          if (key_side ? j < tok : j <= tok) {
            const float d = expf(static_cast<float>(G - Gs[j])) * scal[j];
            v = key_side ? -ef[i + e] * d : a.scale * ef[i + e] * d;
          }
          p[e] = v;
          // running sums over the columns before, in the place of the terms
          const float m = j < tok ? v * kk[i + e] : 0.f;
          ef[i + e] = run;
          run += m;
        }
        split2(p[0], p[1], hi[i / 2], lo[i / 2]);
      }
      if (half == 0) rowsum[row] = run;
    }
    wait_mma();  // W D^T is done, its tiles' place is free
    {
      uint8_t* dst = smem + L::kBig + (key_side ? kTileBytes : 0);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t off = tile_off(tok, half * 4 + p);
        *reinterpret_cast<uint4*>(dst + off) = make_uint4(hi[4 * p], hi[4 * p + 1], hi[4 * p + 2], hi[4 * p + 3]);
        *reinterpret_cast<uint4*>(dst + 2 * kTileBytes + off) =
            make_uint4(lo[4 * p], lo[4 * p + 1], lo[4 * p + 2], lo[4 * p + 3]);
      }
      float* M = reinterpret_cast<float*>(smem + L::kBig + 4 * kTileBytes) + row * kMLd + half * 32;
#pragma unroll
      for (int i = 0; i < 32; ++i) M[i] = ef[i];
    }
    fence_smem_to_async();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      constexpr uint32_t idP = mma_desc<false, true, KD>(), idT = mma_desc<true, true, KD>();
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const uint64_t q = smem_desc(s0 + L::kQK + ks * 2048, 2 * kTileBytes, 1024);
        const uint64_t k = smem_desc(s0 + L::kQK + kTileBytes + ks * 2048, 2 * kTileBytes, 1024);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const uint32_t ph = big + part * 2 * kTileBytes;
          tc_mma(tmem + kD4, smem_desc(ph + ks * 32, 16, 1024), k, idP, ks + part > 0);
          // transposed, as rows 64..127: the tile before is rows 0..63
          tc_mma(tmem + kD5, smem_desc(ph - kTileBytes + ks * 2048, kTileBytes, 1024), q, idT, ks + part > 0);
          tc_mma(tmem + kD5, smem_desc(ph + ks * 2048, kTileBytes, 1024), k, idT, true);
        }
      }
      tc_commit(bar);
    }
    // ---- meanwhile W D^T, and the sums of dg over i >= t
    if (key_side) {
      const float f = scal[128 + tok] * scal[tok];
#pragma unroll
      for (int c = 0; c < kHalf / 32; ++c) {
        float t[32];
        tc_load32(mine + kD3 + half * kHalf + c * 32, t);
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[c * 32 + i] = fmaf(f, t[i], acc[c * 32 + i]);
      }
    }
    {
      // column t of the running sums: rows i >= t of 32 rows of Ph's or Eh's terms
      const int t = tid & 63, part = tid >> 6;
      const int i0 = (part & 1) * 32, r0 = (part >> 1) * 64 + i0;
      const float* M = reinterpret_cast<const float*>(smem + L::kBig + 4 * kTileBytes) + r0 * kMLd + t;
      float v = 0.f;
#pragma unroll 8
      for (int i = 0; i < 32; ++i) {
        float x = M[i * kMLd];
        if (t >= 32) x += rowsum[r0 + i];  // the second half's sums start at the first half's
        v += i0 + i >= t ? x : 0.f;
      }
      vpart[part * 64 + t] = v;
    }
    __syncthreads();
    if (tid < 64) {
      float v = vpart[tid] + vpart[64 + tid] + vpart[128 + tid] + vpart[192 + tid];
      float pa = 0.f, pb = 0.f, sd = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sd += red[i];
#pragma unroll 8
      for (int i = 0; i < 64; ++i) {
        pa += i >= tid ? (adot[i] + adot[64 + i]) + (adot[128 + i] + adot[192 + i]) : 0.f;
        pb += i < tid ? bsum[i] : 0.f;
      }
      if (tid < live) {
        const long long t = t0 + tid;
        a.dg[t * a.lddg + h] = scal[192] * sd + v + pa + pb;
        const float db = dbs[tid];
        if (a.beta_fp32)
          reinterpret_cast<float*>(a.dbeta)[t * a.lddbeta + h] = db;
        else
          reinterpret_cast<__nv_bfloat16*>(a.dbeta)[t * a.lddbeta + h] = __float2bfloat16_rn(db);
      }
    }
    wait_mma();
#pragma unroll
    for (int c = 0; c < kHalf / 32; ++c) {
      float t[32];
      tc_load32(mine + kD4 + half * kHalf + c * 32, t);
#pragma unroll
      for (int i = 0; i < 32; ++i) acc[c * 32 + i] += t[i];
      if (key_side) {
        tc_load32(mine + kD5 + half * kHalf + c * 32, t);
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[c * 32 + i] += t[i];
      }
    }
    tc_fence_before();
    __syncthreads();
  }
  if (tok < live) {
    uint16_t* dst = key_side ? a.dk + (t0 + tok) * a.lddk : a.dq + (t0 + tok) * a.lddq;
    dst += static_cast<long long>(hk) * KD + half * kHalf;
#pragma unroll
    for (int i = 0; i < kHalf / 8; ++i)
      *reinterpret_cast<uint4*>(dst + i * 8) = f32x8_to_bf16(acc + i * 8);
  }
  if (warp == 0) tmem_free(tmem, 512);
}

}  // namespace gnorm
