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
#pragma once

#include "delta_common.cuh"

namespace gnorm {

constexpr int kGradThreads = 256;
constexpr int kMLd = 65;

template <int KD, int VD>
struct GradSmem {
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + KD / 64 * kTileBytes;
  static constexpr int kDo = kK + KD / 64 * kTileBytes;
  static constexpr int kXh = kDo + VD / 64 * kTileBytes;
  static constexpr int kXl = kXh + VD / 64 * kTileBytes;
  static constexpr int kW = kXl + VD / 64 * kTileBytes;
  // S, then D (hi and lo tiles); then Ph and Eh + Eh^T (hi and lo) and the pair terms
  static constexpr int kBig = kW + 2 * (VD / 64) * kTileBytes;
  static constexpr int kState = 2 * (VD / 64) * (KD / 64) * kTileBytes;
  static constexpr int kPairs = 4 * kTileBytes + 64 * kMLd * 4;
  static constexpr int kScal = kBig + (kState > kPairs ? kState : kPairs);
  static constexpr int kBytes = kScal + 4096;
};

template <int KD, int VD>
__global__ void __launch_bounds__(kGradThreads, 1) delta_grad_kernel(const __grid_constant__ DeltaArgs a) {
  using L = GradSmem<KD, VD>;
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kNT = KD / 16;  // 8-column tiles of a warp's half of K
  constexpr int kVT = VD / 64, kKT = KD / 64;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int mw = warp & 3, nw = warp >> 2;  // 16 tokens, half of the columns
  const long long slot = blockIdx.x;
  const int hk = blockIdx.y;
  grid_dependency_wait();
  allow_dependent_launch();
  const int b = seq_of_slot(a.seq, slot, lane);
  const long long chunk = slot - seq_base(a.seq, b);
  const long long t0 = seq_start(a.seq, b) + chunk * kChunk;
  const long long left = seq_end(a.seq, b) - t0;
  if (b == a.seq.B || chunk < 0 || left <= 0) return;
  const int live = static_cast<int>(left < kChunk ? left : kChunk);
  const uint32_t s0 = smem_u32(smem);
  double* Gs = reinterpret_cast<double*>(smem + L::kScal);          // [64]
  float* scal = reinterpret_cast<float*>(smem + L::kScal + 512);    // beta, gamma, lambda, e^{G_C}
  float* adot = scal + 256;                                         // [2][64]
  float* bsum = adot + 128;                                         // [64]
  float* dbs = bsum + 64;                                           // [64]
  float* red = dbs + 64;                                            // [8]
  const int i0 = mw * 16;
  const int ra = i0 + (lane >> 2), rb = ra + 8;

  load_rows<kGradThreads>(s0 + L::kQ, a.q + t0 * a.ldq + static_cast<long long>(hk) * KD, a.ldq, KD, live, tid);
  load_rows<kGradThreads>(s0 + L::kK, a.k + t0 * a.ldk + static_cast<long long>(hk) * KD, a.ldk, KD, live, tid);
  float dq[kNT][4], dk[kNT][4];
#pragma unroll
  for (int n = 0; n < kNT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) dq[n][e] = dk[n][e] = 0.f;

  const int group = a.Hv / a.Hk;
  for (int r = 0; r < group; ++r) {
    const int h = hk * group + r;
    const long long hs = slot * a.Hv + h;
    const float4* S4 = reinterpret_cast<const float4*>(a.s_ws + hs * KD * VD * 4);
    const float4* D4 = reinterpret_cast<const float4*>(a.d_ws + hs * KD * VD * 4);
    load_rows<kGradThreads>(s0 + L::kDo, a.dout + t0 * a.lddo + static_cast<long long>(h) * VD, a.lddo, VD, live, tid);
    load_rows<kGradThreads>(s0 + L::kXh, a.dv + t0 * a.lddv + static_cast<long long>(h) * VD, a.lddv, VD, live, tid);
    load_flat<kGradThreads>(s0 + L::kXl, a.x_ws + hs * (kVT * kTileBytes), kVT * kTileBytes, tid);
    load_flat<kGradThreads>(s0 + L::kW, a.w_ws + hs * (3 * kVT * kTileBytes), 2 * kVT * kTileBytes, tid);
    cp_commit();
    // a state in fragment order -> hi and lo tiles [v][k]
    auto state_tiles = [&](const float4* src) {
#pragma unroll 4
      for (int f = tid; f < KD * VD / 4; f += kGradThreads) {
        const float4 x = src[f];
        const int ln = f & 31, n = (f >> 5) % (KD / 8), strip = (f >> 5) / (KD / 8);
        const int v = strip * 16 + (ln >> 2);
        uint32_t off = ((v >> 6) * kKT + (n >> 3)) * kTileBytes + tile_off(v & 63, n & 7) + (ln & 3) * 4;
        uint32_t hi, lo;
        uint8_t* big = smem + L::kBig;
        split2(x.x, x.y, hi, lo);
        *reinterpret_cast<uint32_t*>(big + off) = hi;
        *reinterpret_cast<uint32_t*>(big + L::kState / 2 + off) = lo;
        off = ((v >> 6) * kKT + (n >> 3)) * kTileBytes + tile_off((v & 63) + 8, n & 7) + (ln & 3) * 4;
        split2(x.z, x.w, hi, lo);
        *reinterpret_cast<uint32_t*>(big + off) = hi;
        *reinterpret_cast<uint32_t*>(big + L::kState / 2 + off) = lo;
      }
    };
    state_tiles(S4);
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
    cp_wait<0>();
    __syncthreads();

    const float ga = scal[64 + ra], gb = scal[64 + rb];
    // ---- products with S: dO S^T and dX S^T
    {
      float acc[kNT][4], acc2[kNT][4];
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = acc2[n][e] = 0.f;
#pragma unroll
      for (int kb = 0; kb < VD / 16; ++kb) {
        const uint32_t toff = (kb >> 2) * kTileBytes;
        const int c0 = (kb & 3) * 16;
        uint32_t ao[4], xh[4], xl[4];
        ldsm4(ao, addr_a(s0 + L::kDo + toff, i0, c0, lane));
        ldsm4(xh, addr_a(s0 + L::kXh + toff, i0, c0, lane));
        ldsm4(xl, addr_a(s0 + L::kXl + toff, i0, c0, lane));
#pragma unroll
        for (int nb = 0; nb < kNT / 2; ++nb) {
          const int col = nw * (KD / 2) + nb * 16;
          const uint32_t tile = s0 + L::kBig + ((kb >> 2) * kKT + (col >> 6)) * kTileBytes;
          uint32_t bh[4], bl[4];
          ldsm4t(bh, addr_bt(tile, c0, col & 63, lane));
          ldsm4t(bl, addr_bt(tile + L::kState / 2, c0, col & 63, lane));
          mma16816(acc[2 * nb], ao, bh[0], bh[1]);
          mma16816(acc[2 * nb + 1], ao, bh[2], bh[3]);
          mma16816(acc2[2 * nb], xh, bh[0], bh[1]);
          mma16816(acc2[2 * nb + 1], xh, bh[2], bh[3]);
          mma16816(acc[2 * nb], ao, bl[0], bl[1]);
          mma16816(acc[2 * nb + 1], ao, bl[2], bl[3]);
          mma16816(acc2[2 * nb], xl, bh[0], bh[1]);
          mma16816(acc2[2 * nb + 1], xl, bh[2], bh[3]);
          mma16816(acc2[2 * nb], xh, bl[0], bl[1]);
          mma16816(acc2[2 * nb + 1], xh, bl[2], bl[3]);
        }
      }
      // scale the rows, add, and the rows' products with q and k (a_i)
      float da = 0.f, db = 0.f;
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        const int col = nw * (KD / 2) + n * 8;
        const uint32_t oa = (col >> 6) * kTileBytes + tile_off(ra, (col & 63) >> 3) + (lane & 3) * 4;
        const uint32_t ob = (col >> 6) * kTileBytes + tile_off(rb, (col & 63) >> 3) + (lane & 3) * 4;
        const uint32_t qa = *reinterpret_cast<const uint32_t*>(smem + L::kQ + oa);
        const uint32_t qb = *reinterpret_cast<const uint32_t*>(smem + L::kQ + ob);
        const uint32_t ka = *reinterpret_cast<const uint32_t*>(smem + L::kK + oa);
        const uint32_t kb2 = *reinterpret_cast<const uint32_t*>(smem + L::kK + ob);
        const float sa = a.scale * ga, sb = a.scale * gb;
        acc[n][0] *= sa;
        acc[n][1] *= sa;
        acc[n][2] *= sb;
        acc[n][3] *= sb;
        acc2[n][0] *= -ga;
        acc2[n][1] *= -ga;
        acc2[n][2] *= -gb;
        acc2[n][3] *= -gb;
        da += acc[n][0] * bf_lo(qa) + acc[n][1] * bf_hi(qa) + acc2[n][0] * bf_lo(ka) + acc2[n][1] * bf_hi(ka);
        db += acc[n][2] * bf_lo(qb) + acc[n][3] * bf_hi(qb) + acc2[n][2] * bf_lo(kb2) + acc2[n][3] * bf_hi(kb2);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dq[n][e] += acc[n][e];
          dk[n][e] += acc2[n][e];
        }
      }
      da += __shfl_xor_sync(0xffffffffu, da, 1);
      da += __shfl_xor_sync(0xffffffffu, da, 2);
      db += __shfl_xor_sync(0xffffffffu, db, 1);
      db += __shfl_xor_sync(0xffffffffu, db, 2);
      if ((lane & 3) == 0) {
        adot[nw * 64 + ra] = da;
        adot[nw * 64 + rb] = db;
      }
    }
    __syncthreads();
    // ---- D takes S's place; <S, D>
    state_tiles(D4);
    {
      float v = 0.f;
#pragma unroll 4
      for (int f = tid; f < KD * VD / 4; f += kGradThreads) {
        const float4 x = S4[f], y = D4[f];
        v += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
      if (lane == 0) red[warp] = v;
    }
    __syncthreads();
    // ---- lambda beta W D^T
    {
      float acc[kNT][4];
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
#pragma unroll
      for (int kb = 0; kb < VD / 16; ++kb) {
        const uint32_t toff = (kb >> 2) * kTileBytes;
        const int c0 = (kb & 3) * 16;
        uint32_t wh[4], wl[4];
        ldsm4(wh, addr_a(s0 + L::kW + toff, i0, c0, lane));
        ldsm4(wl, addr_a(s0 + L::kW + kVT * kTileBytes + toff, i0, c0, lane));
#pragma unroll
        for (int nb = 0; nb < kNT / 2; ++nb) {
          const int col = nw * (KD / 2) + nb * 16;
          const uint32_t tile = s0 + L::kBig + ((kb >> 2) * kKT + (col >> 6)) * kTileBytes;
          uint32_t bh[4], bl[4];
          ldsm4t(bh, addr_bt(tile, c0, col & 63, lane));
          ldsm4t(bl, addr_bt(tile + L::kState / 2, c0, col & 63, lane));
          mma16816(acc[2 * nb], wh, bh[0], bh[1]);
          mma16816(acc[2 * nb + 1], wh, bh[2], bh[3]);
          mma16816(acc[2 * nb], wl, bh[0], bh[1]);
          mma16816(acc[2 * nb + 1], wl, bh[2], bh[3]);
          mma16816(acc[2 * nb], wh, bl[0], bl[1]);
          mma16816(acc[2 * nb + 1], wh, bl[2], bl[3]);
        }
      }
      const float fa = scal[128 + ra] * scal[ra], fb = scal[128 + rb] * scal[rb];
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        dk[n][0] = fmaf(fa, acc[n][0], dk[n][0]);
        dk[n][1] = fmaf(fa, acc[n][1], dk[n][1]);
        dk[n][2] = fmaf(fb, acc[n][2], dk[n][2]);
        dk[n][3] = fmaf(fb, acc[n][3], dk[n][3]);
      }
    }
    // ---- E, F, K K^T, Q K^T: rows i0.., columns 32 nw .. +31
    float E[4][4], F[4][4], kk[4][4], qk[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) E[n][e] = F[n][e] = kk[n][e] = qk[n][e] = 0.f;
#pragma unroll
    for (int kb = 0; kb < VD / 16; ++kb) {
      const uint32_t toff = (kb >> 2) * kTileBytes;
      const int c0 = (kb & 3) * 16;
      uint32_t ao[4], xh[4], xl[4];
      ldsm4(ao, addr_a(s0 + L::kDo + toff, i0, c0, lane));
      ldsm4(xh, addr_a(s0 + L::kXh + toff, i0, c0, lane));
      ldsm4(xl, addr_a(s0 + L::kXl + toff, i0, c0, lane));
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        uint32_t bh[4], bl[4];
        ldsm4(bh, addr_b(s0 + L::kW + toff, nw * 32 + nb * 16, c0, lane));
        ldsm4(bl, addr_b(s0 + L::kW + kVT * kTileBytes + toff, nw * 32 + nb * 16, c0, lane));
        mma16816(F[2 * nb], ao, bh[0], bh[1]);
        mma16816(F[2 * nb + 1], ao, bh[2], bh[3]);
        mma16816(E[2 * nb], xh, bh[0], bh[1]);
        mma16816(E[2 * nb + 1], xh, bh[2], bh[3]);
        mma16816(F[2 * nb], ao, bl[0], bl[1]);
        mma16816(F[2 * nb + 1], ao, bl[2], bl[3]);
        mma16816(E[2 * nb], xl, bh[0], bh[1]);
        mma16816(E[2 * nb + 1], xl, bh[2], bh[3]);
        mma16816(E[2 * nb], xh, bl[0], bl[1]);
        mma16816(E[2 * nb + 1], xh, bl[2], bl[3]);
      }
    }
#pragma unroll
    for (int kb = 0; kb < KD / 16; ++kb) {
      const uint32_t toff = (kb >> 2) * kTileBytes;
      const int c0 = (kb & 3) * 16;
      uint32_t ak[4], aq[4];
      ldsm4(ak, addr_a(s0 + L::kK + toff, i0, c0, lane));
      ldsm4(aq, addr_a(s0 + L::kQ + toff, i0, c0, lane));
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        uint32_t bk[4];
        ldsm4(bk, addr_b(s0 + L::kK + toff, nw * 32 + nb * 16, c0, lane));
        mma16816(kk[2 * nb], ak, bk[0], bk[1]);
        mma16816(kk[2 * nb + 1], ak, bk[2], bk[3]);
        mma16816(qk[2 * nb], aq, bk[0], bk[1]);
        mma16816(qk[2 * nb + 1], aq, bk[2], bk[3]);
      }
    }
    __syncthreads();  // D has been read: its place takes the pair tiles
    uint8_t* ph = smem + L::kBig;  // Ph hi, lo, Eh + Eh^T hi, lo
    float* M = reinterpret_cast<float*>(ph + 4 * kTileBytes);
    {
      const double Ga = Gs[ra], Gb = Gs[rb];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int c = nw * 32 + n * 8 + 2 * (lane & 3);
        float p[4], x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = e < 2 ? ra : rb, j = c + (e & 1);
          const double G = e < 2 ? Ga : Gb;
          const float d = j <= i ? expf(static_cast<float>(G - Gs[j])) * scal[j] : 0.f;
          p[e] = j <= i ? a.scale * F[n][e] * d : 0.f;
          x[e] = j < i ? E[n][e] * d : 0.f;
          M[i * kMLd + j] = j < i ? p[e] * qk[n][e] - x[e] * kk[n][e] : 0.f;
        }
        uint32_t hi, lo;
        const uint32_t oa = tile_off(ra, c >> 3) + (c & 7) * 2, ob = tile_off(rb, c >> 3) + (c & 7) * 2;
        split2(p[0], p[1], hi, lo);
        *reinterpret_cast<uint32_t*>(ph + oa) = hi;
        *reinterpret_cast<uint32_t*>(ph + kTileBytes + oa) = lo;
        split2(p[2], p[3], hi, lo);
        *reinterpret_cast<uint32_t*>(ph + ob) = hi;
        *reinterpret_cast<uint32_t*>(ph + kTileBytes + ob) = lo;
        // Eh below the diagonal and its mirror above; each place is written once
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = e < 2 ? ra : rb, j = c + (e & 1);
          if (j <= i) {
            const __nv_bfloat16 xh = __float2bfloat16_rn(x[e]);
            const __nv_bfloat16 xl = __float2bfloat16_rn(x[e] - __bfloat162float(xh));
            const uint32_t oij = tile_off(i, j >> 3) + (j & 7) * 2, oji = tile_off(j, i >> 3) + (i & 7) * 2;
            *reinterpret_cast<__nv_bfloat16*>(ph + 2 * kTileBytes + oij) = xh;
            *reinterpret_cast<__nv_bfloat16*>(ph + 3 * kTileBytes + oij) = xl;
            if (j < i) {
              *reinterpret_cast<__nv_bfloat16*>(ph + 2 * kTileBytes + oji) = xh;
              *reinterpret_cast<__nv_bfloat16*>(ph + 3 * kTileBytes + oji) = xl;
            }
          }
        }
      }
    }
    __syncthreads();
    // ---- dQ += Ph K;  dK += Ph^T Q - (Eh + Eh^T) K
    {
      float neg[kNT][4];
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) neg[n][e] = 0.f;
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        uint32_t ph4[4], pl4[4], th[4], tl[4], eh[4], el[4];
        const uint32_t P = s0 + L::kBig;
        ldsm4(ph4, addr_a(P, i0, kb * 16, lane));
        ldsm4(pl4, addr_a(P + kTileBytes, i0, kb * 16, lane));
        ldsm4t(th, addr_at(P, kb * 16, i0, lane));
        ldsm4t(tl, addr_at(P + kTileBytes, kb * 16, i0, lane));
        ldsm4(eh, addr_a(P + 2 * kTileBytes, i0, kb * 16, lane));
        ldsm4(el, addr_a(P + 3 * kTileBytes, i0, kb * 16, lane));
#pragma unroll
        for (int nb = 0; nb < kNT / 2; ++nb) {
          const int col = nw * (KD / 2) + nb * 16;
          uint32_t bk[4], bq[4];
          ldsm4t(bk, addr_bt(s0 + L::kK + (col >> 6) * kTileBytes, kb * 16, col & 63, lane));
          ldsm4t(bq, addr_bt(s0 + L::kQ + (col >> 6) * kTileBytes, kb * 16, col & 63, lane));
          if (kb <= mw) {
            mma16816(dq[2 * nb], ph4, bk[0], bk[1]);
            mma16816(dq[2 * nb + 1], ph4, bk[2], bk[3]);
            mma16816(dq[2 * nb], pl4, bk[0], bk[1]);
            mma16816(dq[2 * nb + 1], pl4, bk[2], bk[3]);
          }
          if (kb >= mw) {
            mma16816(dk[2 * nb], th, bq[0], bq[1]);
            mma16816(dk[2 * nb + 1], th, bq[2], bq[3]);
            mma16816(dk[2 * nb], tl, bq[0], bq[1]);
            mma16816(dk[2 * nb + 1], tl, bq[2], bq[3]);
          }
          mma16816(neg[2 * nb], eh, bk[0], bk[1]);
          mma16816(neg[2 * nb + 1], eh, bk[2], bk[3]);
          mma16816(neg[2 * nb], el, bk[0], bk[1]);
          mma16816(neg[2 * nb + 1], el, bk[2], bk[3]);
        }
      }
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) dk[n][e] -= neg[n][e];
    }
    // ---- dg and dbeta.  M's rows become their running sums over j < t, then column t is
    // summed over i >= t.
    if (tid < 64) {
      float* row = M + tid * kMLd;
      float run = 0.f;
#pragma unroll 8
      for (int j = 0; j < 64; ++j) {
        const float m = row[j];
        row[j] = run;
        run += m;
      }
    }
    __syncthreads();
    if (tid < 64) {
      float v = 0.f, pa = 0.f, pb = 0.f, sd = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sd += red[i];
#pragma unroll 8
      for (int i = 0; i < 64; ++i) {
        v += i >= tid ? M[i * kMLd + tid] : 0.f;
        pa += i >= tid ? adot[i] + adot[64 + i] : 0.f;
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
    __syncthreads();
  }
#pragma unroll
  for (int n = 0; n < kNT; ++n) {
    const long long col = static_cast<long long>(hk) * KD + nw * (KD / 2) + n * 8 + 2 * (lane & 3);
    if (ra < live) {
      *reinterpret_cast<uint32_t*>(a.dq + (t0 + ra) * a.lddq + col) = pack_bf16x2(dq[n][0], dq[n][1]);
      *reinterpret_cast<uint32_t*>(a.dk + (t0 + ra) * a.lddk + col) = pack_bf16x2(dk[n][0], dk[n][1]);
    }
    if (rb < live) {
      *reinterpret_cast<uint32_t*>(a.dq + (t0 + rb) * a.lddq + col) = pack_bf16x2(dq[n][2], dq[n][3]);
      *reinterpret_cast<uint32_t*>(a.dk + (t0 + rb) * a.lddk + col) = pack_bf16x2(dk[n][2], dk[n][3]);
    }
  }
}

}  // namespace gnorm
