// delta_prep.cuh -- what a chunk of the gated delta rule needs apart from the state, for all
// chunks at once: N = (I + Kb diag(beta))^-1 Kb, P and the decay factors (delta_common.cuh).
//
// One CTA per (chunk, key head): K K^T and Q K^T once (BF16 operands, exact, FP32 sums), then
// for each value head of the group the decays, and N by blocks of 16, in FP32.  Bound by the
// dependent steps of the substitution, 64 if taken row by row, so only blocks of 8 on the diagonal
// are (column j of N solves n_i = Kb_ij - sum_{l<i} Kb_il beta_l n_l); the others follow as products on the tensor cores, operands in three BF16
// parts, one distance from the diagonal after another:
//
//   R = Kb_pr - sum_{r<=q<p} (Kb_pq beta) N_qr    N_pr = R - N_pp (beta R)
//
// N's parts are read where they go out, beta R passes through N_pr's place.  8192 tokens x 16
// heads: 50 us (all 64 steps 76, blocks of 16 by substitution and FP32 products 57), 65 MB
// written, four CTAs an SM in the latency of their phases.
#pragma once

#include "delta_common.cuh"

namespace gnorm {

constexpr int kPrepThreads = 128;
constexpr int kKbLd = 68;  // floats of a row of Kb in shared memory

template <int KD>
GNORM_HD constexpr int prep_tile_area() {  // the q and k tiles, then the parts that go out
  return KD / 64 * 2 * kTileBytes > kPrepTri ? KD / 64 * 2 * kTileBytes : static_cast<int>(kPrepTri);
}
template <int KD>
GNORM_HD constexpr int prep_smem() {
  return prep_tile_area<KD>() + 64 * kKbLd * 4 + 64 * 8 + 1024;  // Kb; G; scalars
}

template <int KD>
__global__ void __launch_bounds__(kPrepThreads, 4) delta_prep_kernel(const __grid_constant__ DeltaArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kTiles = KD / 64;
  constexpr int kTileArea = prep_tile_area<KD>();
  float* kb = reinterpret_cast<float*>(smem + kTileArea);
  float2* Gs = reinterpret_cast<float2*>(kb + 64 * kKbLd);
  float* scal = reinterpret_cast<float*>(Gs + 64);  // beta, gamma, lambda [64], e^{G_C}
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long slot = blockIdx.x;
  const int hk = blockIdx.y;
  grid_dependency_wait();
  allow_dependent_launch();
  const int b = seq_of_slot(a.seq, slot, lane);
  const long long chunk = slot - seq_base(a.seq, b);
  const long long t0 = seq_start(a.seq, b) + chunk * kChunk;
  const long long left = seq_end(a.seq, b) - t0;
  if (chunk < 0 || left <= 0) return;
  const int live = static_cast<int>(left < kChunk ? left : kChunk);
  if (b == a.seq.B) {  // tokens behind the last sequence
    if (hk != 0) return;
    for (int z = 0; z < a.n_zero; ++z)
      for (int r = warp; r < live; r += kPrepThreads / 32)
        for (int i = lane * 2; i < a.zero_row[z]; i += 64)
          *reinterpret_cast<uint16_t*>(a.zero_p[z] + (t0 + r) * a.zero_ld[z] + i) = 0;
    return;
  }
  // The four warps' shares of the work below differ (the lower rows have more columns); CTAs that
  // share an SM, a multiple of its number apart, give them to different schedulers.
  const int rot = static_cast<int>((static_cast<unsigned>(slot) + gridDim.x * hk) / static_cast<unsigned>(a.sms));
  const int wr = (warp + rot) & 3;
  const int group = a.Hv / a.Hk;
  // g and beta of two tokens a lane, for the warp that sums them, a head ahead
  float4 gb = make_float4(0.f, 0.f, 0.f, 0.f);
  auto load_g = [&](int h) {
    const int ta = 2 * lane, tb = ta + 1;
    gb.x = ta < live ? clamp_decay(a.g[(t0 + ta) * a.ldg + h]) : 0.f;
    gb.y = tb < live ? clamp_decay(a.g[(t0 + tb) * a.ldg + h]) : 0.f;
    gb.z = ta < live ? load_beta(a, t0 + ta, h) : 0.f;
    gb.w = tb < live ? load_beta(a, t0 + tb, h) : 0.f;
  };
  const uint32_t sq = smem_u32(smem), sk = sq + kTiles * kTileBytes;
  load_rows<kPrepThreads>(sq, a.q + t0 * a.ldq + static_cast<long long>(hk) * KD, a.ldq, KD, live, tid);
  load_rows<kPrepThreads>(sk, a.k + t0 * a.ldk + static_cast<long long>(hk) * KD, a.ldk, KD, live, tid);
  cp_commit();
  if (wr == 0) load_g(hk * group);
  cp_wait<0>();
  __syncthreads();

  // rows 16 wr .. +15 of K K^T and Q K^T, columns up to the diagonal block
  const int i0 = wr * 16;
  float kk[8][4], qk[8][4];
#pragma unroll
  for (int n = 0; n < 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) kk[n][e] = qk[n][e] = 0.f;
#pragma unroll
  for (int kb16 = 0; kb16 < KD / 16; ++kb16) {
    const uint32_t toff = (kb16 >> 2) * kTileBytes;
    const int c0 = (kb16 & 3) * 16;
    uint32_t ak[4], aq[4];
    ldsm4(ak, addr_a(sk + toff, i0, c0, lane));
    ldsm4(aq, addr_a(sq + toff, i0, c0, lane));
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
      if (nb <= wr) {
        uint32_t bk[4];
        ldsm4(bk, addr_b(sk + toff, nb * 16, c0, lane));
        mma16816(kk[2 * nb], ak, bk[0], bk[1]);
        mma16816(kk[2 * nb + 1], ak, bk[2], bk[3]);
        mma16816(qk[2 * nb], aq, bk[0], bk[1]);
        mma16816(qk[2 * nb + 1], aq, bk[2], bk[3]);
      }
    }
  }
  __syncthreads();  // the q and k tiles are free

  uint8_t* tiles = smem;  // N in three parts, P in three parts
  for (int r = 0; r < group; ++r) {
    const int h = hk * group + r;
    if (wr == 0) {
      // running sum of g in FP64: differences of far terms stay exact to FP32
      const int ta = 2 * lane, tb = ta + 1;
      const float4 cur = gb;
      if (r + 1 < group) load_g(h + 1);
      double s = static_cast<double>(cur.x) + static_cast<double>(cur.y);
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += o;
      }
      const double total = __shfl_sync(0xffffffffu, s, 31);
      const double Ga = s - static_cast<double>(cur.y);
      Gs[ta] = decay_sum(Ga);
      Gs[tb] = decay_sum(s);
      scal[ta] = cur.z;
      scal[tb] = cur.w;
      scal[64 + ta] = expf(static_cast<float>(Ga));
      scal[64 + tb] = expf(static_cast<float>(s));
      scal[128 + ta] = expf(static_cast<float>(total - Ga));
      scal[128 + tb] = expf(static_cast<float>(total - s));
      if (lane == 0) scal[192] = expf(static_cast<float>(total));
    }
    __syncthreads();
    // Kb (FP32, zero on and above the diagonal) and the P tiles
    const int ra = i0 + (lane >> 2), rb = ra + 8;
    const float2 Ga = Gs[ra], Gb = Gs[rb];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      if (n > 2 * wr + 1) break;  // above the diagonal block: nothing is read there
      const int c = n * 8 + 2 * (lane & 3);
      const float2 G0 = Gs[c], G1 = Gs[c + 1];
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      if (c <= ra) d[0] = decay_between(Ga, G0);
      if (c + 1 <= ra) d[1] = decay_between(Ga, G1);
      if (c <= rb) d[2] = decay_between(Gb, G0);
      if (c + 1 <= rb) d[3] = decay_between(Gb, G1);
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = d[e] != 0.f ? qk[n][e] * d[e] : 0.f;
      *reinterpret_cast<float2*>(kb + ra * kKbLd + c) =
          make_float2(c < ra ? kk[n][0] * d[0] : 0.f, c + 1 < ra ? kk[n][1] * d[1] : 0.f);
      *reinterpret_cast<float2*>(kb + rb * kKbLd + c) =
          make_float2(c < rb ? kk[n][2] * d[2] : 0.f, c + 1 < rb ? kk[n][3] * d[3] : 0.f);
      {
        uint32_t pa[3], pb[3];
        split3(p[0], p[1], pa);
        split3(p[2], p[3], pb);
        uint8_t* dst = tiles + 3 * kTriBytes;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          *reinterpret_cast<uint32_t*>(dst + part * kTriBytes + tri_off(ra, c)) = pa[part];
          *reinterpret_cast<uint32_t*>(dst + part * kTriBytes + tri_off(rb, c)) = pb[part];
        }
      }
    }
    __syncthreads();
    // The diagonal blocks, a warp each: its two 8 x 8 blocks by substitution, a column per lane
    // (lanes 16..31 repeat it), then the block below them by two products in FP32.
    {
      const float* beta = scal + i0;
      float* blk = kb + i0 * kKbLd + i0;
      {
        const int at = ((lane >> 3) & 1) * 8, j = lane & 7;
        float* sub = blk + at * kKbLd + at;
        float n[8], x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 c0 = *reinterpret_cast<const float4*>(sub + i * kKbLd);
          const float4 c1 = *reinterpret_cast<const float4*>(sub + i * kKbLd + 4);
          const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
          float s = i > j ? sub[i * kKbLd + j] : 0.f;
#pragma unroll
          for (int l = 0; l < i; ++l) s = fmaf(-c[l], x[l], s);
          n[i] = i > j ? s : 0.f;
          x[i] = beta[at + i] * n[i];
        }
        __syncwarp();
        if (lane < 16) {
#pragma unroll
          for (int i = 0; i < 8; ++i) sub[i * kKbLd + j] = n[i];
        }
        __syncwarp();
      }
      const int row = lane >> 2, c = 2 * (lane & 3);
      float* low = blk + (8 + row) * kKbLd;  // this row of the lower blocks
      float2 v = *reinterpret_cast<const float2*>(low + c);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float m = low[k] * beta[k];
        const float2 y = *reinterpret_cast<const float2*>(blk + k * kKbLd + c);
        v.x = fmaf(-m, y.x, v.x);
        v.y = fmaf(-m, y.y, v.y);
      }
      float* up = blk + row * kKbLd + 8 + c;  // the upper right block is free
      *reinterpret_cast<float2*>(up) = make_float2(beta[8 + row] * v.x, beta[8 + row] * v.y);
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float m = low[8 + k];
        const float2 y = *reinterpret_cast<const float2*>(blk + k * kKbLd + 8 + c);
        v.x = fmaf(-m, y.x, v.x);
        v.y = fmaf(-m, y.y, v.y);
      }
      auto put = [&](int i, int j, float2 u) {
        uint32_t parts[3];
        split3(u.x, u.y, parts);
#pragma unroll
        for (int m = 0; m < 3; ++m)
          *reinterpret_cast<uint32_t*>(tiles + m * kTriBytes + tri_off(i0 + i, i0 + j)) = parts[m];
      };
      put(row, c, *reinterpret_cast<const float2*>(blk + row * kKbLd + c));
      put(row, 8 + c, make_float2(0.f, 0.f));
      put(8 + row, c, v);
      put(8 + row, 8 + c, *reinterpret_cast<const float2*>(low + 8 + c));
    }
    __syncthreads();
    // the blocks below, one distance from the diagonal after another
    const uint32_t tri = sq;  // the parts in shared memory
    // this lane's matrix row of the 16 x 16 block (p, r): the left operand's matrices in its order
    // (rows first), the right one's and a product's own in theirs
    auto left_at = [&](int p, int r) {
      return tri + (tri_row(2 * p + ((lane >> 3) & 1)) + 2 * r + (lane >> 4)) * 128 + (lane & 7) * 16;
    };
    auto right_at = [&](int p, int r) { return left_at(p, r); };  // (transposing loads: k first)
    {
      const int row = lane >> 2, col = 2 * (lane & 3);
      for (int d = 1; d < 4; ++d) {
        // three blocks, two, one: to the warps that have fewer columns above
        const int r = d == 1 ? wr : d == 2 ? 2 - wr : -wr, p = r + d;
        if (d > 1) __syncthreads();
        if (r < 0 || p > 3) continue;
        // accumulators: two tiles of eight columns, in FP32
        float x[2][4], y[2][4];
        const float* kp = kb + (p * 16 + row) * kKbLd + col;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float2 u = *reinterpret_cast<const float2*>(kp + r * 16 + t * 8);
          const float2 v = *reinterpret_cast<const float2*>(kp + 8 * kKbLd + r * 16 + t * 8);
          x[t][0] = u.x;
          x[t][1] = u.y;
          x[t][2] = v.x;
          x[t][3] = v.y;
#pragma unroll
          for (int e = 0; e < 4; ++e) y[t][e] = 0.f;
        }
        // x -= the products of A's parts and of a block's parts, the larger and the smaller ones
        // in sums of their own
        auto product = [&](const uint32_t (*A)[4], uint32_t at) {
#pragma unroll
          for (int n = 0; n < 3; ++n) {
            uint32_t b[4];
            ldsm4t(b, at + n * kTriBytes);
#pragma unroll
            for (int m = 0; m + n < 3; ++m) {
              float(*acc)[4] = m + n == 0 ? x : y;
              mma16816(acc[0], A[m], b[0], b[1]);
              mma16816(acc[1], A[m], b[2], b[3]);
            }
          }
        };
        for (int q = r; q < p; ++q) {
          // -Kb_pq diag(beta)
          uint32_t A[3][4];
          const float2 b0 = *reinterpret_cast<const float2*>(scal + q * 16 + col);
          const float2 b1 = *reinterpret_cast<const float2*>(scal + q * 16 + 8 + col);
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // rows 0 and 8, then columns 8 on
            const float2 u = *reinterpret_cast<const float2*>(kp + (i & 1) * 8 * kKbLd + q * 16 + (i >> 1) * 8);
            const float2 be = i < 2 ? b0 : b1;
            uint32_t parts[3];
            split3(-u.x * be.x, -u.y * be.y, parts);
#pragma unroll
            for (int m = 0; m < 3; ++m) A[m][i] = parts[m];
          }
          product(A, right_at(q, r));
        }
        // R times beta into its own place, then N_pr = R - N_pp (beta R)
        auto put = [&](float f0, float f1) {
          uint32_t f[3][4];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            uint32_t u[3], v[3];
            split3(f0 * x[t][0], f0 * x[t][1], u);
            split3(f1 * x[t][2], f1 * x[t][3], v);
#pragma unroll
            for (int m = 0; m < 3; ++m) {
              f[m][2 * t] = u[m];
              f[m][2 * t + 1] = v[m];
            }
          }
          __syncwarp();
#pragma unroll
          for (int m = 0; m < 3; ++m) stsm4(left_at(p, r) + m * kTriBytes, f[m]);
          __syncwarp();
        };
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[t][e] += y[t][e];
            y[t][e] = 0.f;
          }
        put(scal[p * 16 + row], scal[p * 16 + 8 + row]);
        uint32_t A[3][4];
#pragma unroll
        for (int m = 0; m < 3; ++m) {
          ldsm4(A[m], left_at(p, p) + m * kTriBytes);
#pragma unroll
          for (int i = 0; i < 4; ++i) A[m][i] ^= 0x80008000u;
        }
        product(A, right_at(p, r));
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[t][e] += y[t][e];
        put(1.f, 1.f);
      }
    }
    __syncthreads();
    uint8_t* dst = a.prep + (slot * a.Hv + h) * kPrepBytes;
    for (int i = tid * 16; i < kPrepTri; i += kPrepThreads * 16)
      *reinterpret_cast<uint4*>(dst + i) = *reinterpret_cast<const uint4*>(tiles + i);
    for (int i = tid; i < 193; i += kPrepThreads)
      reinterpret_cast<float*>(dst + kPrepTri)[i] = scal[i];
    __syncthreads();
  }
}

}  // namespace gnorm
