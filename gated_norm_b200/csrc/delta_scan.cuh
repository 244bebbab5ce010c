// delta_scan.cuh -- the chunk-after-chunk part of the gated delta rule, forward and backward
// (formulas and notation: delta_common.cuh).
//
// A warp owns 16 of the state's V columns for the whole sequence and keeps them, transposed,
// as FP32 accumulators in registers (S^T: 16 x K).  Everything is computed transposed, so
// each intermediate is the left operand of the next product and goes from accumulator to
// operand layout inside the thread's registers: no shared-memory round trip, no barrier and
// no other warp on the path from one chunk's state to the next.  The right operands (q, k, N,
// P) are tiles in shared memory that all warps of the CTA read, double-buffered with
// asynchronous copies.
#pragma once

#include "delta_common.cuh"

namespace gnorm {

constexpr int kScanWarps = 4;  // 64 columns of V per CTA
constexpr int kScanThreads = kScanWarps * 32;

template <int KD, bool kBwd>
struct ScanStage {
  static constexpr int kQ = 0;
  static constexpr int kK = KD / 64 * kTileBytes;
  static constexpr int kN = 2 * kK;  // N hi, N lo, P hi, P lo, scalars
  static constexpr int kScal = kN + 4 * kTileBytes;
  static constexpr int kV = kScal + 1024;  // v (forward) or do (backward)
  static constexpr int kW = kV + kTileBytes;  // W hi, W lo (backward)
  static constexpr int kBytes = kBwd ? kW + 2 * kTileBytes : kW;
};

// Fragment order of a 16 x K strip of FP32 values: tile n (8 columns), lane, four values.
__device__ __forceinline__ long long frag_off(int KD, int strip, int n, int lane) {
  return ((static_cast<long long>(strip) * (KD / 8) + n) * 32 + lane) * 16;
}

// acc (16 x 64 tokens) += A (16 x 16 at k16 block, hi and lo) times the transposed rows of
// the 64-row tile at columns c0: an exact right operand.
__device__ __forceinline__ void mul_rows_exact(float acc[8][4], const uint32_t hi[4],
                                               const uint32_t lo[4], uint32_t tile, int c0,
                                               int lane) {
#pragma unroll
  for (int nb = 0; nb < 4; ++nb) {
    uint32_t b[4];
    ldsm4(b, addr_b(tile, nb * 16, c0, lane));
    mma16816(acc[2 * nb], hi, b[0], b[1]);
    mma16816(acc[2 * nb + 1], hi, b[2], b[3]);
    mma16816(acc[2 * nb], lo, b[0], b[1]);
    mma16816(acc[2 * nb + 1], lo, b[2], b[3]);
  }
}

// acc (16 x 64) += A (16 x 64, split) M^T for a lower triangular 64 x 64 M given as hi and lo
// tiles: column block nb takes the k blocks up to nb.
__device__ __forceinline__ void mul_lower_t(float acc[8][4], const uint32_t (*hi)[4],
                                            const uint32_t (*lo)[4], uint32_t mhi, uint32_t mlo,
                                            int lane) {
#pragma unroll
  for (int nb = 0; nb < 4; ++nb) {
#pragma unroll
    for (int kb = 0; kb <= nb; ++kb) {
      uint32_t b[4], c[4];
      ldsm4(b, addr_b(mhi, nb * 16, kb * 16, lane));
      ldsm4(c, addr_b(mlo, nb * 16, kb * 16, lane));
      mma16816(acc[2 * nb], hi[kb], b[0], b[1]);
      mma16816(acc[2 * nb + 1], hi[kb], b[2], b[3]);
      mma16816(acc[2 * nb], lo[kb], b[0], b[1]);
      mma16816(acc[2 * nb + 1], lo[kb], b[2], b[3]);
      mma16816(acc[2 * nb], hi[kb], c[0], c[1]);
      mma16816(acc[2 * nb + 1], hi[kb], c[2], c[3]);
    }
  }
}

// The same against M itself (k are M's rows): column block nb takes the k blocks from nb on.
// kExact: A is exact (lo unused).
template <bool kExact>
__device__ __forceinline__ void mul_lower(float acc[8][4], const uint32_t (*hi)[4],
                                          const uint32_t (*lo)[4], uint32_t mhi, uint32_t mlo,
                                          int lane) {
#pragma unroll
  for (int nb = 0; nb < 4; ++nb) {
#pragma unroll
    for (int kb = nb; kb < 4; ++kb) {
      uint32_t b[4], c[4];
      ldsm4t(b, addr_bt(mhi, kb * 16, nb * 16, lane));
      ldsm4t(c, addr_bt(mlo, kb * 16, nb * 16, lane));
      mma16816(acc[2 * nb], hi[kb], b[0], b[1]);
      mma16816(acc[2 * nb + 1], hi[kb], b[2], b[3]);
      if constexpr (!kExact) {
        mma16816(acc[2 * nb], lo[kb], b[0], b[1]);
        mma16816(acc[2 * nb + 1], lo[kb], b[2], b[3]);
      }
      mma16816(acc[2 * nb], hi[kb], c[0], c[1]);
      mma16816(acc[2 * nb + 1], hi[kb], c[2], c[3]);
    }
  }
}

// S^T (16 x KD) += A (16 x 64 tokens, split) times the rows of a [64, KD] tensor (exact).
template <int KD>
__device__ __forceinline__ void rank_update(float st[KD / 8][4], const uint32_t (*hi)[4],
                                            const uint32_t (*lo)[4], uint32_t tiles, int lane) {
#pragma unroll
  for (int kb = 0; kb < 4; ++kb) {
#pragma unroll
    for (int nb = 0; nb < KD / 16; ++nb) {
      uint32_t b[4];
      ldsm4t(b, addr_bt(tiles + (nb >> 2) * kTileBytes, kb * 16, (nb & 3) * 16, lane));
      mma16816(st[2 * nb], hi[kb], b[0], b[1]);
      mma16816(st[2 * nb + 1], hi[kb], b[2], b[3]);
      mma16816(st[2 * nb], lo[kb], b[0], b[1]);
      mma16816(st[2 * nb + 1], lo[kb], b[2], b[3]);
    }
  }
}

// x (16 x 64 tokens, accumulator layout) times f[token], as split fragments.
__device__ __forceinline__ void split_scaled(const float x[8][4], const float* f, float s,
                                             uint32_t (*hi)[4], uint32_t (*lo)[4], int lane) {
#pragma unroll
  for (int kb = 0; kb < 4; ++kb) {
    float t[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float2 w = *reinterpret_cast<const float2*>(f + (2 * kb + u) * 8 + 2 * (lane & 3));
      t[u][0] = x[2 * kb + u][0] * (w.x * s);
      t[u][1] = x[2 * kb + u][1] * (w.y * s);
      t[u][2] = x[2 * kb + u][2] * (w.x * s);
      t[u][3] = x[2 * kb + u][3] * (w.y * s);
    }
    split_frag(t[0], t[1], hi[kb], lo[kb]);
  }
}

// The strip's 16 columns of a [64 tokens, 64] tile in shared memory, as packed pairs in the
// accumulator layout of its transpose: r[n][0] rows lane/4, r[n][1] rows lane/4 + 8.
__device__ __forceinline__ void load_strip(uint32_t r[8][2], uint32_t tile, int col0, int lane) {
#pragma unroll
  for (int tb = 0; tb < 4; ++tb) {
    uint32_t f[4];
    ldsm4t(f, addr_at(tile, tb * 16, col0, lane));
    r[2 * tb][0] = f[0];
    r[2 * tb][1] = f[1];
    r[2 * tb + 1][0] = f[2];
    r[2 * tb + 1][1] = f[3];
  }
}

// The other way: pairs into the strip's columns of the tile, then 16-byte stores of its rows.
__device__ __forceinline__ void stage_strip(const uint32_t r[8][2], uint32_t tile, int col0,
                                            int lane) {
#pragma unroll
  for (int tb = 0; tb < 4; ++tb) {
    const uint32_t f[4] = {r[2 * tb][0], r[2 * tb][1], r[2 * tb + 1][0], r[2 * tb + 1][1]};
    stsm4t(addr_at(tile, tb * 16, col0, lane), f);
  }
}

template <int KD>
__device__ __forceinline__ void load_state(float st[KD / 8][4], const float* p, int V, int v0,
                                           int lane) {
  // p: [KD, V] of this (sequence, head); st: the transposed strip
  const int va = v0 + (lane >> 2);
#pragma unroll
  for (int n = 0; n < KD / 8; ++n) {
    const int k0 = n * 8 + 2 * (lane & 3);
    st[n][0] = p[static_cast<long long>(k0) * V + va];
    st[n][1] = p[static_cast<long long>(k0 + 1) * V + va];
    st[n][2] = p[static_cast<long long>(k0) * V + va + 8];
    st[n][3] = p[static_cast<long long>(k0 + 1) * V + va + 8];
  }
}
template <int KD>
__device__ __forceinline__ void store_state(const float st[KD / 8][4], float* p, int V, int v0,
                                            int lane) {
  const int va = v0 + (lane >> 2);
#pragma unroll
  for (int n = 0; n < KD / 8; ++n) {
    const int k0 = n * 8 + 2 * (lane & 3);
    p[static_cast<long long>(k0) * V + va] = st[n][0];
    p[static_cast<long long>(k0 + 1) * V + va] = st[n][1];
    p[static_cast<long long>(k0) * V + va + 8] = st[n][2];
    p[static_cast<long long>(k0 + 1) * V + va + 8] = st[n][3];
  }
}

// Forward.  kOut: writes o and the final state.  kSave: writes every chunk's S and W for the
// backward (which runs this pass again instead of keeping them since the forward).
template <int KD, bool kOut, bool kSave>
__global__ void __launch_bounds__(kScanThreads, 1) delta_scan_fwd_kernel(const __grid_constant__ DeltaArgs a) {
  using St = ScanStage<KD, false>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int vt = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int hk = h / (a.Hv / a.Hk);
  const int col0 = warp * 16, v0 = vt * 64 + col0, strip = v0 / 16;
  grid_dependency_wait();
  allow_dependent_launch();
  const long long start = seq_start(a.seq, b), end = seq_end(a.seq, b);
  const long long base = seq_base(a.seq, b);
  const int chunks = static_cast<int>((end - start + kChunk - 1) / kChunk);
  const uint32_t sbase = smem_u32(smem);

  auto issue = [&](int c) {
    const uint32_t st = sbase + (c & 1) * St::kBytes;
    const long long t0 = start + static_cast<long long>(c) * kChunk;
    const int live = static_cast<int>(end - t0 < kChunk ? end - t0 : kChunk);
    if constexpr (kOut)
      load_rows<kScanThreads>(st + St::kQ, a.q + t0 * a.ldq + static_cast<long long>(hk) * KD, a.ldq,
                              KD, live);
    load_rows<kScanThreads>(st + St::kK, a.k + t0 * a.ldk + static_cast<long long>(hk) * KD, a.ldk,
                            KD, live);
    const uint8_t* prep = a.prep + ((base + c) * a.Hv + h) * kPrepBytes;
    load_flat<kScanThreads>(st + St::kN, prep, kOut ? 4 * kTileBytes : 2 * kTileBytes);
    load_flat<kScanThreads>(st + St::kScal, prep + kPrepTiles, 784);
    load_rows<kScanThreads>(st + St::kV, a.v + t0 * a.ldv + static_cast<long long>(h) * a.V + vt * 64,
                            a.ldv, 64, live);
    cp_commit();
  };

  float st[KD / 8][4];
  const long long head_state = (static_cast<long long>(b) * a.Hv + h) * KD * a.V;
  if (a.state_in != nullptr) {
    load_state<KD>(st, a.state_in + head_state, a.V, v0, lane);
  } else {
#pragma unroll
    for (int n = 0; n < KD / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) st[n][e] = 0.f;
  }
  if (chunks > 0) issue(0);
  for (int c = 0; c < chunks; ++c) {
    if (c + 1 < chunks) {
      issue(c + 1);
      cp_wait<1>();
    } else {
      cp_wait<0>();
    }
    __syncthreads();
    const uint32_t sg = sbase + (c & 1) * St::kBytes;
    const float* scal = reinterpret_cast<const float*>(smem + (c & 1) * St::kBytes + St::kScal);
    const long long t0 = start + static_cast<long long>(c) * kChunk;
    const int live = static_cast<int>(end - t0 < kChunk ? end - t0 : kChunk);
    const long long hs = (base + c) * a.Hv + h;
    if constexpr (kSave) {
      uint8_t* p = a.s_ws + hs * KD * a.V * 4;
#pragma unroll
      for (int n = 0; n < KD / 8; ++n)
        *reinterpret_cast<float4*>(p + frag_off(KD, strip, n, lane)) =
            make_float4(st[n][0], st[n][1], st[n][2], st[n][3]);
    }
    // S^T K^T and S^T Q^T
    float x[8][4], o[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[n][e] = o[n][e] = 0.f;
#pragma unroll
    for (int kb = 0; kb < KD / 16; ++kb) {
      uint32_t hi[4], lo[4];
      split_frag(st[2 * kb], st[2 * kb + 1], hi, lo);
      const uint32_t toff = (kb >> 2) * kTileBytes;
      mul_rows_exact(x, hi, lo, sg + St::kK + toff, (kb & 3) * 16, lane);
      if constexpr (kOut) mul_rows_exact(o, hi, lo, sg + St::kQ + toff, (kb & 3) * 16, lane);
    }
    // X = V - gamma K S
    {
      uint32_t vv[8][2];
      load_strip(vv, sg + St::kV, col0, lane);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const float2 gm = *reinterpret_cast<const float2*>(scal + 64 + n * 8 + 2 * (lane & 3));
        x[n][0] = fmaf(-gm.x, x[n][0], bf_lo(vv[n][0]));
        x[n][1] = fmaf(-gm.y, x[n][1], bf_hi(vv[n][0]));
        x[n][2] = fmaf(-gm.x, x[n][2], bf_lo(vv[n][1]));
        x[n][3] = fmaf(-gm.y, x[n][3], bf_hi(vv[n][1]));
        o[n][0] *= gm.x;
        o[n][1] *= gm.y;
        o[n][2] *= gm.x;
        o[n][3] *= gm.y;
      }
    }
    uint32_t hi[4][4], lo[4][4];
    // W = X - N (beta X): with the sign in the operand
    split_scaled(x, scal, -1.f, hi, lo, lane);
    mul_lower_t(x, hi, lo, sg + St::kN, sg + St::kN + kTileBytes, lane);
    if constexpr (kSave) {
      // W as hi and lo tiles, through the strip's columns of the v tile (this warp's alone)
      uint32_t wh[8][2], wl[8][2];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        split2(x[n][0], x[n][1], wh[n][0], wl[n][0]);
        split2(x[n][2], x[n][3], wh[n][1], wl[n][1]);
      }
      uint8_t* p = a.w_ws + hs * (2LL * a.V / 64 * kTileBytes) + vt * kTileBytes;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        __syncwarp();
        stage_strip(part == 0 ? wh : wl, sg + St::kV, col0, lane);
        __syncwarp();
        uint8_t* dst = p + part * (a.V / 64) * kTileBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t off = tile_off(i * 16 + (lane >> 1), (col0 >> 3) + (lane & 1));
          *reinterpret_cast<uint4*>(dst + off) =
              *reinterpret_cast<const uint4*>(smem + (c & 1) * St::kBytes + St::kV + off);
        }
      }
    }
    // Y = beta W
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const float2 be = *reinterpret_cast<const float2*>(scal + n * 8 + 2 * (lane & 3));
      x[n][0] *= be.x;
      x[n][1] *= be.y;
      x[n][2] *= be.x;
      x[n][3] *= be.y;
    }
    if constexpr (kOut) {
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) split_frag(x[2 * kb], x[2 * kb + 1], hi[kb], lo[kb]);
      mul_lower_t(o, hi, lo, sg + St::kN + 2 * kTileBytes, sg + St::kN + 3 * kTileBytes, lane);
      uint32_t ob[8][2];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        ob[n][0] = pack_bf16x2(a.scale * o[n][0], a.scale * o[n][1]);
        ob[n][1] = pack_bf16x2(a.scale * o[n][2], a.scale * o[n][3]);
      }
      __syncwarp();
      stage_strip(ob, sg + St::kV, col0, lane);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = i * 16 + (lane >> 1);
        if (row < live)
          *reinterpret_cast<uint4*>(a.o + (t0 + row) * a.ldo + static_cast<long long>(h) * a.V + v0 +
                                    (lane & 1) * 8) =
              *reinterpret_cast<const uint4*>(smem + (c & 1) * St::kBytes + St::kV +
                                              tile_off(row, (col0 >> 3) + (lane & 1)));
      }
    }
    // S' = e^{G_C} S + K^T (lambda Y)
    split_scaled(x, scal + 128, 1.f, hi, lo, lane);
    const float whole = scal[192];
#pragma unroll
    for (int n = 0; n < KD / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) st[n][e] *= whole;
    rank_update<KD>(st, hi, lo, sg + St::kK, lane);
    __syncthreads();  // the stage may be filled again
  }
  if (kOut && a.state_out != nullptr)
    store_state<KD>(st, a.state_out + head_state, a.V, v0, lane);
}

// Sums r[n][e] over the 16 rows of the strip (rows lane/4 and lane/4 + 8 of every column) and
// leaves column n * 8 + 2 (lane % 4) + e's sum in lanes 0..3.
__device__ __forceinline__ void strip_sums(float r[8][2], float* out, int lane) {
#pragma unroll
  for (int n = 0; n < 8; ++n) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) r[n][e] += __shfl_xor_sync(0xffffffffu, r[n][e], off);
    }
    if (lane < 4) *reinterpret_cast<float2*>(out + n * 8 + 2 * lane) = make_float2(r[n][0], r[n][1]);
  }
}

// Backward, from the last chunk to the first.  D^T (16 x K per warp) is the gradient of the
// state after the chunk:
//   dY = scale P^T dO + lambda K D    U = dY - N^T (beta dY)    dX = dV = beta U
//   dbeta = W . U    b = lambda beta (K D) . W  (for dg)
//   D' = e^{G_C} D + Q^T (scale gamma dO) - K^T (gamma dX)
// It writes dv, what dX has below BF16, D of every chunk and each strip's share of the two
// row sums.
template <int KD>
__global__ void __launch_bounds__(kScanThreads, 1) delta_scan_bwd_kernel(const __grid_constant__ DeltaArgs a) {
  using St = ScanStage<KD, true>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int vt = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int hk = h / (a.Hv / a.Hk);
  const int col0 = warp * 16, v0 = vt * 64 + col0, strip = v0 / 16;
  grid_dependency_wait();
  allow_dependent_launch();
  const long long start = seq_start(a.seq, b), end = seq_end(a.seq, b);
  const long long base = seq_base(a.seq, b);
  const int chunks = static_cast<int>((end - start + kChunk - 1) / kChunk);
  const uint32_t sbase = smem_u32(smem);

  auto issue = [&](int c) {
    const uint32_t st = sbase + (c & 1) * St::kBytes;
    const long long t0 = start + static_cast<long long>(c) * kChunk;
    const int live = static_cast<int>(end - t0 < kChunk ? end - t0 : kChunk);
    load_rows<kScanThreads>(st + St::kQ, a.q + t0 * a.ldq + static_cast<long long>(hk) * KD, a.ldq,
                            KD, live);
    load_rows<kScanThreads>(st + St::kK, a.k + t0 * a.ldk + static_cast<long long>(hk) * KD, a.ldk,
                            KD, live);
    const long long hs = (base + c) * a.Hv + h;
    const uint8_t* prep = a.prep + hs * kPrepBytes;
    load_flat<kScanThreads>(st + St::kN, prep, 4 * kTileBytes);
    load_flat<kScanThreads>(st + St::kScal, prep + kPrepTiles, 784);
    load_rows<kScanThreads>(st + St::kV,
                            a.dout + t0 * a.lddo + static_cast<long long>(h) * a.V + vt * 64, a.lddo,
                            64, live);
    const uint8_t* w = a.w_ws + hs * (2LL * a.V / 64 * kTileBytes) + vt * kTileBytes;
    load_flat<kScanThreads>(st + St::kW, w, kTileBytes);
    load_flat<kScanThreads>(st + St::kW + kTileBytes, w + (a.V / 64) * kTileBytes, kTileBytes);
    cp_commit();
  };

  float d[KD / 8][4];
  const long long head_state = (static_cast<long long>(b) * a.Hv + h) * KD * a.V;
  if (a.dstate_out != nullptr) {
    load_state<KD>(d, a.dstate_out + head_state, a.V, v0, lane);
  } else {
#pragma unroll
    for (int n = 0; n < KD / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) d[n][e] = 0.f;
  }
  if (chunks > 0) issue(chunks - 1);
  for (int c = chunks - 1; c >= 0; --c) {
    if (c > 0) {
      issue(c - 1);
      cp_wait<1>();
    } else {
      cp_wait<0>();
    }
    __syncthreads();
    uint8_t* stage = smem + (c & 1) * St::kBytes;
    const uint32_t sg = sbase + (c & 1) * St::kBytes;
    const float* scal = reinterpret_cast<const float*>(stage + St::kScal);
    const long long t0 = start + static_cast<long long>(c) * kChunk;
    const int live = static_cast<int>(end - t0 < kChunk ? end - t0 : kChunk);
    const long long hs = (base + c) * a.Hv + h;
    {
      uint8_t* p = a.d_ws + hs * KD * a.V * 4;
#pragma unroll
      for (int n = 0; n < KD / 8; ++n)
        *reinterpret_cast<float4*>(p + frag_off(KD, strip, n, lane)) =
            make_float4(d[n][0], d[n][1], d[n][2], d[n][3]);
    }
    // D^T K^T, scaled by lambda
    float y[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) y[n][e] = 0.f;
#pragma unroll
    for (int kb = 0; kb < KD / 16; ++kb) {
      uint32_t hi[4], lo[4];
      split_frag(d[2 * kb], d[2 * kb + 1], hi, lo);
      mul_rows_exact(y, hi, lo, sg + St::kK + (kb >> 2) * kTileBytes, (kb & 3) * 16, lane);
    }
    float w[8][4];
    {
      uint32_t wh[8][2], wl[8][2];
      load_strip(wh, sg + St::kW, col0, lane);
      load_strip(wl, sg + St::kW + kTileBytes, col0, lane);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        w[n][0] = bf_lo(wh[n][0]) + bf_lo(wl[n][0]);
        w[n][1] = bf_hi(wh[n][0]) + bf_hi(wl[n][0]);
        w[n][2] = bf_lo(wh[n][1]) + bf_lo(wl[n][1]);
        w[n][3] = bf_hi(wh[n][1]) + bf_hi(wl[n][1]);
      }
    }
    float* dots = a.dots + (hs * (a.V / 16) + strip) * 128;
    {
      float r[8][2];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const int t = n * 8 + 2 * (lane & 3);
        const float2 lm = *reinterpret_cast<const float2*>(scal + 128 + t);
        const float2 be = *reinterpret_cast<const float2*>(scal + t);
        y[n][0] *= lm.x;
        y[n][1] *= lm.y;
        y[n][2] *= lm.x;
        y[n][3] *= lm.y;
        r[n][0] = be.x * fmaf(y[n][0], w[n][0], y[n][2] * w[n][2]);
        r[n][1] = be.y * fmaf(y[n][1], w[n][1], y[n][3] * w[n][3]);
      }
      strip_sums(r, dots, lane);
    }
    // + scale P^T dO
    uint32_t dof[8][2];
    load_strip(dof, sg + St::kV, col0, lane);
    uint32_t hi[4][4], lo[4][4];
    {
      float p[8][4];
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) p[n][e] = 0.f;
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        hi[kb][0] = dof[2 * kb][0];
        hi[kb][1] = dof[2 * kb][1];
        hi[kb][2] = dof[2 * kb + 1][0];
        hi[kb][3] = dof[2 * kb + 1][1];
      }
      mul_lower<true>(p, hi, hi, sg + St::kN + 2 * kTileBytes, sg + St::kN + 3 * kTileBytes, lane);
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[n][e] = fmaf(a.scale, p[n][e], y[n][e]);
    }
    // U = dY - N^T (beta dY)
    split_scaled(y, scal, -1.f, hi, lo, lane);
    mul_lower<false>(y, hi, lo, sg + St::kN, sg + St::kN + kTileBytes, lane);
    {
      float r[8][2];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        r[n][0] = fmaf(y[n][0], w[n][0], y[n][2] * w[n][2]);
        r[n][1] = fmaf(y[n][1], w[n][1], y[n][3] * w[n][3]);
      }
      strip_sums(r, dots + 64, lane);
    }
    // dX = beta U: dv, and what is left below BF16
    uint32_t xh[8][2], xl[8][2];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const float2 be = *reinterpret_cast<const float2*>(scal + n * 8 + 2 * (lane & 3));
      y[n][0] *= be.x;
      y[n][1] *= be.y;
      y[n][2] *= be.x;
      y[n][3] *= be.y;
      split2(y[n][0], y[n][1], xh[n][0], xl[n][0]);
      split2(y[n][2], y[n][3], xh[n][1], xl[n][1]);
    }
    __syncwarp();
    stage_strip(xh, sg + St::kW, col0, lane);
    stage_strip(xl, sg + St::kW + kTileBytes, col0, lane);
    __syncwarp();
    {
      uint8_t* xlo = a.x_ws + hs * (a.V / 64 * kTileBytes) + vt * kTileBytes;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = i * 16 + (lane >> 1);
        const uint32_t off = tile_off(row, (col0 >> 3) + (lane & 1));
        *reinterpret_cast<uint4*>(xlo + off) =
            *reinterpret_cast<const uint4*>(stage + St::kW + kTileBytes + off);
        if (row < live)
          *reinterpret_cast<uint4*>(a.dv + (t0 + row) * a.lddv + static_cast<long long>(h) * a.V +
                                    v0 + (lane & 1) * 8) =
              *reinterpret_cast<const uint4*>(stage + St::kW + off);
      }
    }
    // D' = e^{G_C} D + Q^T (scale gamma dO) - K^T (gamma dX)
    const float whole = scal[192];
#pragma unroll
    for (int n = 0; n < KD / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) d[n][e] *= whole;
    split_scaled(y, scal + 64, -1.f, hi, lo, lane);
    rank_update<KD>(d, hi, lo, sg + St::kK, lane);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      y[n][0] = bf_lo(dof[n][0]);
      y[n][1] = bf_hi(dof[n][0]);
      y[n][2] = bf_lo(dof[n][1]);
      y[n][3] = bf_hi(dof[n][1]);
    }
    split_scaled(y, scal + 64, a.scale, hi, lo, lane);
    rank_update<KD>(d, hi, lo, sg + St::kQ, lane);
    __syncthreads();
  }
  if (a.dstate_in != nullptr) store_state<KD>(d, a.dstate_in + head_state, a.V, v0, lane);
}

}  // namespace gnorm
