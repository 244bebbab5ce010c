// delta_scan.cuh -- the chunk-after-chunk part of the gated delta rule, forward and backward
// (formulas and notation: delta_common.cuh).
//
// Bound by the way from one chunk's state to the next, three small products in a row
// (X = V - gamma K S, W = X - N beta X, S' = e^{G_C} S + K^T lambda Y) for every chunk of the
// longest sequence.  So the work of a head is spread as widely as its products allow: a strip
// of 16 of the state's V columns (an instruction's 16 rows, everything being computed
// transposed) belongs to a group of four warps, one per scheduler of the SM, and a head of
// 128 columns to eight strips on up to eight SMs.  Within a strip a warp owns a quarter of
// the state's K columns, in registers for the whole sequence, and two of the chunk's eight
// token tiles, w and 7 - w, whose shares of a triangular product add up to the same for every
// warp.  Each intermediate goes from accumulators to the other warps as ready left operands
// through shared memory, one barrier of the group per product.  Four more warps per strip, one
// beside each of the others on its scheduler, take what the way from state to state does not
// need: the copies of the right operands (q, k, N, P, double-buffered), in the forward
// the output, in the backward the terms of dO.
//
// What only the call's inputs decide (the sequence's place, its state, the first q, k and v) is
// fetched before the wait for the kernel before, which is this call's own and has itself
// waited for everything older.
//
// The tensor cores of the fifth generation take at least 64 rows an instruction: a head's 128
// columns would be one tile on one SM, its 66000 values a chunk would be cut and scaled by
// that SM alone, and the other SMs would wait -- the heads of a layer are fewer than the SMs.
// (delta_head.cuh does that, for batches of many heads; delta_cols.cuh gives 32 columns an SM
// with the tokens as rows, for the forward of heads too many for a strip an SM.)
//
// A chunk of 128 x 128 heads takes, with a strip per SM, 2800 cycles without the output and 3400
// with it (S K 690, X 195, N 740, Y 285, the update 690, the state's parts 150), the backward's
// 3900: 8192 tokens x 16 heads 197, 229 and 279 us.  One warp issues an m16n8k16 every 14 cycles
// whatever its independent sums, two on a scheduler every 8.  Eight state warps, halves of each
// product added through shared memory, were slower (253 us for 232), operands fetched a step
// ahead as well where two strips share an SM (849 us for 780): shared memory, 80% busy there,
// is the other bound.
#pragma once

#include "delta_common.cuh"
#include "tcgen05.cuh"

namespace gnorm {

constexpr int kGroupThreads = 128;  // four warps on the state of a strip of 16 columns ...
constexpr int kStripThreads = 256;  // ... and four beside them

// Named barriers of a strip: among its state warps, among the others, and from one to the other
// (bar.arrive on one side, bar.sync on the other).
enum { kBarState = 1, kBarSide = 2, kBarA = 3, kBarB = 4, kBarC = 5, kBarsPerStrip = 5 };
__device__ __forceinline__ void bar_arrive(int id, int nthreads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

// A strip of W (16 columns): the three parts, each as 8 x 8 matrices [piece of 8 columns][tile
// of 8 tokens], in the workspace as in shared memory.
constexpr int kStripBytes = 2048;
__device__ __forceinline__ uint32_t strip_off(int piece, int token) {
  return static_cast<uint32_t>(((piece * 8 + (token >> 3)) * 8 + (token & 7)) * 16);
}

// Shared memory of a CTA: two stages, then each group's exchange buffers, then two barriers.
template <int KD, int G, bool kBwd>
struct ScanStage {
  static constexpr int kQ = 0;
  static constexpr int kK = KD / 64 * kTileBytes;
  static constexpr int kTri = 2 * kK;  // N, then P (three parts each)
  static constexpr int kScal = kTri + 6 * kTriBytes;
  static constexpr int kV = kScal + 1024;   // v (forward) or do (backward): rows of 16 G columns
  static constexpr int kW = kV + G * 2048;  // W's three parts (backward)
  static constexpr int kBytes = kW + (kBwd ? 3 * kStripBytes : 0);
};
constexpr int kFragBytes = 512;  // left operand of one 16 x 16 block, one part
template <int KD, bool kBwd>
struct ScanExchange {
  static constexpr int kState = KD / 16 * 3 * kFragBytes;
  static constexpr int kS = 0;  // the state, three parts; twice in the forward
  static constexpr int kX = (kBwd ? 1 : 2) * kState;      // beta X (beta dY)
  static constexpr int kY = kX + 12 * kFragBytes;         // lambda Y (gamma dX)
  static constexpr int kO = kY + 12 * kFragBytes;         // Y, two parts (scale gamma dO, three)
  static constexpr int kP = kO + (kBwd ? 12 : 8) * kFragBytes;  // scale P^T dO, FP32
  static constexpr int kR = kP + (kBwd ? 4096 : 0);             // Q^T (scale gamma dO), FP32
  static constexpr int kL = kR + (kBwd ? KD * 64 : 0);          // lambda K D, FP32
  static constexpr int kU = kL + (kBwd ? 4096 : 0);             // U, FP32
  static constexpr int kBytes = kU + (kBwd ? 4096 : 0);
};
template <int KD, int G, bool kBwd>
GNORM_HD constexpr int scan_smem() {
  return 2 * ScanStage<KD, G, kBwd>::kBytes + G * ScanExchange<KD, kBwd>::kBytes + 16 + 1024;  // 1024: alignment
}

// Fragment order of a 16 x K strip of FP32 values: tile n (8 columns), lane, four values.
__device__ __forceinline__ long long frag_off(int KD, int strip, int n, int lane) {
  return ((static_cast<long long>(strip) * (KD / 8) + n) * 32 + lane) * 16;
}

__device__ __forceinline__ void lds4(uint32_t r[4], uint32_t addr) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void sts2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// What a warp needs to know of its place: its token tiles and lane addresses.
struct ScanLane {
  int warp, lane;
  __device__ __forceinline__ ScanLane(int w, int l) : warp(w), lane(l) {}
  __device__ __forceinline__ int tile(int i) const { return i == 0 ? warp : 7 - warp; }
  // token of column e (0, 1) of this lane in own tile i
  __device__ __forceinline__ int token(int i) const { return tile(i) * 8 + 2 * (lane & 3); }
  // right operand: rows are the own tokens of a 64 x 64 tile
  __device__ __forceinline__ uint32_t rows(uint32_t t, int col0) const {
    return t + tile_off(tile(lane >> 4) * 8 + (lane & 7), (col0 >> 3) + ((lane >> 3) & 1));
  }
  // the own tokens of a strip of v or do, whose columns start `col` bytes into a row
  template <int G>
  __device__ __forceinline__ uint32_t strip(uint32_t s, int col) const {
    return s + (tile(lane >> 4) * 8 + (lane & 7)) * (G * 32) + ((lane >> 3) & 1) * 16 + col;
  }
  // the own tokens of a part of W
  __device__ __forceinline__ uint32_t wstrip(uint32_t s) const {
    return s + strip_off((lane >> 3) & 1, tile(lane >> 4) * 8 + (lane & 7));
  }
  // 16-byte piece `lane & 1` of own token `lane / 2`
  __device__ __forceinline__ int row() const { return tile(lane >> 4) * 8 + ((lane >> 1) & 7); }
};

// Writes an own token tile (accumulator layout, scaled by f) as left operand parts.
template <int kParts>
__device__ __forceinline__ void put_tile(uint32_t buf, int tile, int lane, const float x[4]) {
  uint32_t a[3], b[3];
  if constexpr (kParts == 3) {
    split3(x[0], x[1], a);
    split3(x[2], x[3], b);
  } else {
    split2(x[0], x[1], a[0], a[1]);
    split2(x[2], x[3], b[0], b[1]);
  }
#pragma unroll
  for (int p = 0; p < kParts; ++p)
    sts2(buf + ((tile >> 1) * kParts + p) * kFragBytes + lane * 16 + (tile & 1) * 8, a[p], b[p]);
}

// The warp's part of the state (columns n0 * 8 ..) as left operand, three parts.
template <int KD>
__device__ __forceinline__ void put_state(uint32_t buf, int warp, int lane,
                                          const float st[KD / 32][4]) {
#pragma unroll
  for (int kb = 0; kb < KD / 64; ++kb) {
    uint32_t f[4][3];
    split3(st[2 * kb][0], st[2 * kb][1], f[0]);
    split3(st[2 * kb][2], st[2 * kb][3], f[1]);
    split3(st[2 * kb + 1][0], st[2 * kb + 1][1], f[2]);
    split3(st[2 * kb + 1][2], st[2 * kb + 1][3], f[3]);
#pragma unroll
    for (int p = 0; p < 3; ++p)
      asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                       buf + ((warp * (KD / 64) + kb) * 3 + p) * kFragBytes + lane * 16),
                   "r"(f[0][p]), "r"(f[1][p]), "r"(f[2][p]), "r"(f[3][p])
                   : "memory");
  }
}

// D = A B.
__device__ __forceinline__ void mma16816_0(float d[4], const uint32_t a[4], uint32_t b0,
                                           uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void zero_tiles(float x[2][4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) x[i][e] = 0.f;
}

// acc (own tokens) = state (kParts of its three parts) times the rows of a [64, KD] tensor.
template <int KD, int kParts>
__device__ __forceinline__ void state_product(float acc[2][4], uint32_t sbuf, uint32_t tiles,
                                              const ScanLane& me) {
  float x[kParts][2][4];
  uint32_t rows[4];  // the swizzled addresses of a tile's four column blocks
#pragma unroll
  for (int i = 0; i < 4; ++i) rows[i] = me.rows(tiles, i * 16);
#pragma unroll
  for (int kb = 0; kb < KD / 16; ++kb) {
    uint32_t b[4];
    ldsm4(b, rows[kb & 3] + (kb >> 2) * kTileBytes);
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      uint32_t a[4];
      lds4(a, sbuf + (kb * 3 + p) * kFragBytes + me.lane * 16);
      if (kb == 0) {
        mma16816_0(x[p][0], a, b[0], b[1]);
        mma16816_0(x[p][1], a, b[2], b[3]);
      } else {
        mma16816(x[p][0], a, b[0], b[1]);
        mma16816(x[p][1], a, b[2], b[3]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc[i][e] = x[kParts - 1][i][e];
#pragma unroll
      for (int p = kParts - 2; p >= 0; --p) acc[i][e] += x[p][i][e];
    }
}

// acc (own tokens) += A (16 x 64 tokens, kA parts in `abuf`) times the lower triangular M
// (kM parts): kTrans = false: sum over j <= i of A_j M_ij, own tokens i; true: sum over i >= j
// of A_i M_ij, own tokens j.  Products of parts a + m < kOrder are taken, each order in sums
// of its own.
template <bool kTrans, int kA, int kM, int kOrder>
__device__ __forceinline__ void tri_product(float acc[2][4], const uint32_t* exact, uint32_t abuf,
                                            uint32_t tri, const ScanLane& me) {
  float x[kOrder][2][4];
#pragma unroll
  for (int o = 0; o < kOrder; ++o) zero_tiles(x[o]);
#pragma unroll
  for (int kb = 0; kb < 4; ++kb) {
    const bool use0 = kTrans ? kb >= me.tile(0) >> 1 : kb <= me.tile(0) >> 1;
    const bool use1 = kTrans ? kb >= me.tile(1) >> 1 : kb <= me.tile(1) >> 1;
    if (use0 || use1) {
      // a tile that takes no part reads the other's matrices
      const int t = (me.lane >> 4) ? (use1 ? me.tile(1) : me.tile(0)) : (use0 ? me.tile(0) : me.tile(1));
      const int hf = (me.lane >> 3) & 1;
      const int m = kTrans ? tri_row(2 * kb + hf) + t : tri_row(t) + 2 * kb + hf;
      const uint32_t addr = tri + m * 128 + (me.lane & 7) * 16;
      uint32_t b[kM][4];
#pragma unroll
      for (int p = 0; p < kM; ++p) {
        if constexpr (kTrans)
          ldsm4t(b[p], addr + p * kTriBytes);
        else
          ldsm4(b[p], addr + p * kTriBytes);
      }
#pragma unroll
      for (int q = 0; q < kA; ++q) {
        uint32_t a[4];
        if (exact != nullptr) {
#pragma unroll
          for (int e = 0; e < 4; ++e) a[e] = exact[kb * 4 + e];
        } else {
          lds4(a, abuf + (kb * kA + q) * kFragBytes + me.lane * 16);
        }
#pragma unroll
        for (int p = 0; p < kM; ++p) {
          if (q + p < kOrder) {
            if (use0) mma16816(x[q + p][0], a, b[p][0], b[p][1]);
            if (use1) mma16816(x[q + p][1], a, b[p][2], b[p][3]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v = x[kOrder - 1][i][e];
#pragma unroll
      for (int o = kOrder - 2; o >= 0; --o) v += x[o][i][e];
      acc[i][e] += v;
    }
}

// The warp's part of S^T += A (16 x 64 tokens, three parts) times the rows of a [64, KD] tensor;
// kNeg: -=.
template <int KD, bool kNeg>
__device__ __forceinline__ void rank_update(float st[KD / 32][4], uint32_t abuf, uint32_t tiles,
                                            const ScanLane& me) {
  constexpr int kNB = KD / 64;
  uint32_t rows[kNB];
#pragma unroll
  for (int nb = 0; nb < kNB; ++nb) {
    const int col = (me.warp * kNB + nb) * 16;
    rows[nb] = addr_bt(tiles + (col >> 6) * kTileBytes, 0, col & 63, me.lane);
  }
#pragma unroll
  for (int kb = 0; kb < 4; ++kb) {
    uint32_t b[kNB][4];
#pragma unroll
    for (int nb = 0; nb < kNB; ++nb) ldsm4t(b[nb], rows[nb] + kb * 2048);  // 16 tokens further
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      uint32_t a[4];
      lds4(a, abuf + (kb * 3 + p) * kFragBytes + me.lane * 16);
      if constexpr (kNeg) {
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] ^= 0x80008000u;
      }
#pragma unroll
      for (int nb = 0; nb < kNB; ++nb) {
        mma16816(st[2 * nb], a, b[nb][0], b[nb][1]);
        mma16816(st[2 * nb + 1], a, b[nb][2], b[nb][3]);
      }
    }
  }
}

// The warp's part of a state [KD, V], transposed.
template <int KD>
__device__ __forceinline__ void load_state(float st[KD / 32][4], const float* p, int V, int v0,
                                           const ScanLane& me) {
  const int va = v0 + (me.lane >> 2);
#pragma unroll
  for (int n = 0; n < KD / 32; ++n) {
    const int k0 = (me.warp * (KD / 32) + n) * 8 + 2 * (me.lane & 3);
    st[n][0] = p[static_cast<long long>(k0) * V + va];
    st[n][1] = p[static_cast<long long>(k0 + 1) * V + va];
    st[n][2] = p[static_cast<long long>(k0) * V + va + 8];
    st[n][3] = p[static_cast<long long>(k0 + 1) * V + va + 8];
  }
}
template <int KD>
__device__ __forceinline__ void store_state(const float st[KD / 32][4], float* p, int V, int v0,
                                            const ScanLane& me) {
  const int va = v0 + (me.lane >> 2);
#pragma unroll
  for (int n = 0; n < KD / 32; ++n) {
    const int k0 = (me.warp * (KD / 32) + n) * 8 + 2 * (me.lane & 3);
    p[static_cast<long long>(k0) * V + va] = st[n][0];
    p[static_cast<long long>(k0 + 1) * V + va] = st[n][1];
    p[static_cast<long long>(k0) * V + va + 8] = st[n][2];
    p[static_cast<long long>(k0 + 1) * V + va + 8] = st[n][3];
  }
}

// Own tokens of a strip (address of this lane's matrix row) as FP32 in accumulator layout.
__device__ __forceinline__ void get_strip(float x[2][4], uint32_t addr) {
  uint32_t f[4];
  ldsm4t(f, addr);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[i][0] = bf_lo(f[2 * i]);
    x[i][1] = bf_hi(f[2 * i]);
    x[i][2] = bf_lo(f[2 * i + 1]);
    x[i][3] = bf_hi(f[2 * i + 1]);
  }
}

// Own tokens as BF16 pairs through shared memory that is this warp's alone (`addr`: this lane's
// matrix row, `own`: where it then finds the 16 bytes of token me.row(), piece lane & 1).
__device__ __forceinline__ uint4 turn_strip(const uint32_t f[4], uint32_t addr, const uint8_t* own) {
  __syncwarp();
  stsm4t(addr, f);
  __syncwarp();
  return *reinterpret_cast<const uint4*>(own);
}

// Own tokens in FP32 from a warp to the one beside it.
__device__ __forceinline__ void put_fp32(float4* buf, const float x[2][4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) buf[i * 32] = make_float4(x[i][0], x[i][1], x[i][2], x[i][3]);
}
__device__ __forceinline__ void get_fp32(float x[2][4], const float4* buf) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 v = buf[i * 32];
    x[i][0] = v.x;
    x[i][1] = v.y;
    x[i][2] = v.z;
    x[i][3] = v.w;
  }
}

// Forward.  kOut: writes o and the final state.  kSave: writes every chunk's S and W for the
// backward (which runs this pass again instead of keeping them since the forward).
template <int KD, int G, bool kOut, bool kSave>
__global__ void __launch_bounds__(G * kStripThreads, 1)
    delta_scan_fwd_kernel(const __grid_constant__ DeltaArgs a, const __grid_constant__ DeltaMaps maps) {
  using St = ScanStage<KD, G, false>;
  using Ex = ScanExchange<KD, false>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int group = threadIdx.x / kStripThreads;
  const bool side = (threadIdx.x & kGroupThreads) != 0;
  const ScanLane me((threadIdx.x >> 5) & 3, threadIdx.x & 31);
  const int lane = me.lane;
  const int bars = group * kBarsPerStrip;
  const int h = blockIdx.y;
  const int hk = h / (a.Hv / a.Hk);
  const int vc = blockIdx.x * 16 * G;  // the CTA's first column
  const int v0 = vc + group * 16, strip = v0 / 16;
  const int b = seq_by_length(a.seq, blockIdx.z, lane);
  const long long start = seq_start(a.seq, b), end = seq_end(a.seq, b);
  const long long base = seq_base(a.seq, b);
  const int chunks = static_cast<int>((end - start + kChunk - 1) / kChunk);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t ex = sbase + 2 * St::kBytes + group * Ex::kBytes;
  // W in FP32 from a state warp to the one beside it (kSave), in the place of Y's two parts
  float4* wbuf = reinterpret_cast<float4*>(smem + 2 * St::kBytes + group * Ex::kBytes + Ex::kO) +
                 me.warp * 64 + lane;

  uint64_t* full = reinterpret_cast<uint64_t*>(smem + 2 * St::kBytes + G * Ex::kBytes);
  if (threadIdx.x == 0) {
    mbar_init(&full[0], 1);
    mbar_init(&full[1], 1);
    fence_barrier_init();
  }
  __syncthreads();

  if (side) {
    const int tid = group * kGroupThreads + (threadIdx.x & (kGroupThreads - 1));
    // one thread: the call's inputs, and what the kernel before has made of them
    auto issue_inputs = [&](int c) {
      uint8_t* st = smem + (c & 1) * St::kBytes;
      uint64_t* bar = &full[c & 1];
      const int t0 = static_cast<int>(start + static_cast<long long>(c) * kChunk);
      mbar_arrive_expect_tx(bar, (kOut ? 5 : 3) * kTriBytes + 784 + (kOut ? 2 : 1) * St::kK + G * 2048);
#pragma unroll
      for (int kt = 0; kt < KD / 64; ++kt)
        tma_load_2d(st + St::kK + kt * kTileBytes, &maps.k, hk * KD + kt * 64, t0, bar);
      tma_load_2d(st + St::kV, &maps.v, h * a.V + vc, t0, bar);
      if constexpr (kOut) {
#pragma unroll
        for (int kt = 0; kt < KD / 64; ++kt)
          tma_load_2d(st + St::kQ + kt * kTileBytes, &maps.q, hk * KD + kt * 64, t0, bar);
      }
    };
    auto issue_prep = [&](int c) {
      uint8_t* st = smem + (c & 1) * St::kBytes;
      const uint8_t* prep = a.prep + ((base + c) * a.Hv + h) * kPrepBytes;
      bulk_copy_g2s(st + St::kScal, prep + kPrepTri, 784, &full[c & 1]);
      bulk_copy_g2s(st + St::kTri, prep, (kOut ? 5 : 3) * kTriBytes, &full[c & 1]);
    };
    bool alive = true;
    if (chunks > 0 && tid == 0) issue_inputs(0);
    grid_dependency_wait();
    allow_dependent_launch();
    if (chunks > 0 && tid == 0) issue_prep(0);
    for (int c = 0; c < chunks; ++c) {
      const long long left = end - start - static_cast<long long>(c) * kChunk;
      if ((tid < 32 || left < kChunk) && alive)
        alive = mbar_spin(&full[c & 1], (c >> 1) & 1, a.err, kErrWaitFull);
      if (left < kChunk) {
        uint8_t* st = smem + (c & 1) * St::kBytes;
        const int live = static_cast<int>(left);
        clear_rows<G * kGroupThreads>(st + St::kK, 128, KD / 64, kTileBytes, live, tid);
        if constexpr (kOut) clear_rows<G * kGroupThreads>(st + St::kQ, 128, KD / 64, kTileBytes, live, tid);
        clear_rows<G * kGroupThreads>(st + St::kV, G * 32, 1, 0, live, tid);
      }
      // what this thread wrote into the other stage comes before the copies into it
      fence_smem_to_async();
      __syncthreads();  // stage c has arrived, the other one is free, the state can be read
      if (c + 1 < chunks && tid == 0) {
        issue_prep(c + 1);
        issue_inputs(c + 1);
      }
      if constexpr (kOut) {
        uint8_t* stage = smem + (c & 1) * St::kBytes;
        const uint32_t sg = sbase + (c & 1) * St::kBytes;
        const float* scal = reinterpret_cast<const float*>(stage + St::kScal);
        const long long t0 = start + static_cast<long long>(c) * kChunk;
        const int live = static_cast<int>(end - t0 < kChunk ? end - t0 : kChunk);
        // O = scale (gamma Q S + P Y)
        float o[2][4];
        state_product<KD, 2>(o, ex + Ex::kS + (c & 1) * Ex::kState, sg + St::kQ, me);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 gm = *reinterpret_cast<const float2*>(scal + 64 + me.token(i));
          o[i][0] *= gm.x;
          o[i][1] *= gm.y;
          o[i][2] *= gm.x;
          o[i][3] *= gm.y;
        }
        named_barrier_sync(bars + kBarA, kStripThreads);  // Y can be read
        tri_product<false, 2, 2, 2>(o, nullptr, ex + Ex::kO, sg + St::kTri + 3 * kTriBytes, me);
        uint32_t f[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          f[2 * i] = pack_bf16x2(a.scale * o[i][0], a.scale * o[i][1]);
          f[2 * i + 1] = pack_bf16x2(a.scale * o[i][2], a.scale * o[i][3]);
        }
        const int row = me.row();
        const uint4 v = turn_strip(f, me.strip<G>(sg + St::kV, group * 32),
                                   stage + St::kV + row * (G * 32) + group * 32 + (lane & 1) * 16);
        if (row < live)
          *reinterpret_cast<uint4*>(a.o + (t0 + row) * a.ldo + static_cast<long long>(h) * a.V + v0 +
                                    (lane & 1) * 8) = v;
      }
      if constexpr (kSave) {
        // W as the three parts' tiles, turned through the own tokens of v
        uint8_t* stage = smem + (c & 1) * St::kBytes;
        const uint32_t sg = sbase + (c & 1) * St::kBytes;
        const long long hs = (base + c) * a.Hv + h;
        named_barrier_sync(bars + kBarA, kStripThreads);  // W can be read, v has been
        float x[2][4];
        get_fp32(x, wbuf);
        uint32_t f[3][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t p[3];
          split3(x[i][0], x[i][1], p);
#pragma unroll
          for (int q = 0; q < 3; ++q) f[q][2 * i] = p[q];
          split3(x[i][2], x[i][3], p);
#pragma unroll
          for (int q = 0; q < 3; ++q) f[q][2 * i + 1] = p[q];
        }
        uint8_t* p = a.w_ws + (hs * (a.V / 16) + strip) * (3LL * kStripBytes) +
                     strip_off(lane & 1, me.row());
#pragma unroll
        for (int q = 0; q < 3; ++q)
          *reinterpret_cast<uint4*>(p + q * kStripBytes) =
              turn_strip(f[q], me.strip<G>(sg + St::kV, group * 32),
                         stage + St::kV + me.row() * (G * 32) + group * 32 + (lane & 1) * 16);
      }
    }
    return;
  }

  float st[KD / 32][4];
  const long long head_state = (static_cast<long long>(b) * a.Hv + h) * KD * a.V;
  if (a.state_in != nullptr) {
    load_state<KD>(st, a.state_in + head_state, a.V, v0, me);
  } else {
#pragma unroll
    for (int n = 0; n < KD / 32; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) st[n][e] = 0.f;
  }
  grid_dependency_wait();
  allow_dependent_launch();
  for (int c = 0; c < chunks; ++c) {
    const uint32_t sbuf = ex + Ex::kS + (c & 1) * Ex::kState;
    put_state<KD>(sbuf, me.warp, lane, st);
    __syncthreads();
    uint8_t* stage = smem + (c & 1) * St::kBytes;
    const uint32_t sg = sbase + (c & 1) * St::kBytes;
    const float* scal = reinterpret_cast<const float*>(stage + St::kScal);
    const long long hs = (base + c) * a.Hv + h;
    // X = V - gamma K S
    float x[2][4], y[2][4];
    state_product<KD, 3>(x, sbuf, sg + St::kK, me);
    get_strip(y, me.strip<G>(sg + St::kV, group * 32));
    float2 be[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 gm = *reinterpret_cast<const float2*>(scal + 64 + me.token(i));
      be[i] = *reinterpret_cast<const float2*>(scal + me.token(i));
      x[i][0] = fmaf(-gm.x, x[i][0], y[i][0]);
      x[i][1] = fmaf(-gm.y, x[i][1], y[i][1]);
      x[i][2] = fmaf(-gm.x, x[i][2], y[i][2]);
      x[i][3] = fmaf(-gm.y, x[i][3], y[i][3]);
      // the sign of W = X - N (beta X) is in the operand
      const float t[4] = {-be[i].x * x[i][0], -be[i].y * x[i][1], -be[i].x * x[i][2],
                          -be[i].y * x[i][3]};
      put_tile<3>(ex + Ex::kX, me.tile(i), lane, t);
    }
    named_barrier_sync(bars + kBarState, kGroupThreads);
    tri_product<false, 3, 3, 3>(x, nullptr, ex + Ex::kX, sg + St::kTri, me);
    // Y = beta W
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 lm = *reinterpret_cast<const float2*>(scal + 128 + me.token(i));
      y[i][0] = be[i].x * x[i][0];
      y[i][1] = be[i].y * x[i][1];
      y[i][2] = be[i].x * x[i][2];
      y[i][3] = be[i].y * x[i][3];
      if constexpr (kOut) put_tile<2>(ex + Ex::kO, me.tile(i), lane, y[i]);
      y[i][0] *= lm.x;
      y[i][1] *= lm.y;
      y[i][2] *= lm.x;
      y[i][3] *= lm.y;
      put_tile<3>(ex + Ex::kY, me.tile(i), lane, y[i]);
    }
    if constexpr (kSave) put_fp32(wbuf, x);
    bar_arrive(bars + kBarA, kStripThreads);
    if constexpr (kSave) {
      uint8_t* p = a.s_ws + hs * KD * a.V * 4;
#pragma unroll
      for (int n = 0; n < KD / 32; ++n)
        *reinterpret_cast<float4*>(p + frag_off(KD, strip, me.warp * (KD / 32) + n, lane)) =
            make_float4(st[n][0], st[n][1], st[n][2], st[n][3]);
    }
    // S' = e^{G_C} S + K^T (lambda Y)
    const float whole = scal[192];
#pragma unroll
    for (int n = 0; n < KD / 32; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) st[n][e] *= whole;
    named_barrier_sync(bars + kBarState, kGroupThreads);
    rank_update<KD, false>(st, ex + Ex::kY, sg + St::kK, me);
  }
  if (kOut && a.state_out != nullptr)
    store_state<KD>(st, a.state_out + head_state, a.V, v0, me);
}

// Sums r[i][e] over the 16 rows of the strip and leaves the sums of own tokens in `out`.
__device__ __forceinline__ void strip_sums(float r[2][2], float* out, const ScanLane& me) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) r[i][e] += __shfl_xor_sync(0xffffffffu, r[i][e], off);
    }
    if (me.lane < 4) *reinterpret_cast<float2*>(out + me.token(i)) = make_float2(r[i][0], r[i][1]);
  }
}

// Backward, from the last chunk to the first.  D^T is the gradient of the state after the
// chunk:
//   dY = scale P^T dO + lambda K D    U = dY - N^T (beta dY)    dX = dV = beta U
//   dbeta = W . U    b = lambda beta (K D) . W  (for dg)
//   D' = e^{G_C} D + Q^T (scale gamma dO) - K^T (gamma dX)
// It writes dv, what dX has below BF16 (two parts more), D of every chunk and each strip's share of
// the two row sums.
template <int KD>
__global__ void __launch_bounds__(kStripThreads, 1)
    delta_scan_bwd_kernel(const __grid_constant__ DeltaArgs a, const __grid_constant__ DeltaMaps maps) {
  using St = ScanStage<KD, 1, true>;
  using Ex = ScanExchange<KD, true>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const bool side = threadIdx.x >= kGroupThreads;
  const ScanLane me((threadIdx.x >> 5) & 3, threadIdx.x & 31);
  const int lane = me.lane;
  const int h = blockIdx.y;
  const int hk = h / (a.Hv / a.Hk);
  const int v0 = blockIdx.x * 16, strip = blockIdx.x;
  const int b = seq_by_length(a.seq, blockIdx.z, lane);
  const long long start = seq_start(a.seq, b), end = seq_end(a.seq, b);
  const long long base = seq_base(a.seq, b);
  const int chunks = static_cast<int>((end - start + kChunk - 1) / kChunk);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t ex = sbase + 2 * St::kBytes;
  float4* pbuf = reinterpret_cast<float4*>(smem + 2 * St::kBytes + Ex::kP) + me.warp * 64 + lane;
  float4* lbuf = reinterpret_cast<float4*>(smem + 2 * St::kBytes + Ex::kL) + me.warp * 64 + lane;
  float4* ubuf = reinterpret_cast<float4*>(smem + 2 * St::kBytes + Ex::kU) + me.warp * 64 + lane;
  float4* rbuf =
      reinterpret_cast<float4*>(smem + 2 * St::kBytes + Ex::kR) + me.warp * (KD / 32) * 32 + lane;

  uint64_t* full = reinterpret_cast<uint64_t*>(smem + 2 * St::kBytes + Ex::kBytes);
  if (threadIdx.x == 0) {
    mbar_init(&full[0], 1);
    mbar_init(&full[1], 1);
    fence_barrier_init();
  }
  __syncthreads();

  if (side) {
    const int tid = threadIdx.x - kGroupThreads;
    // one thread: the call's inputs, and what the kernels before have made of them
    auto issue_inputs = [&](int c) {
      uint8_t* st = smem + (c & 1) * St::kBytes;
      uint64_t* bar = &full[c & 1];
      const int t0 = static_cast<int>(start + static_cast<long long>(c) * kChunk);
      mbar_arrive_expect_tx(bar, 6 * kTriBytes + 784 + 3 * kStripBytes + 2 * St::kK + 2048);
      tma_load_2d(st + St::kV, &maps.do_strip, h * a.V + v0, t0, bar);
#pragma unroll
      for (int kt = 0; kt < KD / 64; ++kt) {
        tma_load_2d(st + St::kK + kt * kTileBytes, &maps.k, hk * KD + kt * 64, t0, bar);
        tma_load_2d(st + St::kQ + kt * kTileBytes, &maps.q, hk * KD + kt * 64, t0, bar);
      }
    };
    auto issue_made = [&](int c) {
      uint8_t* st = smem + (c & 1) * St::kBytes;
      uint64_t* bar = &full[c & 1];
      const long long hs = (base + c) * a.Hv + h;
      const uint8_t* prep = a.prep + hs * kPrepBytes;
      bulk_copy_g2s(st + St::kTri, prep, 6 * kTriBytes, bar);
      bulk_copy_g2s(st + St::kScal, prep + kPrepTri, 784, bar);
      bulk_copy_g2s(st + St::kW, a.w_ws + (hs * (a.V / 16) + strip) * (3LL * kStripBytes),
                    3 * kStripBytes, bar);
    };
    bool alive = true;
    uint32_t phases = 0;  // a bit per stage
    if (chunks > 0 && tid == 0) issue_inputs(chunks - 1);
    grid_dependency_wait();
    allow_dependent_launch();
    if (chunks > 0 && tid == 0) issue_made(chunks - 1);
    for (int c = chunks - 1; c >= 0; --c) {
      const long long left = end - start - static_cast<long long>(c) * kChunk;
      if ((tid < 32 || left < kChunk) && alive)
        alive = mbar_spin(&full[c & 1], (phases >> (c & 1)) & 1u, a.err, kErrWaitFull);
      if (left < kChunk) {
        uint8_t* st = smem + (c & 1) * St::kBytes;
        clear_rows<kGroupThreads>(st + St::kQ, 128, 2 * (KD / 64), kTileBytes, static_cast<int>(left), tid);
        clear_rows<kGroupThreads>(st + St::kV, 32, 1, 0, static_cast<int>(left), tid);
      }
      phases ^= 1u << (c & 1);
      // what this thread wrote into the other stage comes before the copies into it
      fence_smem_to_async();
      __syncthreads();  // stage c has arrived, the other one is free, D can be read
      const uint32_t sg = sbase + (c & 1) * St::kBytes;
      const float* scal = reinterpret_cast<const float*>(smem + (c & 1) * St::kBytes + St::kScal);
      // scale P^T dO
      uint32_t dof[16];
#pragma unroll
      for (int kb = 0; kb < 4; ++kb)
        ldsm4t(dof + 4 * kb, sg + St::kV + (kb * 16 + ((lane >> 4) << 3) + (lane & 7)) * 32 +
                                 ((lane >> 3) & 1) * 16);
      float t[2][4];
      zero_tiles(t);
      tri_product<true, 1, 3, 3>(t, dof, 0, sg + St::kTri + 3 * kTriBytes, me);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        pbuf[i * 32] = make_float4(a.scale * t[i][0], a.scale * t[i][1], a.scale * t[i][2],
                                   a.scale * t[i][3]);
      bar_arrive(kBarA, kStripThreads);
      if (c > 0 && tid == 0) {
        issue_inputs(c - 1);
        issue_made(c - 1);
      }
      // Q^T (scale gamma dO)
      get_strip(t, me.strip<1>(sg + St::kV, 0));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 gm = *reinterpret_cast<const float2*>(scal + 64 + me.token(i));
        const float sx = a.scale * gm.x, sy = a.scale * gm.y;
        const float z[4] = {sx * t[i][0], sy * t[i][1], sx * t[i][2], sy * t[i][3]};
        put_tile<3>(ex + Ex::kO, me.tile(i), lane, z);
      }
      named_barrier_sync(kBarSide, kGroupThreads);
      float r[KD / 32][4];
#pragma unroll
      for (int n = 0; n < KD / 32; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) r[n][e] = 0.f;
      rank_update<KD, false>(r, ex + Ex::kO, sg + St::kQ, me);
#pragma unroll
      for (int n = 0; n < KD / 32; ++n) rbuf[n * 32] = make_float4(r[n][0], r[n][1], r[n][2], r[n][3]);
      bar_arrive(kBarB, kStripThreads);
      // what leaves: dv, what dX has below BF16, the row sums of b and dbeta (the own tokens of
      // W are this warp's alone)
      uint8_t* stage = smem + (c & 1) * St::kBytes;
      const long long t0 = start + static_cast<long long>(c) * kChunk;
      const int live = static_cast<int>(end - t0 < kChunk ? end - t0 : kChunk);
      const long long hs = (base + c) * a.Hv + h;
      float w[2][4], y[2][4];
      get_strip(w, me.wstrip(sg + St::kW + 2 * kStripBytes));
#pragma unroll
      for (int p = 1; p >= 0; --p) {
        get_strip(t, me.wstrip(sg + St::kW + p * kStripBytes));
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) w[i][e] += t[i][e];
      }
      named_barrier_sync(kBarC, kStripThreads);  // lambda K D and U can be read
      get_fp32(y, lbuf);
      get_fp32(t, ubuf);
      float rb[2][2], rd[2][2];
      uint32_t x[3][4];  // dX in three parts
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 be = *reinterpret_cast<const float2*>(scal + me.token(i));
        rb[i][0] = be.x * fmaf(y[i][0], w[i][0], y[i][2] * w[i][2]);
        rb[i][1] = be.y * fmaf(y[i][1], w[i][1], y[i][3] * w[i][3]);
        rd[i][0] = fmaf(t[i][0], w[i][0], t[i][2] * w[i][2]);
        rd[i][1] = fmaf(t[i][1], w[i][1], t[i][3] * w[i][3]);
        uint32_t p[3], q[3];
        split3(be.x * t[i][0], be.y * t[i][1], p);
        split3(be.x * t[i][2], be.y * t[i][3], q);
#pragma unroll
        for (int m = 0; m < 3; ++m) {
          x[m][2 * i] = p[m];
          x[m][2 * i + 1] = q[m];
        }
      }
      const int row = me.row();
      const uint8_t* own = stage + St::kW + strip_off(lane & 1, row);
      const uint4 vh = turn_strip(x[0], me.wstrip(sg + St::kW), own);
#pragma unroll
      for (int m = 1; m < 3; ++m)
        *reinterpret_cast<uint4*>(a.x_ws + ((hs * 2 + m - 1) * (a.V / 64) + v0 / 64) * kTileBytes +
                                  tile_off(row, ((v0 & 63) >> 3) + (lane & 1))) =
            turn_strip(x[m], me.wstrip(sg + St::kW), own);
      if (row < live)
        *reinterpret_cast<uint4*>(a.dv + (t0 + row) * a.lddv + static_cast<long long>(h) * a.V + v0 +
                                  (lane & 1) * 8) = vh;
      float* dots = a.dots + (hs * (a.V / 16) + strip) * 128;
      strip_sums(rb, dots, me);
      strip_sums(rd, dots + 64, me);
    }
    return;
  }

  float d[KD / 32][4];
  const long long head_state = (static_cast<long long>(b) * a.Hv + h) * KD * a.V;
  if (a.dstate_out != nullptr) {
    load_state<KD>(d, a.dstate_out + head_state, a.V, v0, me);
  } else {
#pragma unroll
    for (int n = 0; n < KD / 32; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) d[n][e] = 0.f;
  }
  grid_dependency_wait();
  allow_dependent_launch();
  for (int c = chunks - 1; c >= 0; --c) {
    put_state<KD>(ex + Ex::kS, me.warp, lane, d);
    __syncthreads();
    const uint32_t sg = sbase + (c & 1) * St::kBytes;
    const float* scal = reinterpret_cast<const float*>(smem + (c & 1) * St::kBytes + St::kScal);
    const long long hs = (base + c) * a.Hv + h;
    // lambda K D
    float y[2][4];
    state_product<KD, 3>(y, ex + Ex::kS, sg + St::kK, me);
    float2 be[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 lm = *reinterpret_cast<const float2*>(scal + 128 + me.token(i));
      be[i] = *reinterpret_cast<const float2*>(scal + me.token(i));
      y[i][0] *= lm.x;
      y[i][1] *= lm.y;
      y[i][2] *= lm.x;
      y[i][3] *= lm.y;
    }
    put_fp32(lbuf, y);
    named_barrier_sync(kBarA, kStripThreads);  // scale P^T dO can be read
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 p = pbuf[i * 32];
      y[i][0] += p.x;
      y[i][1] += p.y;
      y[i][2] += p.z;
      y[i][3] += p.w;
      const float u[4] = {-be[i].x * y[i][0], -be[i].y * y[i][1], -be[i].x * y[i][2],
                          -be[i].y * y[i][3]};
      put_tile<3>(ex + Ex::kX, me.tile(i), lane, u);
    }
    named_barrier_sync(kBarState, kGroupThreads);
    // U = dY - N^T (beta dY)
    tri_product<true, 3, 3, 3>(y, nullptr, ex + Ex::kX, sg + St::kTri, me);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // gamma dX, dX = beta U
      const float2 gm = *reinterpret_cast<const float2*>(scal + 64 + me.token(i));
      const float fx = gm.x * be[i].x, fy = gm.y * be[i].y;
      const float u[4] = {fx * y[i][0], fy * y[i][1], fx * y[i][2], fy * y[i][3]};
      put_tile<3>(ex + Ex::kY, me.tile(i), lane, u);
    }
    put_fp32(ubuf, y);
    bar_arrive(kBarC, kStripThreads);
    {
      uint8_t* p = a.d_ws + hs * KD * a.V * 4;
#pragma unroll
      for (int n = 0; n < KD / 32; ++n)
        *reinterpret_cast<float4*>(p + frag_off(KD, strip, me.warp * (KD / 32) + n, lane)) =
            make_float4(d[n][0], d[n][1], d[n][2], d[n][3]);
    }
    // D' = e^{G_C} D + Q^T (scale gamma dO) - K^T (gamma dX)
    const float whole = scal[192];
#pragma unroll
    for (int n = 0; n < KD / 32; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) d[n][e] *= whole;
    named_barrier_sync(kBarState, kGroupThreads);
    rank_update<KD, true>(d, ex + Ex::kY, sg + St::kK, me);
    named_barrier_sync(kBarB, kStripThreads);  // the term of dO can be read
#pragma unroll
    for (int n = 0; n < KD / 32; ++n) {
      const float4 q = rbuf[n * 32];
      d[n][0] += q.x;
      d[n][1] += q.y;
      d[n][2] += q.z;
      d[n][3] += q.w;
    }
  }
  if (a.dstate_in != nullptr) store_state<KD>(d, a.dstate_in + head_state, a.V, v0, me);
}

}  // namespace gnorm
