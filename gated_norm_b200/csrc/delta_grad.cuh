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
// A CTA takes a chunk and key head, goes through the value heads of the group and adds their dQ
// and dK in registers, so the sum over shared heads has a fixed order.
//
// Everything here is products of 64-token tiles, done by tcgen05.  An instruction has 128
// rows; the 64 of a query-side product and the 64 of the key-side product with the same right
// operand are one: [dO; dX] S^T, [dO; dX] W^T, [Q; K] K^T, [Ph; -Eh] K.  Rows 0..63 of every
// accumulator belong to dQ, rows 64..127 to dK, and where only the key side has a product
// (W D^T, the transposed Ph and Eh, the further parts of dX) the upper rows multiply
// whatever tile lies before it and are not read.  A thread owns one row and a quarter of the columns.
// dg is FP32, so what it comes from, the products with S and F and E, has S, W and dX in three parts
// (24 bits; in two dg was 2e-6 to 3e-6 off, now 4e-7 to 5e-7).  What reaches only dq and dk, which
// are BF16, is in two: D, Ph, Eh and W against D.
//
// The products of a chunk and head take about 8000 cycles of the tensor cores, what it reads
// (S and D in FP32, W, dX, dO, q, k: 300 KB) as long again.  A CTA stays on its SM and goes through
// its chunks; the next one's tiles are copied, its states, q and k brought to L2 and its scalars
// computed behind the products of the current one.  8192 tokens x 16 heads of 128 x 128: 248 us,
// 33000 cycles a chunk and head (211 with two parts); what is left are the phases that follow one
// another -- S cut and stored, products, D cut and stored, products, pair terms, products -- with
// one CTA's shared memory and all of tensor memory in use.  S's third part has the place of q and
// k until its product is done.  Its product first, and q and k copied and multiplied behind the
// other ones, was slower (forward and backward 1073 us for 1066).
#pragma once

#include <type_traits>

#include "delta_common.cuh"
#include "delta_scan.cuh"
#include "tcgen05.cuh"

namespace gnorm {

// Brings the box of a tile at these coordinates to L2.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1)
               : "memory");
}

constexpr int kGradThreads = 512;
constexpr int kMLd = 65;

template <int KD, int VD>
struct GradSmem {
  // S's third part; then [q][k] of each 64 columns of K
  static constexpr int kQK = 0;
  static constexpr int kQKBytes = KD / 64 * 2 * kTileBytes;
  // the third parts of W and dX: [W][dX] of each 64 columns of V; then [do] and the first two:
  // [dX hi][dX lo][W hi][W lo]
  static constexpr int kA3 = kQK + kQKBytes;
  static constexpr int kA = kA3 + VD / 64 * 2 * kTileBytes;
  static_assert(VD / 64 * (KD / 64) * kTileBytes <= kQKBytes, "S's third part");
  // S's first two parts, then D (hi and lo tiles); then Ph, -Eh (hi, then lo) and the pair terms'
  // running sums; then dq and dk on their way out
  static constexpr int kBig = kA + VD / 64 * 5 * kTileBytes;
  static constexpr int kState = 2 * (VD / 64) * (KD / 64) * kTileBytes;
  static constexpr int kPairs = 4 * kTileBytes + 128 * kMLd * 4;
  static constexpr int kScal = kBig + (kState > kPairs ? kState : kPairs);
  // per item, twice: decay sums [64], beta, gamma, lambda, e^{G_C}, b and dbeta sums
  static constexpr int kItem = 512 + 1024 + 512;
  static constexpr int kWork = kScal + 2 * kItem;  // sums within an item
  static constexpr int kBytes = kWork + (3 * 512 + 16) * 4 + 88 + 1024;  // 1024: alignment
};

// What a CTA works on: a chunk and key head with live tokens, and one of its value heads.
struct GradItem {
  long long unit, slot, t0;
  int hk, r, live;
};
static_assert(sizeof(GradItem) <= 48, "the next item's place");

template <int KD, int VD>
__global__ void __launch_bounds__(kGradThreads, 1) delta_grad_kernel(const __grid_constant__ DeltaArgs a, const __grid_constant__ DeltaMaps maps) {
  using L = GradSmem<KD, VD>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  constexpr int kVT = VD / 64, kKT = KD / 64;
  constexpr int kCols = KD / 4;                         // columns of K per thread
  constexpr int kPair = KD * VD / 8 / kGradThreads;     // pairs of a state's float4 per thread
  // tensor memory columns (the second use of a range follows the reads of the first)
  constexpr uint32_t kD1 = 0, kD5 = 0;                  // [dO; dX] S^T     | [-; Ph^T] Q - [-; Eh^T] K
  constexpr uint32_t kD3 = 128, kD2b = 128;             // [-; dX lo] W^T   | [-; W] D^T
  constexpr uint32_t kD4 = 256, kD1b = 256;             // [-; dX lo] S^T   | [Ph; -Eh] K
  constexpr uint32_t kD2 = 384, kKK = 448;              // [dO; dX] W^T,  [Q; K] K^T
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = (warp & 3) * 32 + lane;               // 0..63 dQ, 64..127 dK
  const int cq = warp >> 2;                             // quarter of the columns
  const bool key_side = (warp & 2) != 0;
  const int tok = row & 63;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t s0 = smem_u32(smem);
  float* adot = reinterpret_cast<float*>(smem + L::kWork);          // [8][64]
  float* vpart = adot + 512;                                        // [8][64]
  float* rowsum = vpart + 512;                                      // [4][128]
  float* red = rowsum + 512;                                        // [16]
  uint64_t* bar = reinterpret_cast<uint64_t*>(red + 16);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bar + 1);
  uint64_t *full = bar + 2, *qk_full = bar + 3, *kk_done = bar + 10;
  GradItem* next = reinterpret_cast<GradItem*>(bar + 4);

  const int group = a.Hv / a.Hk;
  const long long units = a.slots * a.Hk;
  // the first unit from u on (in this CTA's steps) that has tokens
  auto find = [&](long long u) {
    GradItem it{};
    for (; u < units; u += gridDim.x) {
      it.slot = u / a.Hk;
      const int b = seq_of_slot(a.seq, it.slot, lane);
      const long long chunk = it.slot - seq_base(a.seq, b);
      it.t0 = seq_start(a.seq, b) + chunk * kChunk;
      const long long left = seq_end(a.seq, b) - it.t0;
      if (b == a.seq.B || chunk < 0 || left <= 0) continue;
      it.hk = static_cast<int>(u - it.slot * a.Hk);
      it.live = static_cast<int>(left < kChunk ? left : kChunk);
      break;
    }
    it.unit = u;
    return it;
  };
  auto next_item = [&](const GradItem& c) {
    if (c.r + 1 == group) return find(c.unit + gridDim.x);
    GradItem it = c;
    ++it.r;
    return it;
  };
  GradItem cur = find(blockIdx.x);
  grid_dependency_wait();  // (the kernel before is this call's own: see delta_scan.cuh)
  allow_dependent_launch();
  if (cur.unit >= units) return;

  // two neighbouring column tiles of a strip per warp and step
  auto pair_off = [&](int i) { return ((warp + i * (kGradThreads / 32)) * 2) * 32 + lane; };
  // one thread's copies, and every thread's pieces of W
  auto load_tiles = [&](const GradItem& it) {
    const int h = it.hk * group + it.r;
    const long long hs = it.slot * a.Hv + h;
    const int t0 = static_cast<int>(it.t0);
    uint8_t* base = smem + L::kA;
    if (tid == 0) {
      const uint8_t* x = a.x_ws + hs * 2 * kVT * kTileBytes;
      mbar_arrive_expect_tx(full, 4 * kVT * kTileBytes);
#pragma unroll
      for (int vt = 0; vt < kVT; ++vt) {
        uint8_t* at = base + vt * 5 * kTileBytes;
        tma_load_2d(at, &maps.do_tile, h * VD + vt * 64, t0, full);
        tma_load_2d(at + kTileBytes, &maps.dv, h * VD + vt * 64, t0, full);
        bulk_copy_g2s(at + 2 * kTileBytes, x + vt * kTileBytes, kTileBytes, full);
        bulk_copy_g2s(smem + L::kA3 + (2 * vt + 1) * kTileBytes, x + (kVT + vt) * kTileBytes, kTileBytes, full);
      }
    }
#pragma unroll
    for (int vt = 0; vt < kVT; ++vt) {
      // W's three parts, from strips of 16 columns: a 16-byte piece per thread and part
      const uint32_t at = s0 + L::kA + vt * 5 * kTileBytes;
      const int r = tid >> 3, p = tid & 7;
      const uint8_t* w = a.w_ws + (hs * (VD / 16) + vt * 4 + (p >> 1)) * (3LL * kStripBytes) + strip_off(p & 1, r);
      cp16(at + 3 * kTileBytes + tile_off(r, p), w, true);
      cp16(at + 4 * kTileBytes + tile_off(r, p), w + kStripBytes, true);
      cp16(s0 + L::kA3 + 2 * vt * kTileBytes + tile_off(r, p), w + 2 * kStripBytes, true);
    }
    cp_commit();
  };
  // one thread's copies of q and k
  auto load_qk = [&](const GradItem& it) {
    uint8_t* to = smem + L::kQK;
    mbar_arrive_expect_tx(qk_full, 2 * kKT * kTileBytes);
#pragma unroll
    for (int kt = 0; kt < kKT; ++kt) {
      tma_load_2d(to + kt * 2 * kTileBytes, &maps.q, it.hk * KD + kt * 64, static_cast<int>(it.t0), qk_full);
      tma_load_2d(to + (kt * 2 + 1) * kTileBytes, &maps.k, it.hk * KD + kt * 64, static_cast<int>(it.t0), qk_full);
    }
  };
  auto item_scalars = [&](int buf) { return smem + L::kScal + buf * L::kItem; };
  // four warps, `part` 0..3
  auto load_scalars = [&](const GradItem& it, int buf, int part) {
    const int h = it.hk * group + it.r;
    const long long hs = it.slot * a.Hv + h;
    float2* Gs = reinterpret_cast<float2*>(item_scalars(buf));
    float* scal = reinterpret_cast<float*>(item_scalars(buf) + 512);
    if (part == 0) {
      const int ta = 2 * lane, tb = ta + 1;
      const float ga = ta < it.live ? clamp_decay(a.g[(it.t0 + ta) * a.ldg + h]) : 0.f;
      const float gb = tb < it.live ? clamp_decay(a.g[(it.t0 + tb) * a.ldg + h]) : 0.f;
      double s = static_cast<double>(ga) + static_cast<double>(gb);
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += o;
      }
      Gs[ta] = decay_sum(s - static_cast<double>(gb));
      Gs[tb] = decay_sum(s);
    } else if (part == 1) {
      const float* ps = reinterpret_cast<const float*>(a.prep + hs * kPrepBytes + kPrepTri);
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (lane + 32 * i < 193) scal[lane + 32 * i] = ps[lane + 32 * i];
    } else {
      // the strips' shares of b (part 2) and dbeta, in strip order
      const float* p = a.dots + hs * (VD / 16) * 128 + (part - 2) * 64 + 2 * lane;
      float2 v = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < VD / 16; ++i) {
        const float2 x = *reinterpret_cast<const float2*>(p + i * 128);
        v.x += x.x;
        v.y += x.y;
      }
      *reinterpret_cast<float2*>(scal + 256 + (part - 2) * 64 + 2 * lane) = v;
    }
  };

  if (warp == 0) tmem_alloc(tslot, 512);
  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_init(full, 1);
    mbar_init(qk_full, 1);
    mbar_init(kk_done, 1);
    fence_barrier_init();
  }
  load_tiles(cur);
  if (warp < 4) load_scalars(cur, 0, warp);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t mine = tmem + (static_cast<uint32_t>(warp & 3) << 21);  // this warp's lanes
  const uint32_t aA = s0 + L::kA, a3 = s0 + L::kA3, qk = s0 + L::kQK, big = s0 + L::kBig;
  uint32_t phase = 0, arrived = 0;
  bool alive = true;
  auto wait_on = [&](uint64_t* b, uint32_t parity, unsigned bit) {
    if (alive) alive = mbar_spin(b, parity, a.err, bit);
  };
  auto wait_mma = [&]() {
    wait_on(bar, phase, kErrWaitMma);
    phase ^= 1u;
    tc_fence_after();
  };
  // a state in fragment order -> the tiles [v][k] of its first two parts, or of all three, four
  // 8 x 8 matrices a step
  auto state_tiles = [&](auto parts, const float4* x) {
#pragma unroll
    for (int i = 0; i < kPair; ++i) {
      const int pr = warp + i * (kGradThreads / 32);
      const int n = (pr % (KD / 16)) * 2 + (lane >> 4);  // this lane's row of a matrix
      const int v = (pr / (KD / 16)) * 16 + (lane & 15);
      const uint32_t at = ((v >> 6) * kKT + (n >> 3)) * kTileBytes + tile_off(v & 63, n & 7);
      const float2 y[4] = {make_float2(x[2 * i].x, x[2 * i].y), make_float2(x[2 * i].z, x[2 * i].w),
                           make_float2(x[2 * i + 1].x, x[2 * i + 1].y),
                           make_float2(x[2 * i + 1].z, x[2 * i + 1].w)};
      uint32_t p[3][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (decltype(parts)::value == 3) {
          uint32_t t[3];
          split3(y[e].x, y[e].y, t);
          p[0][e] = t[0];
          p[1][e] = t[1];
          p[2][e] = t[2];
        } else {
          split2(y[e].x, y[e].y, p[0][e], p[1][e]);
        }
      }
      stsm4(big + at, p[0]);
      stsm4(big + at + L::kState / 2, p[1]);
      if constexpr (decltype(parts)::value == 3) stsm4(qk + at, p[2]);
    }
  };

  float acc[kCols];  // dQ or dK of this row
  int buf = 0;
  uint32_t item = 0;  // parity of the barriers of q and k and of their product
  while (true) {
    const int h = cur.hk * group + cur.r;
    const long long hs = cur.slot * a.Hv + h;
    const float2* Gs = reinterpret_cast<const float2*>(item_scalars(buf));
    const float* scal = reinterpret_cast<const float*>(item_scalars(buf) + 512);
    if (cur.r == 0) {
#pragma unroll
      for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
    }
    float4 sv[2 * kPair];
    {
      const float4* S4 = reinterpret_cast<const float4*>(a.s_ws + hs * KD * VD * 4);
#pragma unroll
      for (int i = 0; i < kPair; ++i) {
        sv[2 * i] = S4[pair_off(i)];
        sv[2 * i + 1] = S4[pair_off(i) + 32];
      }
    }
    state_tiles(std::integral_constant<int, 3>{}, sv);
    cp_wait<0>();
    wait_on(full, arrived, kErrWaitFull);
    arrived ^= 1u;
    if (cur.live < kChunk) {
#pragma unroll
      for (int vt = 0; vt < kVT; ++vt)
        clear_rows<kGradThreads>(smem + L::kA + vt * 5 * kTileBytes, 128, 2, kTileBytes, cur.live, tid);
    }
    fence_smem_to_async();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      constexpr uint32_t idS = mma_desc<false, true, KD>(), idW = mma_desc<false, false, 64>();
      const uint64_t ad = smem_desc(aA, 16, 1024), sd = smem_desc(big, kTileBytes, 1024);
      const uint64_t a3d = smem_desc(a3, 16, 1024), s3d = smem_desc(qk, kTileBytes, 1024);
#pragma unroll
      for (int ks = 0; ks < VD / 16; ++ks) {
        const uint32_t at = (ks >> 2) * 5 * kTileBytes + (ks & 3) * 32;
        const uint32_t at3 = (ks >> 2) * 2 * kTileBytes + (ks & 3) * 32;
        const uint32_t st = (ks >> 2) * kKT * kTileBytes + (ks & 3) * 2048;
        // [do; dX hi], and as rows 64..127 what dX's second and third parts add
        const uint64_t x0 = desc_at(ad, at), x1 = desc_at(ad, at + kTileBytes), x2 = desc_at(a3d, at3);
        const uint64_t sh = desc_at(sd, st), sl = desc_at(sd, st + L::kState / 2);
        const uint64_t wh = desc_at(ad, at + 3 * kTileBytes), wl = desc_at(ad, at + 4 * kTileBytes);
        tc_mma(tmem + kD1, x0, sh, idS, ks > 0);
        tc_mma(tmem + kD1, x0, sl, idS, true);
        tc_mma(tmem + kD1, x0, desc_at(s3d, st), idS, true);
        tc_mma(tmem + kD1b, x1, sh, idS, ks > 0);
        tc_mma(tmem + kD1b, x1, sl, idS, true);
        tc_mma(tmem + kD1b, x2, sh, idS, true);
        tc_mma(tmem + kD2, x0, wh, idW, ks > 0);
        tc_mma(tmem + kD2, x0, wl, idW, true);
        tc_mma(tmem + kD2, x0, x2, idW, true);  // rows 0..63 there: W's third part
        tc_mma(tmem + kD2b, x1, wh, idW, ks > 0);
        tc_mma(tmem + kD2b, x1, wl, idW, true);
        tc_mma(tmem + kD2b, x2, wh, idW, true);
      }
      tc_commit(bar);
    }
    // meanwhile D, <S, D>, and where to go next
    float4 dd[2 * kPair];
    {
      const float4* D4 = reinterpret_cast<const float4*>(a.d_ws + hs * KD * VD * 4);
#pragma unroll
      for (int i = 0; i < kPair; ++i) {
        dd[2 * i] = D4[pair_off(i)];
        dd[2 * i + 1] = D4[pair_off(i) + 32];
      }
    }
    if (warp == kGradThreads / 32 - 1) {
      const GradItem it = next_item(cur);
      if (lane == 0) *next = it;
    }
    {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < 2 * kPair; ++i)
        v += sv[i].x * dd[i].x + sv[i].y * dd[i].y + sv[i].z * dd[i].z + sv[i].w * dd[i].w;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
      if (lane == 0) red[warp] = v;
    }
    wait_mma();
    // ---- q and k take the place of S's third part, D that of the other two
    if (tid == 0) load_qk(cur);
    state_tiles(std::integral_constant<int, 2>{}, dd);
    // E (key side) or F, and the second part of E before its range is used again
    float ef[16];
    tc_load16(mine + kD2 + cq * 16, ef);
    if (key_side) {
      float t[16];
      tc_load16(mine + kD2b + cq * 16, t);
#pragma unroll
      for (int i = 0; i < 16; ++i) ef[i] += t[i];
    }
    wait_on(qk_full, item, kErrWaitFull);
    if (cur.live < kChunk)
      clear_rows<kGradThreads>(smem + L::kQK, 128, 2 * kKT, kTileBytes, cur.live, tid);
    fence_smem_to_async();
    tc_fence_before();
    __syncthreads();
    const GradItem nxt = *next;
    const bool more = nxt.unit < units;
    if (tid == 0) {
      tc_fence_after();
      constexpr uint32_t idS = mma_desc<false, true, KD>(), idK = mma_desc<false, false, 64>();
      if (cur.r == 0) {
        const uint64_t qd = smem_desc(qk, 16, 1024);
#pragma unroll
        for (int ks = 0; ks < KD / 16; ++ks) {
          const uint32_t at = (ks >> 2) * 2 * kTileBytes + (ks & 3) * 32;
          tc_mma(tmem + kKK, desc_at(qd, at), desc_at(qd, at + kTileBytes), idK, ks > 0);
        }
      }
      tc_commit(kk_done);
      const uint64_t ad = smem_desc(aA, 16, 1024), sd = smem_desc(big, kTileBytes, 1024);
#pragma unroll
      for (int ks = 0; ks < VD / 16; ++ks) {
        const uint32_t at = (ks >> 2) * 5 * kTileBytes + (ks & 3) * 32;
        const uint32_t st = (ks >> 2) * kKT * kTileBytes + (ks & 3) * 2048;
        const uint64_t wh = desc_at(ad, at + 2 * kTileBytes);  // rows 64..127: W hi
        const uint64_t wl = desc_at(ad, at + 3 * kTileBytes);
        const uint64_t dh = desc_at(sd, st), dl = desc_at(sd, st + L::kState / 2);
        tc_mma(tmem + kD3, wh, dh, idS, ks > 0);
        tc_mma(tmem + kD3, wh, dl, idS, true);
        tc_mma(tmem + kD3, wl, dh, idS, true);
      }
      tc_commit(bar);
    }
    // ---- the pair terms: this row's 16 columns of Ph or -Eh, and of their products with q.k or
    // k.k; all zero above the diagonal
    uint32_t hi[8], lo[8];
    float run = 0.f;
    if (cq * 16 <= (warp & 1) * 32 + 31) {
      const float2 G = Gs[tok];
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = cq * 16 + i + e;
          float v = 0.f;
          if (key_side ? j < tok : j <= tok)
            v = (key_side ? -ef[i + e] : a.scale * ef[i + e]) * (decay_between(G, Gs[j]) * scal[j]);
          ef[i + e] = v;
        }
        split2(ef[i], ef[i + 1], hi[i / 2], lo[i / 2]);
      }
      wait_on(kk_done, item, kErrWaitMma);
      tc_fence_after();
      float kk[16];
      tc_load16(mine + kKK + cq * 16, kk);
      // running sums over the columns before, in the place of the terms
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float m = cq * 16 + i < tok ? ef[i] * kk[i] : 0.f;
        ef[i] = run;
        run += m;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) hi[i] = lo[i] = 0u;
#pragma unroll
      for (int i = 0; i < 16; ++i) ef[i] = 0.f;
      if (more) load_scalars(nxt, buf ^ 1, (warp - 8) >> 1);  // warps 8, 10, 12, 14
    }
    rowsum[cq * 128 + row] = run;
    // ---- the products with S: scale the row, add, and its product with q or k (a_i)
    {
      const float f = key_side ? -scal[64 + tok] : a.scale * scal[64 + tok];
      float dot = 0.f;
#pragma unroll
      for (int c = 0; c < kCols / 16; ++c) {
        float t[16];
        tc_load16(mine + kD1 + cq * kCols + c * 16, t);
        if (key_side) {
          float u[16];
          tc_load16(mine + kD1b + cq * kCols + c * 16, u);
#pragma unroll
          for (int i = 0; i < 16; ++i) t[i] += u[i];
        }
        const int col = cq * kCols + c * 16;
        const uint8_t* src = smem + L::kQK + ((col >> 6) * 2 + (key_side ? 1 : 0)) * kTileBytes;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint4 x = *reinterpret_cast<const uint4*>(src + tile_off(tok, ((col & 63) >> 3) + p));
          float xf[8];
          bf16x8_to_f32(x, xf);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float v = f * t[p * 8 + e];
            dot = fmaf(v, xf[e], dot);
            acc[c * 16 + p * 8 + e] += v;
          }
        }
      }
      adot[(cq * 2 + (key_side ? 1 : 0)) * 64 + tok] = dot;
    }
    wait_mma();       // W D^T is done: its tiles' places are free
    __syncthreads();  // and the sums of the row's other quarters are there
    {
      uint8_t* dst = smem + L::kBig + (key_side ? kTileBytes : 0);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t off = tile_off(tok, cq * 2 + p);
        *reinterpret_cast<uint4*>(dst + off) = make_uint4(hi[4 * p], hi[4 * p + 1], hi[4 * p + 2], hi[4 * p + 3]);
        *reinterpret_cast<uint4*>(dst + 2 * kTileBytes + off) =
            make_uint4(lo[4 * p], lo[4 * p + 1], lo[4 * p + 2], lo[4 * p + 3]);
      }
      float before = 0.f;
      for (int c = 0; c < cq; ++c) before += rowsum[c * 128 + row];
      float* M = reinterpret_cast<float*>(smem + L::kBig + 4 * kTileBytes) + row * kMLd + cq * 16;
#pragma unroll
      for (int i = 0; i < 16; ++i) M[i] = ef[i] + before;
    }
    fence_smem_to_async();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      constexpr uint32_t idP = mma_desc<false, true, KD>(), idT = mma_desc<true, true, KD>();
      const uint64_t qd = smem_desc(qk, 2 * kTileBytes, 1024), pd = smem_desc(big, 16, 1024);
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const uint32_t ph = part * 2 * kTileBytes;
        // transposed, as rows 64..127 (rows 0..63, not read, are a q tile's)
        const uint64_t tp = smem_desc(qk, big + ph - qk, 1024);
        const uint64_t te = smem_desc(qk, big + ph + kTileBytes - qk, 1024);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint64_t q = desc_at(qd, ks * 2048), k = desc_at(qd, kTileBytes + ks * 2048);
          tc_mma(tmem + kD4, desc_at(pd, ph + ks * 32), k, idP, ks + part > 0);
          tc_mma(tmem + kD5, desc_at(tp, ks * 2048), q, idT, ks + part > 0);
          tc_mma(tmem + kD5, desc_at(te, ks * 2048), k, idT, true);
        }
      }
      tc_commit(bar);
    }
    // ---- meanwhile the next item's tiles and S, W D^T, and the sums of dg over i >= t
    if (more) {
      load_tiles(nxt);
      if (tid == 32) {  // S and D are read through registers, q and k wait for their place: into L2
        const long long ns = nxt.slot * a.Hv + nxt.hk * group + nxt.r;
        bulk_prefetch_l2(a.s_ws + ns * KD * VD * 4, KD * VD * 4);
        bulk_prefetch_l2(a.d_ws + ns * KD * VD * 4, KD * VD * 4);
        if (nxt.r == 0) {
#pragma unroll
          for (int kt = 0; kt < kKT; ++kt) {
            tma_prefetch_2d(&maps.q, nxt.hk * KD + kt * 64, static_cast<int>(nxt.t0));
            tma_prefetch_2d(&maps.k, nxt.hk * KD + kt * 64, static_cast<int>(nxt.t0));
          }
        }
      }
    }
    if (key_side) {
      const float f = scal[128 + tok] * scal[tok];
#pragma unroll
      for (int c = 0; c < kCols / 16; ++c) {
        float t[16];
        tc_load16(mine + kD3 + cq * kCols + c * 16, t);
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[c * 16 + i] = fmaf(f, t[i], acc[c * 16 + i]);
      }
    }
    {
      // column t of the running sums: rows i >= t of 16 rows of Ph's or Eh's terms
      const int t = tid & 63, part = tid >> 6;
      const int i0 = (part & 3) * 16, r0 = (part >> 2) * 64 + i0;
      const float* M = reinterpret_cast<const float*>(smem + L::kBig + 4 * kTileBytes) + r0 * kMLd + t;
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) v += i0 + i >= t ? M[i * kMLd] : 0.f;
      vpart[part * 64 + t] = v;
    }
    __syncthreads();
    if (warp == 0) {
      // two tokens a lane: sums of a over i >= t and of b over j < t
      float sd = 0.f, sa[2], pb[2], v[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kGradThreads / 32; ++i) sd += red[i];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int t = lane + 32 * u;
        sa[u] = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          sa[u] += adot[c * 64 + t];
          v[u] += vpart[c * 64 + t];
        }
        pb[u] = scal[256 + t];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const float x = __shfl_down_sync(0xffffffffu, sa[u], off);
          const float y = __shfl_up_sync(0xffffffffu, pb[u], off);
          if (lane + off < 32) sa[u] += x;
          if (lane >= off) pb[u] += y;
        }
      }
      sa[0] += __shfl_sync(0xffffffffu, sa[1], 0);
      const float first = __shfl_sync(0xffffffffu, pb[0], 31);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float incl = __shfl_up_sync(0xffffffffu, pb[u], 1);
        const float before = (lane > 0 ? incl : 0.f) + (u > 0 ? first : 0.f);
        const int tk = lane + 32 * u;
        if (tk < cur.live) {
          const long long t = cur.t0 + tk;
          a.dg[t * a.lddg + h] = scal[192] * sd + v[u] + sa[u] + before;
          const float db = scal[320 + tk];
          if (a.beta_fp32)
            reinterpret_cast<float*>(a.dbeta)[t * a.lddbeta + h] = db;
          else
            reinterpret_cast<__nv_bfloat16*>(a.dbeta)[t * a.lddbeta + h] = __float2bfloat16_rn(db);
        }
      }
    }
    wait_mma();
#pragma unroll
    for (int c = 0; c < kCols / 16; ++c) {
      float t[16];
      tc_load16(mine + kD4 + cq * kCols + c * 16, t);
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[c * 16 + i] += t[i];
      if (key_side) {
        tc_load16(mine + kD5 + cq * kCols + c * 16, t);
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[c * 16 + i] += t[i];
      }
    }
    tc_fence_before();
    if (cur.r + 1 == group) {
      // dq and dk through shared memory, so that a row leaves in whole lines
      uint8_t* out = smem + L::kBig;
#pragma unroll
      for (int i = 0; i < kCols / 8; ++i) {
        const int col = cq * kCols + i * 8;
        *reinterpret_cast<uint4*>(out + ((key_side ? kKT : 0) + (col >> 6)) * kTileBytes +
                                  tile_off(tok, (col & 63) >> 3)) = f32x8_to_bf16(acc + i * 8);
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2 * kKT; ++i) {
        const int r = tid >> 3, p = tid & 7;
        if (r < cur.live) {
          const bool dk = i >= kKT;
          uint16_t* dst = dk ? a.dk + (cur.t0 + r) * a.lddk : a.dq + (cur.t0 + r) * a.lddq;
          *reinterpret_cast<uint4*>(dst + static_cast<long long>(cur.hk) * KD + (i % kKT) * 64 + p * 8) =
              *reinterpret_cast<const uint4*>(out + i * kTileBytes + tile_off(r, p));
        }
      }
    }
    __syncthreads();
    if (!more) break;
    buf ^= 1;
    item ^= 1u;
    cur = nxt;
  }
  if (warp == 0) tmem_free(tmem, 512);
}

}  // namespace gnorm
