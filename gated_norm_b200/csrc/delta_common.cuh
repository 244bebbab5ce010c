// delta_common.cuh -- tiles, tensor-core fragments and argument blocks shared by the kernels
// of the gated delta rule (sm_100a).
//
// The recurrence, per sequence and value head, with S of K x V values:
//
//   S_t = e^{g_t} S_{t-1} + k_t u_t^T    u_t = beta_t (v_t - e^{g_t} S_{t-1}^T k_t)
//   o_t = scale S_t^T q_t
//
// and in chunks of C = 64 tokens (G the running sum of g inside the chunk, gamma_i = e^{G_i},
// lambda_j = e^{G_C - G_j}, D_ij = e^{G_i - G_j}; S the state before the chunk, S' after it):
//
//   Kb_ij = D_ij k_i.k_j (j < i)    P_ij = D_ij q_i.k_j (j <= i)    N = (I + Kb diag(beta))^-1 Kb
//   X = V - gamma K S    W = X - N (beta X)    Y = beta W
//   O = scale (gamma Q S + P Y)    S' = e^{G_C} S + K^T (lambda Y)
//
// N depends on the keys alone, so it and P are computed for all chunks at once
// (delta_prep_kernel); only the products with S run chunk after chunk (delta_scan kernels).
//
// Precision.  q, k, v and do are BF16, so they enter the tensor cores exactly.  States, N, P,
// X, W and their gradients are FP32 values: as a matrix operand each is cut into BF16 parts,
// p0 = bf16(x), p1 = bf16(x - p0), p2 = bf16(x - p0 - p1), and a product against an exact
// operand takes an instruction per part, one of two cut operands the six products whose
// weight is 2^-24 or more.  Three parts hold all 24 bits of an FP32 value, and with FP32 sums
// the chunked form is as exact as FP32 arithmetic.  Two parts (16 to 17 bits) are not enough
// for a state: where the terms of a sum take each other back (one key repeated), it was 4e-4
// off.  Two parts remain where a product only reaches a BF16 output (o, dq, dk), whose half step of
// 2^-8 is 100 times what they leave out.
#pragma once

#include "device_common.cuh"

namespace gnorm {

constexpr int kChunk = 64;               // tokens of a chunk
constexpr int kTileBytes = 64 * 64 * 2;  // a 64 x 64 BF16 tile
// e^g of any g below this is zero in FP32 whatever it multiplies: clamping there keeps sums
// of g finite and their differences exact for g = -inf or the type's lowest value.
constexpr float kMinLogDecay = -200.f;

// ---- 64 x 64 BF16 tiles: rows of 128 bytes, 16-byte pieces XOR-swizzled by the row, so the
// eight rows of an ldmatrix hit eight different bank groups.
__device__ __forceinline__ uint32_t tile_off(int row, int piece) {
  return static_cast<uint32_t>(row * 128 + ((piece ^ (row & 7)) << 4));
}

__device__ __forceinline__ void ldsm4(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t r[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void stsm4(uint32_t addr, const uint32_t r[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t addr, const uint32_t r[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
// D += A B, m16n8k16, BF16 operands, FP32 sums.
__device__ __forceinline__ void mma16816(float d[4], const uint32_t a[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Addresses of one lane for the 16 x 16 block at (row0, col0) of a tile, by what the four
// 8 x 8 matrices become:
// B operand whose columns n are the tile's rows (plain ldmatrix): r[0], r[1] are n 0..7,
// r[2], r[3] are n 8..15 of the k16 at col0.
__device__ __forceinline__ uint32_t addr_b(uint32_t tile, int row0, int col0, int lane) {
  return tile + tile_off(row0 + (lane & 7) + ((lane >> 4) << 3), (col0 >> 3) + ((lane >> 3) & 1));
}
// B operand whose k are the tile's rows (transposing ldmatrix): r[0], r[1] are columns
// col0..+7, r[2], r[3] columns col0+8..+15 of the k16 at row0.
__device__ __forceinline__ uint32_t addr_bt(uint32_t tile, int row0, int col0, int lane) {
  return tile + tile_off(row0 + (lane & 15), (col0 >> 3) + (lane >> 4));
}
// A operand, rows of the tile (plain ldmatrix).
__device__ __forceinline__ uint32_t addr_a(uint32_t tile, int row0, int col0, int lane) {
  return tile + tile_off(row0 + (lane & 15), (col0 >> 3) + (lane >> 4));
}
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// What a BF16 pair leaves of two FP32 values (exact), one packed operation.
__device__ __forceinline__ float2 left_of(float2 x, uint32_t p) {
  return fma2(make_float2(bf_lo(p), bf_hi(p)), splat2(-1.f), x);
}

// Two FP32 values as BF16 pairs: hi, and lo = what hi leaves.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x, y);
  const float2 r = left_of(make_float2(x, y), hi);
  lo = pack_bf16x2(r.x, r.y);
}

// Two FP32 values as BF16 pairs: three parts, 24 bits.
__device__ __forceinline__ void split3(float x, float y, uint32_t p[3]) {
  p[0] = pack_bf16x2(x, y);
  float2 r = left_of(make_float2(x, y), p[0]);
  p[1] = pack_bf16x2(r.x, r.y);
  r = left_of(r, p[1]);
  p[2] = pack_bf16x2(r.x, r.y);
}

// 16-byte asynchronous copy, zero-filled where `live` is false (nothing is read then).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  const int n = live ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Tensor maps over [T, heads x dim] tensors: boxes of 64 tokens, of 64 columns in the layout of
// tile_off, or of a scan's strips of columns as plain rows.  Rows behind the tensor's end arrive
// as zeros; rows behind a sequence's end are the next one's and are cleared after they arrive.
struct DeltaMaps {
  CUtensorMap q, k;         // tiles
  CUtensorMap v, do_strip;  // strips: v (forward scans), do (backward scan)
  CUtensorMap do_tile, dv;  // tiles
};

// ---- sequences and chunk slots.  Chunk c of sequence b has the slot base(b) + c with
// base(b) = start(b) / 64 + b: ceil(len / 64) slots always fit before base(b + 1), so no sum
// over the sequences is needed.  The tokens behind the last sequence are "sequence" B.
struct DeltaSeqs {
  const int* cu = nullptr;  // [B + 1] on the device, or nullptr: B sequences of seqlen tokens
  int B = 0;
  long long seqlen = 0;
  long long T = 0;
};

__device__ __forceinline__ long long seq_start(const DeltaSeqs& s, int b) {
  if (s.cu == nullptr) return static_cast<long long>(b) * s.seqlen;
  long long v = s.cu[b];
  v = v < 0 ? 0 : v;
  return v > s.T ? s.T : v;
}
__device__ __forceinline__ long long seq_end(const DeltaSeqs& s, int b) {
  if (b >= s.B) return s.T;
  const long long lo = seq_start(s, b), hi = seq_start(s, b + 1);
  return hi < lo ? lo : hi;
}
__device__ __forceinline__ long long seq_base(const DeltaSeqs& s, int b) {
  return seq_start(s, b) / kChunk + b;
}
// The sequence (B for the tokens behind the last one) that slot belongs to; a search 32 ways
// wide, every lane of the warp calls.
__device__ __forceinline__ int seq_of_slot(const DeltaSeqs& s, long long slot, int lane) {
  int lo = 0, hi = s.B + 1;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool le = at < hi && seq_base(s, at) <= slot;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    const int last = m == 0 ? 0 : 31 - __clz(m);
    lo += last * step;
    hi = hi < lo + step ? hi : lo + step;
  }
  return lo;
}
// The z-th longest of up to 32 sequences (more: the z-th), so that the CTAs that take longest
// start first; every lane of the warp calls.
__device__ __forceinline__ int seq_by_length(const DeltaSeqs& s, int z, int lane) {
  if (s.cu == nullptr || s.B > 32) return z;
  const long long len = lane < s.B ? seq_end(s, lane) - seq_start(s, lane) : -1;
  int rank = 0;
  for (int j = 0; j < s.B; ++j) {
    const long long other = __shfl_sync(0xffffffffu, len, j);
    rank += other > len || (other == len && j < lane) ? 1 : 0;
  }
  return __ffs(__ballot_sync(0xffffffffu, lane < s.B && rank == z)) - 1;
}
inline long long delta_slots(long long T, long long B) { return T / kChunk + B + 1; }

// Per (slot, value head): N and P in three parts each, then beta, gamma, lambda [64] and
// e^{G_C}.  Both are lower triangular; a part holds the 8 x 8 matrices (128 contiguous bytes,
// an ldmatrix row group) of the 16 x 16 blocks on and below the diagonal: for each 8-row tile t
// the column tiles 0 .. 2 (t / 2) + 1.
GNORM_HD constexpr int tri_row(int t) { return 2 * (t / 2) * (t / 2 + 1) + (t & 1) * 2 * (t / 2 + 1); }
constexpr int kTriBytes = 40 * 128;  // tri_row(8) matrices
__device__ __forceinline__ uint32_t tri_off(int i, int j) {  // element (i, j)
  return static_cast<uint32_t>((tri_row(i >> 3) + (j >> 3)) * 128 + (i & 7) * 16 + (j & 7) * 2);
}
constexpr int kTriGrid = 8192;  // a part in an 8 x 8 grid of matrices, an operand of tcgen05
constexpr long long kPrepTri = 6LL * kTriBytes;
constexpr long long kPrepScal = 1024;
constexpr long long kPrepBytes = kPrepTri + kPrepScal;

struct DeltaArgs {
  DeltaSeqs seq;
  const uint16_t *q = nullptr, *k = nullptr, *v = nullptr;
  const float* g = nullptr;
  const void* beta = nullptr;
  int beta_fp32 = 0;
  long long ldq = 0, ldk = 0, ldv = 0, ldg = 0, ldbeta = 0;
  int Hk = 0, Hv = 0, V = 0;
  float scale = 1.f;
  const float* state_in = nullptr;  // [B, Hv, K, V]
  float* state_out = nullptr;
  uint16_t* o = nullptr;
  long long ldo = 0;
  uint8_t* prep = nullptr;  // [slots, Hv] of kPrepBytes
  // backward
  const uint16_t* dout = nullptr;  // do
  long long lddo = 0;
  uint8_t* s_ws = nullptr;  // [slots, Hv]: S before the chunk, FP32, in fragment order
  uint8_t* d_ws = nullptr;  // [slots, Hv]: the gradient of S after the chunk, likewise
  uint8_t* w_ws = nullptr;  // [slots, Hv, V/16]: W's strips (delta_scan.cuh)
  uint8_t* x_ws = nullptr;  // [slots, Hv]: tiles of dX's second and third parts (dv holds the first)
  float* dots = nullptr;    // [slots, Hv, V/16, 2, 64]: each strip's share of b and dbeta
  const float* dstate_out = nullptr;
  float* dstate_in = nullptr;
  uint16_t *dq = nullptr, *dk = nullptr, *dv = nullptr;
  float* dg = nullptr;
  void* dbeta = nullptr;
  long long lddq = 0, lddk = 0, lddv = 0, lddg = 0, lddbeta = 0;
  unsigned* err = nullptr;  // the device error word
  long long slots = 0;
  int sms = 1;  // of the device
  // rows behind the last sequence that are to be zeroed
  int n_zero = 0;
  uint8_t* zero_p[5] = {};
  long long zero_ld[5] = {};  // bytes
  int zero_row[5] = {};       // bytes
};

__device__ __forceinline__ float load_beta(const DeltaArgs& a, long long tok, int h) {
  const long long i = tok * a.ldbeta + h;
  return a.beta_fp32 ? reinterpret_cast<const float*>(a.beta)[i]
                     : __uint_as_float(
                           static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(a.beta)[i]) << 16);
}
__device__ __forceinline__ float clamp_decay(float g) { return g < kMinLogDecay ? kMinLogDecay : g; }

// The running sum of g inside a chunk as two FP32 values in units of log2: differences of far
// terms keep their digits without FP64 in the inner loops.
__device__ __forceinline__ float2 decay_sum(double G) {
  const double x = G * 1.4426950408889634;
  const float hi = static_cast<float>(x);
  return make_float2(hi, static_cast<float>(x - static_cast<double>(hi)));
}
// e^{G_i - G_j}
__device__ __forceinline__ float decay_between(float2 i, float2 j) {
  return exp2f((i.x - j.x) + (i.y - j.y));
}

// Copies `live` rows of `cols` (a multiple of 64) BF16 values into swizzled tiles (one per 64
// columns), zero below; kThreads threads take part.
template <int kThreads>
__device__ __forceinline__ void load_rows(uint32_t dst, const uint16_t* src, long long ld, int cols,
                                          int live, int tid) {
  const int per = cols >> 3;
  for (int i = tid; i < kChunk * per; i += kThreads) {
    const int row = i / per, p = i - row * per;
    const bool ok = row < live;
    cp16(dst + (p >> 3) * kTileBytes + tile_off(row, p & 7), src + (ok ? row * ld : 0) + p * 8, ok);
  }
}
// Clears rows live .. 63 of `bytes` bytes, `pitch` apart, `n` tiles of `tile` bytes; kThreads
// threads take part.
template <int kThreads>
__device__ __forceinline__ void clear_rows(uint8_t* p, int bytes, int n, int tile, int live, int tid) {
  const int per = bytes >> 4, total = (kChunk - live) * per * n;
  for (int i = tid; i < total; i += kThreads) {
    const int c = i / per, x = i - c * per;
    const int t = c / (kChunk - live), r = live + c - t * (kChunk - live);
    *reinterpret_cast<uint4*>(p + t * tile + r * bytes + x * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
}
}  // namespace gnorm
