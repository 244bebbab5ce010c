// delta_step.cuh -- one token of each sequence through the gated delta rule, the states kept
// in a pool in device memory and updated in place (sm_100a).
//
//   u = beta (v - e^g S^T k)    S <- e^g S + k u^T    o = scale (e^g S^T q + (q.k) u)
//
// (o in this form needs S as it was, so S^T k and S^T q come from one pass and one reduction.)
// Bound by HBM: the state is read and written once, 8 K V bytes a head against 2 (2 K + 2 V)
// of everything else.  A CTA holds VT columns of one head's state in registers: float4 loads
// of whole rows, all issued before the first use, a fixed-order sum over the row groups
// through shared memory, stores straight from the registers.  256 rows x 32 heads of 128 x 128
// (1.08 GB): 183 us, 5.9 TB/s, 91% of the measured copy.  4 rows x 16 heads (8.4 MB): 4.8 us a
// step in a graph of steps, 6 as eager calls; what bounds it are loads that wait for one another:
// the slot, then the state, q and k, then behind two barriers g, beta and v.
#pragma once

#include "delta_common.cuh"

namespace gnorm {

constexpr int kStepThreads = 256;

struct StepArgs {
  const uint16_t *q = nullptr, *k = nullptr, *v = nullptr;
  const float* g = nullptr;
  const void* beta = nullptr;
  int beta_fp32 = 0;
  long long ldq = 0, ldk = 0, ldv = 0, ldg = 0, ldbeta = 0, ldo = 0;
  int Hk = 0, Hv = 0, B = 0;
  float scale = 1.f;
  const int* slots = nullptr;  // [B] or nullptr: row b uses state b
  int pool = 0;
  float* state = nullptr;  // [pool, Hv, K, V], lds values from one slot to the next
  long long lds = 0;
  uint16_t* o = nullptr;
};

template <int KD, int VD, int VT>
__global__ void __launch_bounds__(kStepThreads) delta_step_kernel(const __grid_constant__ StepArgs a) {
  constexpr int kLanes = VT / 4;                   // threads along a row
  constexpr int kGroups = kStepThreads / kLanes;   // row groups
  constexpr int kRows = KD / kGroups;              // rows per thread
  static_assert(kRows >= 1, "a row group has a row");
  __shared__ __align__(16) float part[2][kGroups][VT];
  __shared__ __align__(16) float sk[KD], sq[KD];
  __shared__ float s_qk[KD / 32];
  __shared__ int s_next;
  const int tid = threadIdx.x;
  const int lane4 = tid % kLanes, grp = tid / kLanes;
  const int v0 = blockIdx.x * VT, h = blockIdx.y;
  const int hk = h / (a.Hv / a.Hk);
  int row = blockIdx.z;
  grid_dependency_wait();
  allow_dependent_launch();
  const int slot = a.slots != nullptr ? a.slots[row] : row;
  if (slot < 0 || slot >= a.pool) {  // a padded row: no state, output zero
    if (tid < VT) a.o[row * a.ldo + static_cast<long long>(h) * VD + v0 + tid] = 0;
    return;
  }
  float4 s[kRows];
  float* sp = a.state + slot * a.lds + static_cast<long long>(h) * KD * VD + v0 + lane4 * 4;
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    s[i] = *reinterpret_cast<const float4*>(sp + static_cast<long long>(grp + i * kGroups) * VD);
  // Rows that name the same slot are tokens of one sequence, in row order: the CTA of the
  // first such row takes them one after another, those of the others leave.
  if (a.slots != nullptr) {
    bool earlier = false;
    for (int i = tid; i < row; i += kStepThreads) earlier |= a.slots[i] == slot;
    if (__syncthreads_or(earlier)) return;
  }
  while (true) {
    __syncthreads();
    if (tid == 0) s_next = a.B;
    if (tid < KD) {
      const float kv = __uint_as_float(static_cast<uint32_t>(a.k[row * a.ldk + static_cast<long long>(hk) * KD + tid]) << 16);
      const float qv = __uint_as_float(static_cast<uint32_t>(a.q[row * a.ldq + static_cast<long long>(hk) * KD + tid]) << 16);
      sk[tid] = kv;
      sq[tid] = qv;
      float d = kv * qv;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
      if ((tid & 31) == 0) s_qk[tid >> 5] = d;
    }
    __syncthreads();
    if (a.slots != nullptr) {
      for (int i = row + 1 + tid; i < a.B; i += kStepThreads)
        if (a.slots[i] == slot) {
          atomicMin(&s_next, i);
          break;
        }
    }
    float4 pk = make_float4(0.f, 0.f, 0.f, 0.f), pq = pk;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float kv = sk[grp + i * kGroups], qv = sq[grp + i * kGroups];
      pk.x = fmaf(kv, s[i].x, pk.x);
      pk.y = fmaf(kv, s[i].y, pk.y);
      pk.z = fmaf(kv, s[i].z, pk.z);
      pk.w = fmaf(kv, s[i].w, pk.w);
      pq.x = fmaf(qv, s[i].x, pq.x);
      pq.y = fmaf(qv, s[i].y, pq.y);
      pq.z = fmaf(qv, s[i].z, pq.z);
      pq.w = fmaf(qv, s[i].w, pq.w);
    }
    *reinterpret_cast<float4*>(&part[0][grp][lane4 * 4]) = pk;
    *reinterpret_cast<float4*>(&part[1][grp][lane4 * 4]) = pq;
    __syncthreads();
    const float w = expf(clamp_decay(a.g[row * a.ldg + h]));
    const long long bi = row * a.ldbeta + h;
    const float beta = a.beta_fp32
                           ? reinterpret_cast<const float*>(a.beta)[bi]
                           : __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(a.beta)[bi]) << 16);
    float qk = 0.f;
#pragma unroll
    for (int i = 0; i < KD / 32; ++i) qk += s_qk[i];
    float4 tk = make_float4(0.f, 0.f, 0.f, 0.f), tq = tk;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(&part[0][i][lane4 * 4]);
      tk.x += x.x;
      tk.y += x.y;
      tk.z += x.z;
      tk.w += x.w;
    }
    if (grp == 0) {
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(&part[1][i][lane4 * 4]);
        tq.x += x.x;
        tq.y += x.y;
        tq.z += x.z;
        tq.w += x.w;
      }
    }
    const uint2 vv = *reinterpret_cast<const uint2*>(a.v + row * a.ldv + static_cast<long long>(h) * VD + v0 + lane4 * 4);
    const float4 u = make_float4(beta * fmaf(-w, tk.x, bf_lo(vv.x)), beta * fmaf(-w, tk.y, bf_hi(vv.x)),
                                 beta * fmaf(-w, tk.z, bf_lo(vv.y)), beta * fmaf(-w, tk.w, bf_hi(vv.y)));
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float kv = sk[grp + i * kGroups];
      s[i].x = fmaf(kv, u.x, w * s[i].x);
      s[i].y = fmaf(kv, u.y, w * s[i].y);
      s[i].z = fmaf(kv, u.z, w * s[i].z);
      s[i].w = fmaf(kv, u.w, w * s[i].w);
    }
    if (grp == 0) {
      uint2 out;
      out.x = pack_bf16x2(a.scale * fmaf(qk, u.x, w * tq.x), a.scale * fmaf(qk, u.y, w * tq.y));
      out.y = pack_bf16x2(a.scale * fmaf(qk, u.z, w * tq.z), a.scale * fmaf(qk, u.w, w * tq.w));
      *reinterpret_cast<uint2*>(a.o + row * a.ldo + static_cast<long long>(h) * VD + v0 + lane4 * 4) = out;
    }
    if (a.slots == nullptr) break;
    const int next = s_next;  // written before the last barrier
    if (next >= a.B) break;
    row = next;
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i)
    *reinterpret_cast<float4*>(sp + static_cast<long long>(grp + i * kGroups) * VD) = s[i];
}

}  // namespace gnorm
