// checks.h -- argument checks shared by the extern "C" entry points (internal, host only).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "gnorm.h"
#include "plan.h"

namespace gnorm {

// Properties of the current device that launches depend on, looked up once per device.
struct DeviceInfo {
  bool ready = false;
  int num_sms = 0;
  int smem_optin = 0;
  unsigned* err_word = nullptr;
};
int device_info(DeviceInfo* out);

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

inline bool use_pdl() { return get_tuning().disable_pdl == 0; }

// A memory region an argument covers: a plain byte span, or a [rows, cols] matrix
// with row stride `ld` elements.
struct Region {
  const void* p;
  size_t bytes;     // whole extent
  bool is_mat;
  int64_t rows, cols, ld;
  int elem;  // bytes of an element (is_mat)
};

inline Region span(const void* p, size_t bytes) { return Region{p, bytes, false, 0, 0, 0, 1}; }
inline Region mat(const void* p, int64_t rows, int64_t cols, int64_t ld, int elem = 2) {
  const size_t bytes =
      rows > 0 ? static_cast<size_t>((rows - 1) * ld + cols) * static_cast<size_t>(elem) : 0;
  return Region{p, bytes, true, rows, cols, ld, elem};
}

inline int64_t floor_div(int64_t a, int64_t b) { return a / b - ((a % b != 0) && ((a < 0) != (b < 0))); }

// Exact for two matrices with the same stride in bytes, of any widths (columns of one wider
// buffer, which interleave row by row); whole-extent overlap otherwise.
inline bool overlaps(const Region& a, const Region& b) {
  if (a.p == nullptr || b.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), a1 = a0 + a.bytes;
  const uintptr_t b0 = reinterpret_cast<uintptr_t>(b.p), b1 = b0 + b.bytes;
  if (!(a0 < b1 && b0 < a1)) return false;
  const int64_t L = a.ld * a.elem, na = a.cols * a.elem, nb = b.cols * b.elem;
  // rows of at most a stride each: a row of b meets one or two rows of a
  if (!(a.is_mat && b.is_mat && L == b.ld * b.elem && na <= L && nb <= L)) return true;
  const int64_t d = static_cast<int64_t>(b0 - a0);  // two's complement difference
  const int64_t q = floor_div(d, L), delta = d - q * L;  // b's row j starts in a's row q + j
  auto rows_meet = [&](int64_t off) { return off < a.rows && off + b.rows > 0; };
  if (delta < na && rows_meet(q)) return true;          // b's row starts inside that row
  if (delta + nb > L && rows_meet(q + 1)) return true;  // or runs into a's next row
  return false;
}

// Every output region against every input region and every other output region.
inline bool any_alias(const Region* in, int n_in, const Region* out, int n_out) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlaps(out[i], in[j])) return true;
    for (int j = i + 1; j < n_out; ++j)
      if (overlaps(out[i], out[j])) return true;
  }
  return false;
}

// Row stride in elements: 0 means packed (N); a stride must hold a row and keep rows
// 16-byte aligned.
inline int check_ld(int64_t* ld, int64_t N) {
  if (*ld == 0) *ld = N;
  if (*ld < N) return GNORM_ERR_SHAPE;
  if (*ld % 8 != 0) return GNORM_ERR_ALIGN;
  return GNORM_OK;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace gnorm
