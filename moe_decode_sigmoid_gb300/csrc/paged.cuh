// paged.cuh — device helpers the paged KV-cache kernels share: a sequence's
// rows and lengths with everything the host could not check kept in bounds,
// page look-ups, and E4M3 conversions.
#pragma once

#include "common.cuh"
#include "paged.h"

namespace flint {
namespace pg {

// One sequence's rows: token rows q0 .. q0 + n - 1 at positions first ..
// len - 1 of its cache (first = len - n is negative if kv_len is short).
struct Seq {
  int q0, n, len, first;
};
__device__ __forceinline__ Seq load_seq(const PagedView& b, int s) {
  const int a0 = b.q_start[s], a1 = b.q_start[s + 1], l = b.kv_len[s];
  Seq q;
  q.q0 = min(max(a0, 0), b.n_tokens);
  q.n = min(max(a1, q.q0), b.n_tokens) - q.q0;
  q.len = (int)min((long long)max(l, 0), (long long)b.max_pages << b.page_shift);
  q.first = q.len - q.n;
  return q;
}

// Cache row of a sequence's token at position pos in [0, len), or -1 if its
// page is not one of the cache's.
__device__ __forceinline__ int cache_row(const PagedView& b, int s, int pos) {
  const int page = __ldg(b.page_table + (size_t)s * b.max_pages + (pos >> b.page_shift));
  if ((unsigned)page >= (unsigned)b.n_pages) return -1;
  return (page << b.page_shift) + (pos & ((1 << b.page_shift) - 1));
}

// Two E4M3 codes (low 16 bits, low byte first) -> f16x2: exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(r) : "r"(two));
  return r;
}
// lo, hi -> two E4M3 codes, nearest (ties to even), saturating; NaN stays NaN.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// lo, hi -> two bf16, nearest (ties to even).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h2) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}

}  // namespace pg
}  // namespace flint
