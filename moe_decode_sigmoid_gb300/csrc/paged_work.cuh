// paged_work.cuh — the paged attention's workspace (partial results of rows
// that several CTAs share, and the tickets that find the last of them) and how
// a finished row is written.
#pragma once

#include "paged.cuh"

namespace flint {
namespace pg {

constexpr int MAX_CTAS = 160;  // CTAs of an attention launch (one per SM; GB300 has 152)

// Workspace: a ticket per CTA, then two slots per CTA: one for a row that began
// in an earlier CTA's share and one for a row that goes on in the next one's.
constexpr size_t WS_TICKETS = 4096;
static_assert(MAX_CTAS * 4 <= WS_TICKETS, "tickets fit");

// A slot of the next-token kernel: 8 maxima, 8 sums, 128 x 8 outputs.
constexpr int DEC_ML = 16, DEC_O = HD * 8, DEC_SLOT = DEC_ML + DEC_O;
// Fewest granules in a CTA's share, and the longest row that is never cut.
constexpr int DEC_MIN_SHARE = 16, DEC_WHOLE = 64;

__host__ __device__ constexpr size_t attn_ws_bytes() {
  return WS_TICKETS + sizeof(float) * 2 * MAX_CTAS * (size_t)DEC_SLOT;
}

__device__ __forceinline__ uint32_t* ws_tickets(void* ws) { return static_cast<uint32_t*>(ws); }
__device__ __forceinline__ float* dec_slot(void* ws, int cta, bool begins) {
  return reinterpret_cast<float*>(static_cast<char*>(ws) + WS_TICKETS) +
         (size_t)(2 * cta + (begins ? 1 : 0)) * DEC_SLOT;
}

// Output elements d, d + 1 of a head from its maximum, sum and unscaled
// outputs, with the head's sink in the denominator.
__device__ __forceinline__ void dec_store(const PagedAttnArgs& a, int row, int head, int d, float m,
                                          float l, float o0, float o1) {
  const float sink = a.sinks ? a.sinks[head] * 1.4426950408889634f : -INFINITY;
  const float mm = fmaxf(m, sink);
  const float f = m > -INFINITY ? exp2f(m - mm) : 0.0f;
  const float den = fmaf(l, f, sink > -INFINITY ? exp2f(sink - mm) : 0.0f);
  const float inv = den == 0.0f ? 0.0f : f / den;  // NaN stays NaN
  const size_t nq = (size_t)a.b.nkv * a.b.group;
  *reinterpret_cast<uint32_t*>(a.out + ((size_t)row * nq + head) * HD + d) =
      pack_bf2(o0 * inv, o1 * inv);
}

}  // namespace pg
}  // namespace flint
