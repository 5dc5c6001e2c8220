// paged_work.cuh — the paged attention's workspace (partial results of rows
// that several CTAs share, and the tickets that find the last of them) and how
// a finished row is scaled.
#pragma once

#include "paged.cuh"

namespace flint {
namespace pg {

constexpr int MAX_CTAS = 160;  // CTAs of an attention launch (one per SM; GB300 has 152)

// Workspace: a ticket per CTA and an error word, then two slots per CTA: one
// for a row (or item) that began in an earlier CTA's share and one for one that
// goes on in the next one's.
constexpr size_t WS_HEAD = 4096, WS_ERROR = WS_HEAD - 4;
static_assert(MAX_CTAS * 4 <= WS_ERROR, "tickets fit");

// A slot of the next-token kernel: 8 maxima, 8 sums, 128 x 8 outputs.
constexpr int DEC_ML = 16, DEC_O = HD * 8, DEC_SLOT = DEC_ML + DEC_O;
// Fewest granules in a CTA's share, and the longest row that is never cut.
constexpr int DEC_MIN_SHARE = 16, DEC_WHOLE = 64;

// A slot of the prompt kernel: two tiles of 128 maxima, 128 sums and 128 x 128
// outputs.
constexpr int PR_TILE = 128 * (2 + HD), PR_SLOT = 2 * PR_TILE;
// Fewest key tiles in a CTA's share, the longest item that is never cut, and how
// far a cut moves to an item's end at most: what a join costs, in tiles.
constexpr int PR_MIN_SHARE = 4, PR_WHOLE = 6, PR_MARGIN = 3;

__host__ __device__ constexpr size_t attn_ws_bytes() {
  return WS_HEAD + sizeof(float) * 2 * MAX_CTAS * (size_t)PR_SLOT;
}

__device__ __forceinline__ uint32_t* ws_tickets(void* ws) { return static_cast<uint32_t*>(ws); }
__device__ __forceinline__ void ws_error(void* ws) {
  atomicCAS(reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + WS_ERROR), DEV_OK, DEV_TIMEOUT);
}
__device__ __forceinline__ float* dec_slot(void* ws, int cta, bool begins) {
  return reinterpret_cast<float*>(static_cast<char*>(ws) + WS_HEAD) +
         (size_t)(2 * cta + (begins ? 1 : 0)) * DEC_SLOT;
}
__device__ __forceinline__ float* pr_slot(void* ws, int cta, bool begins, int tile) {
  return reinterpret_cast<float*>(static_cast<char*>(ws) + WS_HEAD) +
         (size_t)(2 * cta + (begins ? 1 : 0)) * PR_SLOT + (size_t)tile * PR_TILE;
}

// What a row's unscaled outputs are multiplied by, from its maximum and sum:
// the head's sink joins the denominator, and a row that saw nothing gets 0.
__device__ __forceinline__ float row_factor(const PagedAttnArgs& a, int head, float m, float l) {
  const float sink = a.sinks ? a.sinks[head] * 1.4426950408889634f : -INFINITY;
  const float mm = fmaxf(m, sink);
  const float f = m > -INFINITY ? exp2f(m - mm) : 0.0f;
  const float den = fmaf(l, f, sink > -INFINITY ? exp2f(sink - mm) : 0.0f);
  return den == 0.0f ? 0.0f : f / den;  // NaN stays NaN
}

}  // namespace pg
}  // namespace flint
