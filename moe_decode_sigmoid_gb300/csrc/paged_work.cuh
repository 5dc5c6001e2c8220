// paged_work.cuh — the paged attention's workspace (partial results of rows
// that several CTAs share, and the tickets that find the last of them) and how
// a finished row is scaled.
#pragma once

#include "paged.cuh"

namespace flint {
namespace pg {

constexpr int MAX_CTAS = 160;  // CTAs of an attention launch (one per SM; GB300 has 152)

// Workspace: three tickets per CTA, the stall word (a test hook) and an error word, then
// two slots per CTA: one for a row (or item) that began in an earlier CTA's share and
// one for one that goes on in the next one's.
constexpr size_t WS_HEAD = 4096, WS_ERROR = WS_HEAD - 4, WS_STALL = WS_HEAD - 8;
static_assert(3 * MAX_CTAS * 4 <= WS_STALL, "tickets fit");

// The cut.  A row (next tokens: a sequence and KV head; prompts: an item, a tile
// pair and KV head) weighs its key granules (tiles) and what it costs besides,
// START of them: its queries, its first keys, its outputs.  The rows' weights are
// laid end to end and cut into equal shares, one per CTA.  A cut near a row's end
// moves to it (a join costs microseconds, MARGIN granules), and a row of at most
// WHOLE is not cut at all; a share is LOW at least (1 x 4 drafts over 1000: 16 us at 4,
// 18 at 9).  START, measured at 32 / 4 heads (other layouts take the same): next
// tokens, 8 x 30K E4M3 61, 59, 58 us at 24, 40, 64, but 128 ragged sequences of 2K
// 47.8, 48.4, 50.5; prompts, windows of 513 (WHOLE 6) 45 us at 3, 49 at 6, and with
// WHOLE 4 50 us.
template <int START, int WHOLE, int MARGIN, int LEAST = 0, int LOW = START + 1>
struct Cut {
  int share, margin;
  __device__ __forceinline__ Cut(int total, int ctas)
      : share(max((total + ctas - 1) / ctas, LOW)), margin(min(share >> 4, MARGIN)) {}
  static __host__ __device__ constexpr int weight(int n) { return n > 0 ? n + START : 0; }
  // Where a cut at place x falls, in a run of rows of n granules each from `first`.
  __device__ __forceinline__ int at(int x, int first, int n) const {
    const int w = weight(n), off = (x - first) % w, rest = w - off;
    if (n <= WHOLE) return off <= rest ? x - off : x + rest;
    return off <= START + margin ? x - off : rest <= margin ? x + rest : x;
  }
  // The granules [from, to) of the row at row0 that the share cur .. end - 1 has.
  __device__ __forceinline__ void part(int cur, int end, int row0, int n, int& from, int& to) const {
    from = cur == row0 ? 0 : cur - row0 - START;
    to = end >= row0 + weight(n) ? n : end - row0 - START;
  }
  // The CTAs c0 .. c1 that share the row at row0; false if one has it whole.
  __device__ __forceinline__ bool shared(int row0, int n, int& c0, int& c1) const {
    const int i0 = (row0 + START + margin) / share + 1, i1 = (row0 + weight(n) - margin - 1) / share;
    c0 = i0 - 1;
    c1 = i1;
    return n > WHOLE && i0 <= i1;
  }
  // Few short rows are dealt out instead, a part of one row a CTA: of R rows of N
  // granules in all, none cut into parts of less than N / (ctas - R), there are at
  // most ctas parts; that is less work a CTA than an equal share, N / ctas + START
  // R / ctas, if N < START (ctas - R).  Returns the parts' size, 0 for shares.
  static __device__ __forceinline__ int deal(int total, int rows, int ctas) {
    const int n = total - START * rows, rest = ctas - rows;
    if (rest <= 0 || (long long)n > (long long)START * rest) return 0;
    return max((n + rest - 1) / rest, LEAST);
  }
  static __device__ __forceinline__ int parts(int n, int size) {
    return n <= 0 ? 0 : n <= LEAST + LEAST / 2 ? 1 : (n + size - 1) / size;
  }
};

// A slot of the next-token kernel, for each group of 8 rows (DEC_ROWS at most): 8
// maxima, 8 sums, 128 x 8 outputs.
constexpr int DEC_ML = 16, DEC_O = HD * 8, DEC_SLOT = DEC_ML + DEC_O;
template <bool FP8>
using DecCut = Cut<FP8 ? 64 : 40, 64, 32, FP8 ? 24 : 16>;

// A slot of the prompt kernel: two tiles of 128 maxima, 128 sums and 128 x 128
// outputs.
constexpr int PR_TILE = 128 * (2 + HD), PR_SLOT = 2 * PR_TILE;
// A call of split items only (no sequence brings more than a tile) has twice the key
// tiles in a step and pays more for an item beside them: 8 x 4 drafts 59 us at 3, 55
// at 8; 64 x 4 over 1000 51, 45.  (By item, the last tiles of prompts too: windows
// 45 -> 49 us.)
template <bool DRAFTS>
using PrCut = Cut<DRAFTS ? 8 : 3, 6, 3, 0, 4>;
static_assert(DEC_ROWS / 8 * DEC_SLOT <= PR_SLOT, "a workspace for either");

__host__ __device__ constexpr size_t attn_ws_bytes() {
  return WS_HEAD + sizeof(float) * 2 * MAX_CTAS * (size_t)PR_SLOT;
}

// The join of the partial results of the CTAs c0 .. c1 that share a row, always in
// the order of its keys: groups of JOIN neighbours first, each by the one of them
// that arrives last, then the groups' results, by the group that arrives last.
// (All of 38 by one CTA: its reads alone took 17 us for 32 rows of 1 x 30K tokens.)
constexpr int JOIN = 8, JOIN_MOST = (MAX_CTAS + JOIN - 1) / JOIN;
struct Join {
  int c0, c1, first, n, stride, kind;
  bool top;  // what this join makes is the row's result
  __device__ __forceinline__ Join(int cta, int c0, int c1)
      : c0(c0), c1(c1), first(c0 + (cta - c0) / JOIN * JOIN), stride(1) {
    n = min(JOIN, c1 - first + 1);
    top = c1 - c0 < JOIN;
    // A CTA may be the first of a row and of a later group of the row before.
    kind = top ? 0 : first == c0 ? 1 : 2;
  }
  __device__ __forceinline__ void up() {
    first = c0;
    n = (c1 - c0) / JOIN + 1;
    stride = JOIN;
    kind = 0;
    top = true;
  }
  __device__ __forceinline__ int cta(int k) const { return first + k * stride; }
  __device__ __forceinline__ bool begins(int k) const { return cta(k) == c0; }
  // One thread of the CTA, all of its results written before: is it the last?
  __device__ __forceinline__ bool arrive(void* ws) const {
    uint32_t* ticket = static_cast<uint32_t*>(ws) + kind * MAX_CTAS + first;
    const bool last = atomicAdd(ticket, 1u) == (uint32_t)(n - 1);
    if (last) *ticket = 0u;  // ready for the next call
    __threadfence();
    return last;
  }
};
__device__ __forceinline__ uint32_t* ws_stall(void* ws) {
  return reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + WS_STALL);
}
__device__ __forceinline__ void ws_error(void* ws) {
  atomicCAS(reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + WS_ERROR), DEV_OK, DEV_TIMEOUT);
}
__device__ __forceinline__ float* dec_slot(void* ws, int cta, bool begins, int groups) {
  return reinterpret_cast<float*>(static_cast<char*>(ws) + WS_HEAD) +
         (size_t)(2 * cta + (begins ? 1 : 0)) * groups * DEC_SLOT;
}
__device__ __forceinline__ float* pr_slot(void* ws, int cta, bool begins, int tile) {
  return reinterpret_cast<float*>(static_cast<char*>(ws) + WS_HEAD) +
         (size_t)(2 * cta + (begins ? 1 : 0)) * PR_SLOT + (size_t)tile * PR_TILE;
}

// An E4M3 cache's weights meet V as f16, relative to 2^m: m stays this much below the
// largest exponent (f16 reaches 2^16, and m lags by up to 8).  bf16 has fp32's range.
template <bool FP8>
constexpr float weight_lift = FP8 ? 7.0f : 0.0f;

// What a value's scale counts as at least, 2^-80: one of zero would take its block's
// weights out of the sum.  (2^15 times 2^80 times 2^23 keys is within fp32.)
constexpr float LEAST_SCALE = 8.271806125530277e-25f;

// What a row's unscaled outputs are multiplied by, from its maximum and sum: the
// head's sink joins the denominator (none for -infinity; 0 in the end for infinity,
// NaN for NaN), and a row that saw nothing gets 0.
__device__ __forceinline__ float row_factor(const PagedAttnArgs& a, int head, float m, float l) {
  const float sink = a.sinks ? a.sinks[head] * 1.4426950408889634f : -INFINITY;
  const float mm = fmaxf(m, sink);
  const float f = m > -INFINITY ? exp2f(m - mm) : 0.0f;
  const float den = fmaf(l, f, sink == -INFINITY ? 0.0f : exp2f(sink - mm));
  return f == 0.0f ? l * 0.0f : f / den;  // a NaN in l stays one
}

}  // namespace pg
}  // namespace flint
