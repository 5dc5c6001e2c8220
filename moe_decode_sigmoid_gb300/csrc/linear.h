// linear.h — argument blocks and launch wrappers of the linear side of a prompt:
// matrix products with an epilogue, plain or grouped (linear_rows.cu, linear_tiles.cu),
// and the selection and combine around the experts' products (moe_prompt.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace flint {
namespace lin {
// Scaled f16: SCALED values of a row have one scale, a power of two by its biased exponent,
// that puts the largest finite one into [2^14, 2^15).  Each is off by 2^-12 of itself at most
// (2^-39 of the largest, if that is more), whatever their range; 2^-9 for the same bytes in bf16.
constexpr int SCALED = 32;
constexpr int MAX_ROWS = 65536;
constexpr int MAX_IN = 65536;
constexpr int MAX_OUT = 1 << 20;
constexpr int GROUP_LIMIT = 1024;
constexpr int FEW_ROWS = 16;       // of a plain product that linear_rows.cu takes
constexpr int FEW_GROUPED = 8;     // of a grouped one, in all
constexpr int MAX_TOKENS = 8192;   // of a selection and of the layer
constexpr int CHUNK = 64;          // tokens a CTA of the selection takes
constexpr int MAX_CHUNKS = MAX_TOKENS / CHUNK;

// Workspace: error and stall word, a mark that it serves the layer, the selection's counts,
// then the layer's arrays.
constexpr size_t WS_ERROR = 0, WS_STALL = 8, WS_LAYER = 16, WS_COUNTS = 256;
constexpr size_t WS_HEAD = WS_COUNTS + 256 * (size_t)MAX_CHUNKS;
}  // namespace lin

enum { ACT_NONE = 0, ACT_SILU = 1, ACT_GELU = 2, ACT_SWIGLU = 3 };

// One call: a plain product is one group of all rows (start null).
struct LinearArgs {
  const uint16_t* x;       // [n_x, n_in] bf16
  const uint16_t* w;       // [n_groups, rows of a matrix, n_in] bf16
  const uint16_t* w_last;  // the last group's matrix lies here (its rows: x's in order), or null
  const float* bias;       // [n_groups, rows of a matrix] or null
  const void* residual;    // [n_rows, n_out] of out's type or null
  void* out;               // [n_rows, n_out]
  const int32_t* start;    // [n_groups + 1] or null
  const int32_t* index;    // [n_rows] row of x, or null
  int n_groups, n_rows, n_x, n_in, n_out, act, out_f32;
  void* ws;
  // Of the layer's tiled products.  A pair is two bf16 rows, hi = bf16(v) and lo =
  // bf16(v - hi), one behind the other: ~16 significant bits and fp32's range.
  int pair_out;            // out is [n_rows, 2 n_out], pairs (SwiGLU, grouped)
  int pair_in;             // x is [n_x, 2 n_in], pairs; out scaled f16 (no activation, grouped,
                           // n_in a multiple of 64, n_out of 32, no index)
  uint8_t* scale;          // [n_rows, n_out / SCALED] of scaled f16
  int w_rows;              // rows of a matrix in memory, of which n_out are used, or 0: as many
};
// A product of few rows (FEW_ROWS, FEW_GROUPED; no last group of its own), and anything.
cudaError_t launch_linear_rows(const LinearArgs& a, cudaStream_t stream);
cudaError_t launch_linear_tiles(const LinearArgs& a, int sms, cudaStream_t stream);

struct SelectArgs {
  const float* logits;     // [n, E]
  const float* bias;       // [E] or null
  int select_only, n;
  int* idx;                // [n, TOPK]
  float* w;                // [n, TOPK]
  int* start;              // [E + 1], [E + 2] with the shared expert's group
  int* row_token;          // [n TOPK], [n (TOPK + 1)] with it
  int* pair_row;           // [n, TOPK]
  int* idx_out;            // optional copies
  float* w_out;
  int shared_group;        // a last group of all tokens
  uint8_t* counts;         // [chunks, E] scratch
};
cudaError_t launch_select(const SelectArgs& a, cudaStream_t stream);

// Columns of H at once: residual and out point at the first one, y and y_shared are
// [rows, cols], bf16 or, with scales, scaled f16.
struct CombineArgs {
  const uint16_t* residual;  // [n, H]
  const void* y;             // [n TOPK, cols]
  const void* y_shared;      // [n, cols] or null
  const int* pair_row;       // [n, TOPK]
  const float* w;            // [n, TOPK]
  uint16_t* out;
  const uint8_t* scale;        // [n TOPK, cols / SCALED], or null
  const uint8_t* scale_shared; // [n, cols / SCALED]
  int n, cols;
};
cudaError_t launch_combine(const CombineArgs& a, cudaStream_t stream);

}  // namespace flint
