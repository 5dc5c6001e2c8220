// paged.h — argument blocks and launch wrappers of the paged KV-cache kernels:
// the append (paged_append.cu) and the attention (paged_decode.cu, paged_prompt.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace flint {
namespace pg {
constexpr int HD = 128;            // head size
constexpr int BLOCK = 16;          // token rows that share a scale
constexpr int MAX_SEQS = 256;
constexpr int MAX_TOKENS = 8192;         // rows of a call
constexpr long long MAX_LENGTH = 1ll << 23;  // tokens of a sequence
constexpr int MAX_KV_HEADS = 8;
constexpr int MAX_GROUP = 8;       // query heads per KV head
constexpr int DEC_ROWS = 16;       // query rows (tokens x group) a KV head has at most in the next-token kernel
}  // namespace pg

// The batch a call works on (flint_paged_batch, the call's rows and the head
// layout), by value.
struct PagedView {
  const int32_t* q_start;     // [n_seqs + 1]
  const int32_t* kv_len;      // [n_seqs]
  const int32_t* page_table;  // [n_seqs, max_pages]
  int n_seqs, n_tokens, max_q;
  int page_shift;             // log2(page size)
  int max_pages, n_pages;
  int nkv, group;             // KV heads, query heads per KV head
};

struct PagedAppendArgs {
  PagedView b;
  const uint16_t* qkv;     // [n_tokens, (nq + 2 nkv) * HD] bf16
  const uint16_t* q_norm;  // [HD] bf16
  const uint16_t* k_norm;  // [HD] bf16
  int rope;                // 0: no rotation
  double inv_freq[pg::HD / 2];  // theta^(-2i/HD), to whole turns in [-pi, pi]
  float eps;
  uint16_t* q_out;         // [n_tokens, nq, HD] bf16
  void* k_cache;           // [n_pages << page_shift, nkv, HD] bf16 or E4M3 codes
  void* v_cache;
  float* k_scale;          // E4M3: [(n_pages << page_shift) / BLOCK, nkv]
  float* v_scale;
};
cudaError_t launch_paged_append(const PagedAppendArgs& a, bool fp8, cudaStream_t stream);

struct PagedAttnArgs {
  PagedView b;
  const uint16_t* q;       // [n_tokens, nq, HD] bf16
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;    // E4M3 cache only
  const float* v_scale;
  const float* sinks;      // [nq] or null
  float scale_log2;        // softmax scale * log2(e)
  int window;              // 0: none
  uint16_t* out;           // [n_tokens, nq, HD] bf16
  void* ws;
};
// A few rows a sequence (max_q * group at most DEC_ROWS), and any number.
cudaError_t launch_paged_decode(const PagedAttnArgs& a, bool fp8, int sms, cudaStream_t stream);
cudaError_t launch_paged_prompt(const PagedAttnArgs& a, bool fp8, int sms, cudaStream_t stream);

size_t paged_attn_workspace_bytes();
// Leading bytes of the workspace that flint_attn_workspace_init clears.
size_t paged_attn_workspace_clear_bytes();
// Where its error word (a device error code) and its stall word lie.
size_t paged_attn_workspace_error_at();
size_t paged_attn_workspace_stall_at();

}  // namespace flint
