// api_paged.cu — the C ABI of the paged KV cache (include/flint_moe.h): the
// append with Q/K norm and rotary embedding, and the attention over the cache.
// Host-side argument checks, argument blocks and launches; nothing here
// allocates, and only flint_attn_get_device_status synchronises.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "flint_moe.h"
#include "host_checks.h"
#include "paged.h"

using namespace flint;

namespace {

constexpr long long MAX_ROWS = 1ll << 30;  // token rows of a cache

// What the kernels' tables and index widths are made for.
static_assert(FLINT_PAGED_MAX_SEQS == pg::MAX_SEQS && FLINT_PAGED_MAX_TOKENS == pg::MAX_TOKENS &&
                  FLINT_KV_BLOCK == pg::BLOCK,
              "the public limits are the kernels'");

flint_status dims_status(const flint_attn_dims* d) {
  if (d == nullptr) return FLINT_ERR_INVALID_ARG;
  if (d->head_dim != pg::HD) return FLINT_ERR_UNSUPPORTED;
  const int n = d->n_kv_heads;
  if (n < 1 || n > pg::MAX_KV_HEADS || (n & (n - 1)) != 0) return FLINT_ERR_UNSUPPORTED;
  for (int g = 1; g <= pg::MAX_GROUP; g *= 2)
    if (d->n_q_heads == n * g) return FLINT_OK;
  return FLINT_ERR_UNSUPPORTED;
}

bool finite_nonneg(float v) { return v >= 0.0f && v <= 3.0e38f; }

// Checks the dims, the batch and the call's rows, and fills the view.
flint_status batch_view(const flint_attn_dims* dims, const flint_paged_batch* b, int32_t n_tokens,
                        PagedView& v) {
  const flint_status st = dims_status(dims);
  if (st != FLINT_OK) return st;
  if (b == nullptr || n_tokens < 1 || n_tokens > FLINT_PAGED_MAX_TOKENS || b->n_seqs < 1 ||
      b->n_seqs > FLINT_PAGED_MAX_SEQS || b->max_q_len < 1 || b->max_pages < 1 || b->n_pages < 1)
    return FLINT_ERR_INVALID_ARG;
  int shift = 4;
  while (shift < 10 && (1 << shift) != b->page_size) ++shift;
  if ((1 << shift) != b->page_size || ((long long)b->max_pages << shift) > pg::MAX_LENGTH ||
      ((long long)b->n_pages << shift) > MAX_ROWS)
    return FLINT_ERR_INVALID_ARG;
  if (!req4(b->q_start) || !req4(b->kv_len) || !req4(b->page_table)) return FLINT_ERR_INVALID_ARG;
  v.q_start = b->q_start;
  v.kv_len = b->kv_len;
  v.page_table = b->page_table;
  v.n_seqs = b->n_seqs;
  v.n_tokens = n_tokens;
  v.max_q = b->max_q_len;
  v.page_shift = shift;
  v.max_pages = b->max_pages;
  v.n_pages = b->n_pages;
  v.nkv = dims->n_kv_heads;
  v.group = dims->n_q_heads / dims->n_kv_heads;
  return FLINT_OK;
}

size_t cache_bytes(const PagedView& v, bool fp8) {
  return ((size_t)v.n_pages << v.page_shift) * v.nkv * pg::HD * (fp8 ? 1 : 2);
}
size_t scale_bytes(const PagedView& v) {
  return (((size_t)v.n_pages << v.page_shift) / pg::BLOCK) * v.nkv * 4;
}

struct Span {
  const void* p;
  size_t n;
};
// True if one of the first n_out spans overlaps any other span.
bool any_overlap(const Span* s, int n, int n_out) {
  for (int i = 0; i < n_out; ++i)
    for (int j = 0; j < n; ++j)
      if (i != j && s[i].p != nullptr && s[j].p != nullptr && overlap(s[i].p, s[i].n, s[j].p, s[j].n))
        return true;
  return false;
}

// A theta below 1 has frequencies of more than a turn a token (the kernel's steps
// of up to 8 tokens in fp32 would be off by 2^-21 of those): whole turns a token
// are whole turns at any position, so each frequency is brought to [-pi, pi], from
// powers of one rounding each and with 2 pi in two parts.
void whole_turns_off(double theta, double* freq) {
  constexpr double TWO_PI_HI = 6.283185307179586;  // 2 pi = HI + LO
  constexpr double TWO_PI_LO = 2.4492935982947064e-16;
  for (int i = 0; i < pg::HD / 2; ++i) {
    const double f = std::pow(theta, -2.0 * i / pg::HD), k = std::rint(f / TWO_PI_HI);
    freq[i] = std::fma(-k, TWO_PI_LO, std::fma(-k, TWO_PI_HI, f));
  }
}

flint_status append(bool fp8, const flint_attn_dims* dims, const flint_paged_batch* batch,
                    int32_t n_tokens, const void* qkv, const void* q_norm, const void* k_norm,
                    float rope_theta, float eps, void* q_out, void* k_cache, void* v_cache,
                    float* k_scale, float* v_scale, cudaStream_t stream) {
  PagedAppendArgs a;
  const flint_status st = batch_view(dims, batch, n_tokens, a.b);
  if (st != FLINT_OK) return st;
  if (!req(qkv) || !req(q_norm) || !req(k_norm) || !req(q_out) || !req(k_cache) || !req(v_cache) ||
      (fp8 && (!req4(k_scale) || !req4(v_scale))) || !finite_nonneg(rope_theta) ||
      !finite_nonneg(eps))
    return FLINT_ERR_INVALID_ARG;
  const int nq = a.b.nkv * a.b.group;
  const size_t c = cache_bytes(a.b, fp8), sc = scale_bytes(a.b);
  const Span spans[] = {{q_out, (size_t)n_tokens * nq * pg::HD * 2},
                        {k_cache, c},
                        {v_cache, c},
                        {k_scale, sc},
                        {v_scale, sc},
                        {qkv, (size_t)n_tokens * (nq + 2 * a.b.nkv) * pg::HD * 2},
                        {q_norm, pg::HD * 2},
                        {k_norm, pg::HD * 2},
                        {a.b.q_start, (size_t)(a.b.n_seqs + 1) * 4},
                        {a.b.kv_len, (size_t)a.b.n_seqs * 4},
                        {a.b.page_table, (size_t)a.b.n_seqs * a.b.max_pages * 4}};
  if (any_overlap(spans, 11, 5)) return FLINT_ERR_INVALID_ARG;
  a.qkv = static_cast<const uint16_t*>(qkv);
  a.q_norm = static_cast<const uint16_t*>(q_norm);
  a.k_norm = static_cast<const uint16_t*>(k_norm);
  a.rope = rope_theta > 0.0f;
  // theta^(-2i/128) for i = 8 hi + lo, from two powers and their products, a
  // dozen roundings deep at most: off by 2^-49, and 64 calls of pow() cost more
  // than the launch (16 of them half a microsecond).
  double hi[8] = {}, lo[8] = {};
  if (a.rope) {
    hi[0] = lo[0] = 1.0;
    hi[1] = std::pow((double)rope_theta, -16.0 / pg::HD);
    lo[1] = std::pow((double)rope_theta, -2.0 / pg::HD);
    for (int i = 2; i < 8; ++i) {
      hi[i] = hi[i >> 1] * hi[i - (i >> 1)];
      lo[i] = lo[i >> 1] * lo[i - (i >> 1)];
    }
  }
  for (int i = 0; i < pg::HD / 2; ++i) a.inv_freq[i] = hi[i >> 3] * lo[i & 7];
  if (a.rope && rope_theta < 1.0f) whole_turns_off(rope_theta, a.inv_freq);
  a.eps = eps;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  return cuda_status(launch_paged_append(a, fp8, stream));
}

flint_status attend(bool fp8, const flint_attn_dims* dims, const flint_paged_batch* batch,
                    int32_t n_tokens, const void* q, const void* k_cache, const void* v_cache,
                    const float* k_scale, const float* v_scale, const float* sinks,
                    float softmax_scale, int32_t window, void* out, void* workspace,
                    size_t ws_bytes, cudaStream_t stream) {
  PagedAttnArgs a;
  const flint_status st = batch_view(dims, batch, n_tokens, a.b);
  if (st != FLINT_OK) return st;
  if (!req(q) || !req(k_cache) || !req(v_cache) || !req(out) || !opt4(sinks) ||
      (fp8 && (!req4(k_scale) || !req4(v_scale))) || !finite_nonneg(softmax_scale) || window < 0)
    return FLINT_ERR_INVALID_ARG;
  if (!req(workspace) || ws_bytes < paged_attn_workspace_bytes()) return FLINT_ERR_WORKSPACE;
  const int nq = a.b.nkv * a.b.group;
  const size_t c = cache_bytes(a.b, fp8), sc = scale_bytes(a.b);
  const Span spans[] = {{out, (size_t)n_tokens * nq * pg::HD * 2},
                        {workspace, ws_bytes},
                        {q, (size_t)n_tokens * nq * pg::HD * 2},
                        {k_cache, c},
                        {v_cache, c},
                        {k_scale, sc},
                        {v_scale, sc},
                        {sinks, (size_t)nq * 4},
                        {a.b.q_start, (size_t)(a.b.n_seqs + 1) * 4},
                        {a.b.kv_len, (size_t)a.b.n_seqs * 4},
                        {a.b.page_table, (size_t)a.b.n_seqs * a.b.max_pages * 4}};
  if (any_overlap(spans, 11, 2)) return FLINT_ERR_INVALID_ARG;
  const int sms = num_sms();
  if (sms <= 0) return FLINT_ERR_CUDA;
  a.q = static_cast<const uint16_t*>(q);
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.sinks = sinks;
  a.scale_log2 = std::fmin(softmax_scale * 1.4426950408889634f, FLT_MAX);
  // Positions lie within -MAX_TOKENS .. MAX_LENGTH: a wider window sees no more,
  // and position - window stays within 32 bits.
  a.window = (int)std::min<long long>(window, 2 * pg::MAX_LENGTH);
  a.out = static_cast<uint16_t*>(out);
  a.ws = workspace;
  return cuda_status(a.b.max_q <= pg::DEC_ROWS / a.b.group ? launch_paged_decode(a, fp8, sms, stream)
                                                           : launch_paged_prompt(a, fp8, sms, stream));
}

}  // namespace

extern "C" {

flint_status flint_qk_norm_rope_kv_paged_bf16(const flint_attn_dims* dims,
                                              const flint_paged_batch* batch, int32_t n_tokens,
                                              const void* qkv_bf16, const void* q_norm_bf16,
                                              const void* k_norm_bf16, float rope_theta, float eps,
                                              void* q_out_bf16, void* k_cache_bf16,
                                              void* v_cache_bf16, cudaStream_t stream) {
  return append(false, dims, batch, n_tokens, qkv_bf16, q_norm_bf16, k_norm_bf16, rope_theta, eps,
                q_out_bf16, k_cache_bf16, v_cache_bf16, nullptr, nullptr, stream);
}

flint_status flint_qk_norm_rope_kv_paged_fp8(const flint_attn_dims* dims,
                                             const flint_paged_batch* batch, int32_t n_tokens,
                                             const void* qkv_bf16, const void* q_norm_bf16,
                                             const void* k_norm_bf16, float rope_theta, float eps,
                                             void* q_out_bf16, uint8_t* k_cache_e4m3,
                                             uint8_t* v_cache_e4m3, float* k_scale, float* v_scale,
                                             cudaStream_t stream) {
  return append(true, dims, batch, n_tokens, qkv_bf16, q_norm_bf16, k_norm_bf16, rope_theta, eps,
                q_out_bf16, k_cache_e4m3, v_cache_e4m3, k_scale, v_scale, stream);
}

size_t flint_attn_workspace_bytes(const flint_attn_dims* dims) {
  return dims_status(dims) == FLINT_OK ? paged_attn_workspace_bytes() : 0;
}

flint_status flint_attn_workspace_init(void* workspace, size_t ws_bytes, cudaStream_t stream) {
  if (!req(workspace) || ws_bytes < paged_attn_workspace_bytes()) return FLINT_ERR_WORKSPACE;
  return cuda_status(cudaMemsetAsync(workspace, 0, paged_attn_workspace_clear_bytes(), stream));
}

flint_status flint_attn_get_device_status(const void* workspace, cudaStream_t stream) {
  if (!req(workspace)) return FLINT_ERR_WORKSPACE;
  uint32_t code = 0;
  if (cudaMemcpyAsync(&code, static_cast<const char*>(workspace) + paged_attn_workspace_error_at(),
                      sizeof(code), cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess) {
    (void)cudaGetLastError();
    return FLINT_ERR_CUDA;
  }
  return static_cast<flint_status>(code);
}

flint_status flint_attn_debug_arm_stall(void* workspace, size_t ws_bytes, cudaStream_t stream) {
  if (!req(workspace) || ws_bytes < paged_attn_workspace_bytes()) return FLINT_ERR_WORKSPACE;
  return cuda_status(cudaMemsetAsync(static_cast<char*>(workspace) + paged_attn_workspace_stall_at(),
                                     1, sizeof(uint32_t), stream));
}

flint_status flint_attn_paged_bf16(const flint_attn_dims* dims, const flint_paged_batch* batch,
                                   int32_t n_tokens, const void* q_bf16, const void* k_cache_bf16,
                                   const void* v_cache_bf16, const float* sinks,
                                   float softmax_scale, int32_t window, void* out_bf16,
                                   void* workspace, size_t ws_bytes, cudaStream_t stream) {
  return attend(false, dims, batch, n_tokens, q_bf16, k_cache_bf16, v_cache_bf16, nullptr, nullptr,
                sinks, softmax_scale, window, out_bf16, workspace, ws_bytes, stream);
}

flint_status flint_attn_paged_fp8(const flint_attn_dims* dims, const flint_paged_batch* batch,
                                  int32_t n_tokens, const void* q_bf16,
                                  const uint8_t* k_cache_e4m3, const uint8_t* v_cache_e4m3,
                                  const float* k_scale, const float* v_scale, const float* sinks,
                                  float softmax_scale, int32_t window, void* out_bf16,
                                  void* workspace, size_t ws_bytes, cudaStream_t stream) {
  return attend(true, dims, batch, n_tokens, q_bf16, k_cache_e4m3, v_cache_e4m3, k_scale, v_scale,
                sinks, softmax_scale, window, out_bf16, workspace, ws_bytes, stream);
}

}  // extern "C"
