// api_prompt.cu — the C ABI of the linear side of a prompt (include/flint_moe.h):
// linear products, plain and grouped by expert, the selection and combine around
// the experts' products, and the layer made of them.  Host-side argument checks,
// argument blocks and launches; nothing here allocates, and only
// flint_prompt_get_device_status synchronises.
#include <cstring>

#include "common.cuh"
#include "flint_moe.h"
#include "host_checks.h"
#include "linear.h"

using namespace flint;

namespace {

static_assert(FLINT_LINEAR_MAX_ROWS == lin::MAX_ROWS && FLINT_LINEAR_MAX_IN == lin::MAX_IN &&
                  FLINT_LINEAR_MAX_OUT == lin::MAX_OUT && FLINT_LINEAR_MAX_GROUPS == lin::GROUP_LIMIT &&
                  FLINT_PAGED_MAX_TOKENS == lin::MAX_TOKENS,
              "the public limits are the kernels'");
static_assert(FLINT_ACT_NONE == ACT_NONE && FLINT_ACT_SILU == ACT_SILU && FLINT_ACT_GELU == ACT_GELU &&
                  FLINT_ACT_SWIGLU == ACT_SWIGLU,
              "the public activations are the kernels'");

// Up to so many tokens the layer is flint_moe_decode_bf16, in a workspace of its own behind
// the head.  Measured with the weights in HBM, decode against products by expert, us: 16
// tokens 95 / 107, 64 202 / 210, 96 228 / 237, 128 257 / 257, 192 281 / 257, 256 337 / 262; with
// skewed routing 64 152 / 159, 96 188 / 191, 128 200 / 189, 192 250 / 206.
constexpr int DECODE_TOKENS = 128;
static_assert(DECODE_TOKENS <= MAX_B, "a batch of the decode call");
constexpr size_t DECODE_WS = align256(lin::WS_HEAD);
size_t decode_ws_bytes(size_t n) { return WsLayout::total((int)(n < DECODE_TOKENS ? n : DECODE_TOKENS)); }

// The layer's arrays behind that, for n tokens: h in pairs of bf16, y in scaled f16 (both rounded
// to bf16, outputs were off by 9e-2 of max(|out - residual|, a tenth of its rms), against 2e-2 of
// the decode call).  y has all columns at once, or above WHOLE_TOKENS, where memory counts more
// than two more launches and h read again (10 to 14 us), half of them in turn.
constexpr size_t COLUMNS = H / 2, WHOLE_TOKENS = 4096;
static_assert(COLUMNS % 256 == 0, "whole tiles of weight rows");
struct Layer {
  size_t logits, idx, w, start, row_token, pair_row, scale, h, y, cols, end;
  explicit Layer(size_t n) : cols(n <= WHOLE_TOKENS ? H : COLUMNS) {
    logits = align256(DECODE_WS + decode_ws_bytes(n));
    if (n <= DECODE_TOKENS) {
      end = logits;
      return;
    }
    idx = align256(logits + n * E * 4);
    w = align256(idx + n * TOPK * 4);
    start = align256(w + n * TOPK * 4);
    row_token = align256(start + (E + 2) * 4);
    pair_row = align256(row_token + n * SLOTS * 4);
    scale = align256(pair_row + n * TOPK * 4);
    h = align256(scale + n * SLOTS * (cols / lin::SCALED));
    y = align256(h + n * SLOTS * I * 4);
    end = align256(y + n * SLOTS * cols * 2);
  }
};

size_t workspace_bytes(int tokens) {
  if (tokens == 0) return align256(lin::WS_HEAD);
  const size_t own = Layer(tokens).end, whole = Layer(tokens < (int)WHOLE_TOKENS ? tokens : WHOLE_TOKENS).end;
  return own > whole ? own : whole;   // (of every call of fewer tokens too)
}

flint_status linear_status(const flint_linear_dims* d) {
  if (d == nullptr) return FLINT_ERR_INVALID_ARG;
  const int of = d->act == FLINT_ACT_SWIGLU ? 16 : 8;
  if (d->act < FLINT_ACT_NONE || d->act > FLINT_ACT_SWIGLU || (d->out_f32 != 0 && d->out_f32 != 1) ||
      d->n_in < 8 || d->n_in > FLINT_LINEAR_MAX_IN || d->n_in % 8 != 0 || d->n_out < of ||
      d->n_out > FLINT_LINEAR_MAX_OUT || d->n_out % of != 0)
    return FLINT_ERR_UNSUPPORTED;
  return FLINT_OK;
}

flint_status moe_status(const flint_moe_dims* d) {
  if (d == nullptr) return FLINT_ERR_INVALID_ARG;
  return d->hidden == H && d->n_experts == E && d->top_k == TOPK && d->inter == I && d->n_shared == S &&
                 (d->offset_mode == FLINT_OFFSET_LOGIT || d->offset_mode == FLINT_OFFSET_SELECT)
             ? FLINT_OK
             : FLINT_ERR_UNSUPPORTED;
}

// An argument's memory.
struct Span {
  const void* p;
  size_t n;
};
// True if one of the first n_out spans overlaps any other one.
template <int N>
bool any_overlap(const Span (&s)[N], int n_out) {
  for (int i = 0; i < n_out; ++i)
    for (int j = 0; j < N; ++j)
      if (i != j && s[i].p != nullptr && s[j].p != nullptr && overlap(s[i].p, s[i].n, s[j].p, s[j].n))
        return true;
  return false;
}

flint_status launch_linear(const LinearArgs& a, cudaStream_t stream) {
  if (a.n_rows <= (a.start != nullptr ? lin::FEW_GROUPED : lin::FEW_ROWS))
    return cuda_status(launch_linear_rows(a, stream));
  const int sms = num_sms();
  if (sms < 2) return FLINT_ERR_CUDA;
  return cuda_status(launch_linear_tiles(a, sms, stream));
}

bool ws_ok(const void* ws, size_t bytes, int tokens) { return req(ws) && bytes >= workspace_bytes(tokens); }

}  // namespace

extern "C" {

size_t flint_prompt_workspace_bytes(int32_t max_tokens) {
  return max_tokens < 0 || max_tokens > FLINT_PAGED_MAX_TOKENS ? 0 : workspace_bytes(max_tokens);
}

flint_status flint_prompt_workspace_init(void* workspace, size_t ws_bytes, cudaStream_t stream) {
  if (!ws_ok(workspace, ws_bytes, 0)) return FLINT_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  const flint_status st = cuda_status(cudaMemsetAsync(ws, 0, lin::WS_COUNTS, stream));
  if (st != FLINT_OK || ws_bytes < workspace_bytes(1)) return st;
  // Of a layer: the decode call's workspace too, and a mark that it is there.
  const size_t rest = ws_bytes - DECODE_WS, most = WsLayout::total(DECODE_TOKENS);
  const flint_status ds = flint_moe_workspace_init(ws + DECODE_WS, rest < most ? rest : most, 0, stream);
  return ds != FLINT_OK ? ds : cuda_status(cudaMemsetAsync(ws + lin::WS_LAYER, 1, 1, stream));
}

flint_status flint_prompt_get_device_status(const void* workspace, cudaStream_t stream) {
  if (!req(workspace)) return FLINT_ERR_WORKSPACE;
  char head[lin::WS_COUNTS] = {};
  if (cudaMemcpyAsync(head, workspace, sizeof(head), cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess) {
    (void)cudaGetLastError();
    return FLINT_ERR_CUDA;
  }
  uint32_t code;
  std::memcpy(&code, head + lin::WS_ERROR, sizeof(code));
  if (code == FLINT_OK && head[lin::WS_LAYER] != 0)
    return flint_moe_get_device_status(static_cast<const char*>(workspace) + DECODE_WS, stream);
  return static_cast<flint_status>(code);
}

flint_status flint_prompt_debug_arm_stall(void* workspace, size_t ws_bytes, cudaStream_t stream) {
  if (!ws_ok(workspace, ws_bytes, 0)) return FLINT_ERR_WORKSPACE;
  return cuda_status(cudaMemsetAsync(static_cast<char*>(workspace) + lin::WS_STALL, 1, sizeof(uint32_t), stream));
}

flint_status flint_linear_bf16(const flint_linear_dims* dims, int32_t n_rows, const void* x_bf16,
                               const void* w_bf16, const float* bias, const void* residual,
                               void* out, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  const flint_status st = linear_status(dims);
  if (st != FLINT_OK) return st;
  if (n_rows < 1 || n_rows > FLINT_LINEAR_MAX_ROWS || !req(x_bf16) || !req(w_bf16) || !opt4(bias) ||
      !aligned16(residual) || !req(out))
    return FLINT_ERR_INVALID_ARG;
  if (!ws_ok(workspace, ws_bytes, 0)) return FLINT_ERR_WORKSPACE;
  const size_t m = (size_t)dims->n_out * (dims->act == FLINT_ACT_SWIGLU ? 2 : 1);
  const size_t o = (size_t)n_rows * dims->n_out * (dims->out_f32 ? 4 : 2);
  const Span spans[] = {{out, o},
                        {workspace, ws_bytes},
                        {x_bf16, (size_t)n_rows * dims->n_in * 2},
                        {w_bf16, m * dims->n_in * 2},
                        {bias, m * 4},
                        {residual == out ? nullptr : residual, o}};
  if (any_overlap(spans, 2) || (residual != nullptr && overlap(residual, o, workspace, ws_bytes)))
    return FLINT_ERR_INVALID_ARG;
  LinearArgs a = {};
  a.x = static_cast<const uint16_t*>(x_bf16);
  a.w = static_cast<const uint16_t*>(w_bf16);
  a.bias = bias;
  a.residual = residual;
  a.out = out;
  a.n_groups = 1;
  a.n_rows = a.n_x = n_rows;
  a.n_in = dims->n_in;
  a.n_out = dims->n_out;
  a.act = dims->act;
  a.out_f32 = dims->out_f32;
  a.ws = workspace;
  return launch_linear(a, stream);
}

flint_status flint_grouped_linear_bf16(const flint_linear_dims* dims, int32_t n_groups,
                                       int32_t n_rows, const int32_t* group_start,
                                       const int32_t* row_index, int32_t n_x, const void* x_bf16,
                                       const void* w_bf16, const float* bias, void* out,
                                       void* workspace, size_t ws_bytes, cudaStream_t stream) {
  const flint_status st = linear_status(dims);
  if (st != FLINT_OK) return st;
  if (n_groups < 1 || n_groups > FLINT_LINEAR_MAX_GROUPS || n_rows < 1 ||
      n_rows > FLINT_LINEAR_MAX_ROWS || n_x < 1 || n_x > FLINT_LINEAR_MAX_ROWS ||
      (row_index == nullptr && n_x != n_rows) || !req4(group_start) || !opt4(row_index) ||
      !req(x_bf16) || !req(w_bf16) || !opt4(bias) || !req(out))
    return FLINT_ERR_INVALID_ARG;
  if (!ws_ok(workspace, ws_bytes, 0)) return FLINT_ERR_WORKSPACE;
  const size_t m = (size_t)dims->n_out * (dims->act == FLINT_ACT_SWIGLU ? 2 : 1);
  const Span spans[] = {{out, (size_t)n_rows * dims->n_out * (dims->out_f32 ? 4 : 2)},
                        {workspace, ws_bytes},
                        {x_bf16, (size_t)n_x * dims->n_in * 2},
                        {w_bf16, n_groups * m * dims->n_in * 2},
                        {bias, n_groups * m * 4},
                        {group_start, (size_t)(n_groups + 1) * 4},
                        {row_index, (size_t)n_rows * 4}};
  if (any_overlap(spans, 2)) return FLINT_ERR_INVALID_ARG;
  LinearArgs a = {};
  a.x = static_cast<const uint16_t*>(x_bf16);
  a.w = static_cast<const uint16_t*>(w_bf16);
  a.bias = bias;
  a.out = out;
  a.start = group_start;
  a.index = row_index;
  a.n_groups = n_groups;
  a.n_rows = n_rows;
  a.n_x = n_x;
  a.n_in = dims->n_in;
  a.n_out = dims->n_out;
  a.act = dims->act;
  a.out_f32 = dims->out_f32;
  a.ws = workspace;
  return launch_linear(a, stream);
}

flint_status flint_moe_select(const flint_moe_dims* dims, int32_t n_tokens, const float* logits,
                              const float* logit_bias, int32_t* topk_idx, float* topk_w,
                              int32_t* group_start, int32_t* row_token, int32_t* pair_row,
                              void* workspace, size_t ws_bytes, cudaStream_t stream) {
  const flint_status st = moe_status(dims);
  if (st != FLINT_OK) return st;
  if (n_tokens < 1 || n_tokens > FLINT_PAGED_MAX_TOKENS || !req4(logits) || !opt4(logit_bias) ||
      !req4(topk_idx) || !req4(topk_w) || !req4(group_start) || !req4(row_token) || !req4(pair_row))
    return FLINT_ERR_INVALID_ARG;
  if (!ws_ok(workspace, ws_bytes, 0)) return FLINT_ERR_WORKSPACE;
  const size_t p = (size_t)n_tokens * TOPK * 4;
  const Span spans[] = {{topk_idx, p},
                        {topk_w, p},
                        {group_start, (E + 1) * 4},
                        {row_token, p},
                        {pair_row, p},
                        {workspace, ws_bytes},
                        {logits, (size_t)n_tokens * E * 4},
                        {logit_bias, E * 4}};
  if (any_overlap(spans, 6)) return FLINT_ERR_INVALID_ARG;
  SelectArgs a = {};
  a.logits = logits;
  a.bias = logit_bias;
  a.select_only = dims->offset_mode == FLINT_OFFSET_SELECT;
  a.n = n_tokens;
  a.idx = topk_idx;
  a.w = topk_w;
  a.start = group_start;
  a.row_token = row_token;
  a.pair_row = pair_row;
  a.counts = reinterpret_cast<uint8_t*>(static_cast<char*>(workspace) + lin::WS_COUNTS);
  return cuda_status(launch_select(a, stream));
}

flint_status flint_moe_combine_bf16(const flint_moe_dims* dims, int32_t n_tokens,
                                    const void* residual_bf16, const void* y_bf16,
                                    const int32_t* pair_row, const float* topk_w,
                                    const void* y_shared_bf16, void* out_bf16,
                                    cudaStream_t stream) {
  const flint_status st = moe_status(dims);
  if (st != FLINT_OK) return st;
  if (n_tokens < 1 || n_tokens > FLINT_PAGED_MAX_TOKENS || !req(residual_bf16) || !req(y_bf16) ||
      !req4(pair_row) || !req4(topk_w) || !aligned16(y_shared_bf16) || !req(out_bf16))
    return FLINT_ERR_INVALID_ARG;
  const size_t rows = (size_t)n_tokens * H * 2, p = (size_t)n_tokens * TOPK * 4;
  const Span spans[] = {{out_bf16, rows},
                        {residual_bf16 == out_bf16 ? nullptr : residual_bf16, rows},
                        {y_bf16, rows * TOPK},
                        {pair_row, p},
                        {topk_w, p},
                        {y_shared_bf16, rows}};
  if (any_overlap(spans, 1)) return FLINT_ERR_INVALID_ARG;
  CombineArgs a = {};
  a.residual = static_cast<const uint16_t*>(residual_bf16);
  a.y = static_cast<const uint16_t*>(y_bf16);
  a.y_shared = static_cast<const uint16_t*>(y_shared_bf16);
  a.pair_row = pair_row;
  a.w = topk_w;
  a.out = static_cast<uint16_t*>(out_bf16);
  a.n = n_tokens;
  a.cols = H;
  return cuda_status(launch_combine(a, stream));
}

flint_status flint_moe_prompt_bf16(const flint_moe_dims* dims, int32_t n_tokens,
                                   const void* x_bf16, const void* residual_bf16,
                                   const void* w_router_bf16, const float* logit_bias,
                                   const void* w13_bf16, const void* w2_bf16,
                                   const void* ws13_bf16, const void* ws2_bf16, void* out_bf16,
                                   int32_t* topk_idx_out, float* topk_w_out,
                                   void* workspace, size_t ws_bytes, cudaStream_t stream) {
  flint_status st = moe_status(dims);
  if (st != FLINT_OK) return st;
  if (n_tokens < 1 || n_tokens > FLINT_PAGED_MAX_TOKENS || !req(x_bf16) || !req(residual_bf16) ||
      !req(w_router_bf16) || !opt4(logit_bias) || !req(w13_bf16) || !req(w2_bf16) ||
      !req(ws13_bf16) || !req(ws2_bf16) || !req(out_bf16) || !opt4(topk_idx_out) || !opt4(topk_w_out))
    return FLINT_ERR_INVALID_ARG;
  if (!ws_ok(workspace, ws_bytes, n_tokens)) return FLINT_ERR_WORKSPACE;
  const size_t rows = (size_t)n_tokens * H * 2, p = (size_t)n_tokens * TOPK * 4;
  const Span spans[] = {{out_bf16, rows},
                        {topk_idx_out, p},
                        {topk_w_out, p},
                        {workspace, ws_bytes},
                        {residual_bf16 == out_bf16 ? nullptr : residual_bf16, rows},
                        {x_bf16, rows},
                        {w_router_bf16, (size_t)E * H * 2},
                        {logit_bias, E * 4},
                        {w13_bf16, (size_t)E * 2 * I * H * 2},
                        {w2_bf16, (size_t)E * H * I * 2},
                        {ws13_bf16, (size_t)S * 2 * I * H * 2},
                        {ws2_bf16, (size_t)S * H * I * 2}};
  if (any_overlap(spans, 4)) return FLINT_ERR_INVALID_ARG;

  char* ws = static_cast<char*>(workspace);
  if (n_tokens <= DECODE_TOKENS)
    return flint_moe_decode_bf16(dims, n_tokens, x_bf16, residual_bf16, w_router_bf16, logit_bias, w13_bf16, w2_bf16,
                                 ws13_bf16, ws2_bf16, out_bf16, topk_idx_out, topk_w_out, ws + DECODE_WS,
                                 decode_ws_bytes(n_tokens), stream);
  const Layer at(n_tokens);
  LinearArgs r = {};
  r.x = static_cast<const uint16_t*>(x_bf16);
  r.w = static_cast<const uint16_t*>(w_router_bf16);
  r.out = ws + at.logits;
  r.n_groups = 1;
  r.n_rows = r.n_x = n_tokens;
  r.n_in = H;
  r.n_out = E;
  r.out_f32 = 1;
  r.ws = workspace;
  if ((st = launch_linear(r, stream)) != FLINT_OK) return st;

  SelectArgs s = {};
  s.logits = reinterpret_cast<const float*>(ws + at.logits);
  s.bias = logit_bias;
  s.select_only = dims->offset_mode == FLINT_OFFSET_SELECT;
  s.n = n_tokens;
  s.idx = reinterpret_cast<int*>(ws + at.idx);
  s.w = reinterpret_cast<float*>(ws + at.w);
  s.start = reinterpret_cast<int*>(ws + at.start);
  s.row_token = reinterpret_cast<int*>(ws + at.row_token);
  s.pair_row = reinterpret_cast<int*>(ws + at.pair_row);
  s.idx_out = topk_idx_out;
  s.w_out = topk_w_out;
  s.shared_group = 1;
  s.counts = reinterpret_cast<uint8_t*>(ws + lin::WS_COUNTS);
  if ((st = cuda_status(launch_select(s, stream))) != FLINT_OK) return st;

  LinearArgs g = {};
  g.x = static_cast<const uint16_t*>(x_bf16);
  g.w = static_cast<const uint16_t*>(w13_bf16);
  g.w_last = static_cast<const uint16_t*>(ws13_bf16);
  g.out = ws + at.h;
  g.start = s.start;
  g.index = s.row_token;
  g.n_groups = E + 1;
  g.n_rows = n_tokens * SLOTS;
  g.n_x = n_tokens;
  g.n_in = H;
  g.n_out = I;
  g.act = ACT_SWIGLU;
  g.pair_out = 1;
  g.ws = workspace;
  if ((st = launch_linear(g, stream)) != FLINT_OK) return st;

  for (size_t c0 = 0; c0 < H; c0 += at.cols) {
    const int cols = (int)(H - c0 < at.cols ? H - c0 : at.cols);
    LinearArgs d = g;
    d.x = reinterpret_cast<const uint16_t*>(ws + at.h);
    d.w = static_cast<const uint16_t*>(w2_bf16) + c0 * I;
    d.w_last = static_cast<const uint16_t*>(ws2_bf16) + c0 * I;
    d.out = ws + at.y;
    d.index = nullptr;
    d.n_x = d.n_rows;
    d.n_in = I;
    d.n_out = cols;
    d.w_rows = H;
    d.scale = reinterpret_cast<uint8_t*>(ws + at.scale);
    d.act = ACT_NONE;
    d.pair_out = 0;
    d.pair_in = 1;
    if ((st = launch_linear(d, stream)) != FLINT_OK) return st;

    CombineArgs c = {};
    c.residual = static_cast<const uint16_t*>(residual_bf16) + c0;
    c.y = ws + at.y;
    c.y_shared = reinterpret_cast<const uint16_t*>(ws + at.y) + (size_t)n_tokens * TOPK * cols;
    c.scale = d.scale;
    c.scale_shared = d.scale + (size_t)n_tokens * TOPK * (cols / lin::SCALED);
    c.pair_row = s.pair_row;
    c.w = s.w;
    c.out = static_cast<uint16_t*>(out_bf16) + c0;
    c.n = n_tokens;
    c.cols = cols;
    if ((st = cuda_status(launch_combine(c, stream))) != FLINT_OK) return st;
  }
  return FLINT_OK;
}

}  // extern "C"
