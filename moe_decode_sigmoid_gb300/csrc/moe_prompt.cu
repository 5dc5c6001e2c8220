// moe_prompt.cu — around the experts' grouped products: the selection of every
// token's experts with the order of all (token, slot) pairs by expert, and the
// weighted sum that brings the experts' rows back to the tokens (bf16 rows, or the layer's
// scaled f16 of some of the columns).
//
// Bound: the selection by latencies and the ranking's issue (8192 tokens 10.6 us: 4.7 of
// ranking, 3.5 of counts and places, two launches; 17 tokens 3.3 us), the combine by HBM (8191
// tokens 48 us, 6.3 TB/s; half the columns of 8192 tokens' scaled f16 25 us, 6.1).
#include <cuda_fp16.h>

#include "common.cuh"
#include "linear.h"
#include "select.cuh"

namespace flint {
namespace {

using namespace lin;

constexpr int COMBINE = 256;                 // threads of the combine
constexpr int THREADS = 1024, WARPS = THREADS / 32;
constexpr int WORDS = CHUNK / 32;
static_assert(CHUNK <= 255, "a chunk's count of an expert fits a byte");

// The top k of one token's scores by one warp, as topk_warp ranks and weighs them.
//
// The k-th largest of the lanes' maxima (each of 8 scores) is at most the k-th largest
// score, and few scores reach it: those go to a lane each, in the experts' order, and are
// ranked there, ties to the lower lane.  Half the instructions of sorting every lane's
// scores, which more than 32 that reach it still take (8192 tokens, 12.0 -> 11.1 us; two
// tokens a warp side by side, 11.8: all of an SM's registers).
__device__ __forceinline__ void topk_any(const float* row, const float* bias, bool select_only,
                                         uint2* slots, int& idx_out, float& w_out) {
  const int lane = threadIdx.x & 31;
  uint32_t k[8], e[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float score = row[lane + 32 * j];
    k[j] = rank_key(bias != nullptr ? score + bias[lane + 32 * j] : score);
    e[j] = (uint32_t)(lane + 32 * j);
  }
  uint32_t top = k[0], least = 0;
#pragma unroll
  for (int j = 1; j < 8; ++j) top = max(top, k[j]);
#pragma unroll
  for (int r = 0; r < TOPK; ++r) {
    least = __reduce_max_sync(0xffffffffu, top);
    const uint32_t m = __ballot_sync(0xffffffffu, top == least);
    if (lane == __ffs(m) - 1) top = 0;   // below every key
  }
  int n = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t m = __ballot_sync(0xffffffffu, k[j] >= least);
    const int at = n + __popc(m & ((1u << lane) - 1u));
    if (k[j] >= least && at < 32) slots[at] = make_uint2(k[j], e[j]);
    n += __popc(m);
  }
  __syncwarp();
  int sel_e[TOPK];
  float sel_v[TOPK];
  if (n <= 32) {
    uint2 mine = make_uint2(0, 0);
    if (lane < n) mine = slots[lane];
#pragma unroll
    for (int r = 0; r < TOPK; ++r) {
      const uint32_t best = __reduce_max_sync(0xffffffffu, mine.x);
      const int win = __ffs(__ballot_sync(0xffffffffu, mine.x == best)) - 1;
      sel_e[r] = (int)__shfl_sync(0xffffffffu, mine.y, win);
      sel_v[r] = key2f(best);
      if (lane == win) mine.x = 0;
    }
  } else {
    topk_rank(k, e, sel_e, sel_v);
  }
  __syncwarp();   // the slots are the next token's
  float mine = 0.0f;
  idx_out = 0;
#pragma unroll
  for (int r = 0; r < TOPK; ++r)
    if (r == lane) {
      mine = sel_v[r];
      idx_out = sel_e[r];
    }
  if (select_only && lane < TOPK) mine = row[idx_out];
  const float s = 1.0f / (1.0f + expf(-mine));
  float sum = 0.0f;
#pragma unroll
  for (int r = 0; r < TOPK; ++r) sum += __shfl_sync(0xffffffffu, s, r);
  w_out = topk_weight(s, sum);
}

// Ranks of a chunk's pairs: an expert's tokens are the bits of a mask (an expert
// is at most once among a token's), so a pair's rank among its expert's is the bits
// below its token's, whatever order the warps ran in.
struct Chunk {
  uint32_t mask[E][WORDS];
  int base[E];      // first row of the expert's pairs of this chunk
  int all[E], before[E];
  int warp_tot[8];
  uint2 slots[WARPS][32];
  int expert[CHUNK * TOPK];
};

__device__ __forceinline__ void copy_choice(const SelectArgs& a, int p, int e, float w) {
  a.idx[p] = e;
  a.w[p] = w;
  if (a.idx_out != nullptr) a.idx_out[p] = e;
  if (a.w_out != nullptr) a.w_out[p] = w;
}

// The top k of the chunk's tokens, a warp each, and the experts' masks.
__device__ __forceinline__ void choose(const SelectArgs& a, Chunk& sh, int t0, int n) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < E * WORDS; i += THREADS) (&sh.mask[0][0])[i] = 0;
  __syncthreads();
  for (int t = warp; t < n; t += WARPS) {
    int e;
    float w;
    topk_any(a.logits + (size_t)(t0 + t) * E, a.bias, a.select_only != 0, sh.slots[warp], e, w);
    if (lane < TOPK) {
      sh.expert[t * TOPK + lane] = e;
      atomicOr(&sh.mask[e][t >> 5], 1u << (t & 31));
      copy_choice(a, (t0 + t) * TOPK + lane, e, w);
    }
  }
  __syncthreads();
}

__device__ __forceinline__ int mask_count(const uint32_t (&m)[WORDS]) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < WORDS; ++i) n += __popc(m[i]);
  return n;
}

// Rows of the chunk's pairs, once sh.base is known.
__device__ __forceinline__ void place(const SelectArgs& a, Chunk& sh, int t0, int n) {
  for (int p = threadIdx.x; p < n * TOPK; p += THREADS) {
    const int t = p / TOPK, e = sh.expert[p];
    int row = sh.base[e];
#pragma unroll
    for (int i = 0; i < WORDS; ++i)
      if (32 * i <= t) row += __popc(sh.mask[e][i] & (t - 32 * i >= 32 ? ~0u : (1u << (t - 32 * i)) - 1u));
    a.row_token[row] = t0 + t;
    a.pair_row[t0 * TOPK + p] = row;
  }
  if (a.shared_group)
    for (int t = threadIdx.x; t < n; t += THREADS) a.row_token[a.n * TOPK + t0 + t] = t0 + t;
}

// The experts' first rows from sh.all, their pairs of all chunks, and sh.before, those of
// the chunks before this one; by all threads.
__device__ __forceinline__ void starts(const SelectArgs& a, Chunk& sh, bool write) {
  if (threadIdx.x < E) {
    int total;
    const int excl = scan256(sh.all[threadIdx.x], sh.warp_tot, &total, [] { named_sync(1, E); });
    sh.base[threadIdx.x] = excl + sh.before[threadIdx.x];
    if (write) a.start[threadIdx.x] = excl;
  }
  if (write && threadIdx.x == E) {
    a.start[E] = a.n * TOPK;
    if (a.shared_group) a.start[E + 1] = a.n * (TOPK + 1);
  }
  __syncthreads();
}

// All tokens in one CTA.
__global__ void __launch_bounds__(THREADS) select_small_kernel(const SelectArgs a) {
  __shared__ Chunk sh;
  pdl_wait();
  pdl_trigger();
  choose(a, sh, 0, a.n);
  if (threadIdx.x < E) {
    sh.all[threadIdx.x] = mask_count(sh.mask[threadIdx.x]);
    sh.before[threadIdx.x] = 0;
  }
  __syncthreads();
  starts(a, sh, true);
  place(a, sh, 0, a.n);
}

// Many tokens, a chunk a CTA: the choice and the chunks' counts, a byte each, ...
__global__ void __launch_bounds__(THREADS) select_choose_kernel(const SelectArgs a) {
  __shared__ Chunk sh;
  pdl_wait();
  pdl_trigger();
  const int t0 = blockIdx.x * CHUNK, n = min(CHUNK, a.n - t0);
  choose(a, sh, t0, n);
  if (threadIdx.x < E) a.counts[blockIdx.x * E + threadIdx.x] = (uint8_t)mask_count(sh.mask[threadIdx.x]);
}

// ... and the rows.  Sixteen groups of 64 threads sum every sixteenth chunk's counts, four
// experts a thread.
__global__ void __launch_bounds__(THREADS) select_place_kernel(const SelectArgs a) {
  __shared__ Chunk sh;
  __shared__ int4 all_of[16][E / 4], before_of[16][E / 4];
  pdl_wait();
  pdl_trigger();
  const int t0 = blockIdx.x * CHUNK, n = min(CHUNK, a.n - t0);
  static_assert(CHUNK * TOPK <= THREADS, "a pair a thread");
  const int e = (int)threadIdx.x < n * TOPK ? a.idx[t0 * TOPK + threadIdx.x] : 0;
  for (int i = threadIdx.x; i < E * WORDS; i += THREADS) (&sh.mask[0][0])[i] = 0;
  const int quad = threadIdx.x & 63, first = threadIdx.x >> 6;
  int all[4] = {}, before[4] = {};
#pragma unroll
  for (int k = 0; k < MAX_CHUNKS / 16; ++k) {
    const int i = first + 16 * k;
    if (i < (int)gridDim.x) {
      const uint32_t v = __ldcg(reinterpret_cast<const uint32_t*>(a.counts + i * E + 4 * quad));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = (v >> (8 * j)) & 255;
        all[j] += c;
        if (i < (int)blockIdx.x) before[j] += c;
      }
    }
  }
  all_of[first][quad] = make_int4(all[0], all[1], all[2], all[3]);
  before_of[first][quad] = make_int4(before[0], before[1], before[2], before[3]);
  __syncthreads();
  if ((int)threadIdx.x < n * TOPK) {
    const int t = threadIdx.x / TOPK;
    sh.expert[threadIdx.x] = e;
    atomicOr(&sh.mask[e][t >> 5], 1u << (t & 31));
  }
  if (threadIdx.x < 2 * E) {
    const int* of = reinterpret_cast<const int*>(threadIdx.x < E ? all_of : before_of);
    int sum = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += of[i * E + (threadIdx.x & (E - 1))];
    (threadIdx.x < E ? sh.all : sh.before)[threadIdx.x & (E - 1)] = sum;
  }
  __syncthreads();
  starts(a, sh, blockIdx.x == 0);
  place(a, sh, t0, n);
}

// Two 16-bit values of an expert's row, without their scale.
template <bool SCALED_F16>
__device__ __forceinline__ float2 two_of(uint32_t w) {
  if constexpr (SCALED_F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(bf_lo(w), bf_hi(w));
}
__device__ __forceinline__ float scale_of(const uint8_t* at) { return __uint_as_float((uint32_t)*at << 23); }

// A token a CTA, 8 values of the row a thread.  A scale, a power of two, goes into its row's
// weight.
template <bool SCALED_F16>
__global__ void __launch_bounds__(COMBINE) combine_kernel(const CombineArgs a) {
  static_assert(H == 8 * COMBINE, "8 values a thread");
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x;
  const size_t at = (size_t)t * H + 8 * threadIdx.x;
  int row[TOPK];
  float w[TOPK];
#pragma unroll
  for (int j = 0; j < TOPK; ++j) {
    row[j] = a.pair_row[t * TOPK + j];
    w[j] = a.w[t * TOPK + j];
  }
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const auto row_part = [&](const void* y, int i) {
    return __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(y) + (size_t)i * a.cols + 8 * threadIdx.x));
  };
  const int block = 8 * threadIdx.x / SCALED;
  uint4 v[TOPK], s = zero;
  float ws = 1.0f;
  const uint4 r = __ldcs(reinterpret_cast<const uint4*>(a.residual + at));
  if (a.y_shared != nullptr) {
    s = row_part(a.y_shared, t);
    if constexpr (SCALED_F16) ws = scale_of(a.scale_shared + (size_t)t * (a.cols / SCALED) + block);
  }
#pragma unroll
  for (int j = 0; j < TOPK; ++j) {
    v[j] = zero;
    if ((unsigned)row[j] < (unsigned)(a.n * TOPK)) {
      v[j] = row_part(a.y, row[j]);
      if constexpr (SCALED_F16) w[j] *= scale_of(a.scale + (size_t)row[j] * (a.cols / SCALED) + block);
    } else {
      w[j] = 0.0f;
    }
  }
  const uint32_t rw[4] = {r.x, r.y, r.z, r.w}, sw[4] = {s.x, s.y, s.z, s.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 shared = two_of<SCALED_F16>(sw[i]);
    float lo = fmaf(ws, shared.x, bf_lo(rw[i])), hi = fmaf(ws, shared.y, bf_hi(rw[i]));
#pragma unroll
    for (int j = 0; j < TOPK; ++j) {
      const float2 y = two_of<SCALED_F16>(i == 0 ? v[j].x : i == 1 ? v[j].y : i == 2 ? v[j].z : v[j].w);
      lo = fmaf(w[j], y.x, lo);
      hi = fmaf(w[j], y.y, hi);
    }
    o[i] = pack_bf2(lo, hi);
  }
  *reinterpret_cast<uint4*>(a.out + at) = make_uint4(o[0], o[1], o[2], o[3]);
}

template <class Args>
cudaError_t launch(void (*kernel)(const Args), int grid, int threads, const Args& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_select(const SelectArgs& a, cudaStream_t stream) {
  const int chunks = (a.n + CHUNK - 1) / CHUNK;
  if (chunks == 1) return launch(select_small_kernel, 1, THREADS, a, stream);
  const cudaError_t e = launch(select_choose_kernel, chunks, THREADS, a, stream);
  return e != cudaSuccess ? e : launch(select_place_kernel, chunks, THREADS, a, stream);
}

cudaError_t launch_combine(const CombineArgs& a, cudaStream_t stream) {
  return a.scale != nullptr ? launch(combine_kernel<true>, a.n, a.cols / 8, a, stream)
                            : launch(combine_kernel<false>, a.n, a.cols / 8, a, stream);
}

}  // namespace flint
