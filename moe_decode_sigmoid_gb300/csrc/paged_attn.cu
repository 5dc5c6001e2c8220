// paged_attn.cu — grouped-query attention over a paged KV cache.
#include "paged.cuh"
#include "paged_work.cuh"

namespace flint {
namespace {

constexpr int WARPS = 4;

template <bool FP8>
__device__ __forceinline__ void load4(const void* cache, const float* scale, size_t row, int nkv,
                                      int kvh, int lane, float (&x)[4]) {
  const size_t at = (row * nkv + kvh) * pg::HD + 4 * lane;
  if constexpr (FP8) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(cache) + at);
    const float s = scale[(row >> 4) * nkv + kvh];
    const float2 p = pg::f16x2_to_f32(pg::e4m3x2_to_f16x2(w & 0xffffu));
    const float2 q = pg::f16x2_to_f32(pg::e4m3x2_to_f16x2(w >> 16));
    x[0] = p.x * s;
    x[1] = p.y * s;
    x[2] = q.x * s;
    x[3] = q.y * s;
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(cache) + at);
    x[0] = bf_lo(w.x);
    x[1] = bf_hi(w.x);
    x[2] = bf_lo(w.y);
    x[3] = bf_hi(w.y);
  }
}

}  // namespace

// One CTA per (row, query head), its warps striding over the keys, each with a
// running maximum, sum and output (4 of the 128 elements a lane).
template <bool FP8>
__global__ void __launch_bounds__(WARPS * 32) paged_attn_kernel(const __grid_constant__ PagedAttnArgs a) {
  using namespace pg;
  __shared__ int s_seq;
  __shared__ float s_m[WARPS], s_l[WARPS], s_o[WARPS][HD];
  pdl_wait();
  pdl_trigger();
  const PagedView& b = a.b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = blockIdx.x, h = blockIdx.y, kvh = h / b.group, nq = b.nkv * b.group;
  if (tid == 0) s_seq = -1;
  __syncthreads();
  for (int s = tid; s < b.n_seqs; s += WARPS * 32) {
    const Seq q = load_seq(b, s);
    if (t >= q.q0 && t < q.q0 + q.n) s_seq = s;
  }
  __syncthreads();
  const int s = s_seq;
  if (s < 0) return;
  const Seq sq = load_seq(b, s);
  const int pos = sq.first + (t - sq.q0);
  const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  float q[4], o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const uint2 w = *reinterpret_cast<const uint2*>(a.q + ((size_t)t * nq + h) * HD + 4 * lane);
  q[0] = bf_lo(w.x);
  q[1] = bf_hi(w.x);
  q[2] = bf_lo(w.y);
  q[3] = bf_hi(w.y);
  float m = -INFINITY, l = 0.0f;
  for (int j = lo + warp; j <= pos; j += WARPS) {
    const int row = cache_row(b, s, j);
    if (row < 0) continue;
    float k[4], v[4];
    load4<FP8>(a.k_cache, a.k_scale, row, b.nkv, kvh, lane, k);
    load4<FP8>(a.v_cache, a.v_scale, row, b.nkv, kvh, lane, v);
    const float sc = a.scale_log2 *
        warp_sum(fmaf(q[0], k[0], fmaf(q[1], k[1], fmaf(q[2], k[2], q[3] * k[3]))));
    const float mn = fmaxf(m, sc);
    const float f = exp2f(m - mn), p = exp2f(sc - mn);
    l = fmaf(l, f, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fmaf(o[i], f, p * v[i]);
    m = mn;
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s_o[warp][4 * lane + i] = o[i];
  __syncthreads();
  float mm = a.sinks ? a.sinks[h] * 1.4426950408889634f : -INFINITY;
  const float sink = mm;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) mm = fmaxf(mm, s_m[i]);
  float ll = sink > -INFINITY ? exp2f(sink - mm) : 0.0f, oo = 0.0f;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    const float f = s_m[i] > -INFINITY ? exp2f(s_m[i] - mm) : 0.0f;
    ll = fmaf(s_l[i], f, ll);
    oo = fmaf(s_o[i][tid], f, oo);
  }
  a.out[((size_t)t * nq + h) * HD + tid] = f2bf(ll > 0.0f ? oo / ll : (ll == 0.0f ? 0.0f : ll));
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, bool fp8, int sms, cudaStream_t stream) {
  if (a.b.max_q == 1) return launch_paged_decode(a, fp8, sms, stream);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.b.n_tokens, a.b.nkv * a.b.group, 1);
  cfg.blockDim = dim3(WARPS * 32, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return fp8 ? cudaLaunchKernelEx(&cfg, paged_attn_kernel<true>, a)
             : cudaLaunchKernelEx(&cfg, paged_attn_kernel<false>, a);
}

size_t paged_attn_workspace_clear_bytes() { return pg::WS_TICKETS; }
size_t paged_attn_workspace_bytes() { return pg::attn_ws_bytes(); }

}  // namespace flint
