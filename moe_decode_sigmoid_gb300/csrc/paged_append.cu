// paged_append.cu — a step's or a prompt's keys and values into a paged cache:
// per-head Q/K RMSNorm, rotary embedding and the cache write (bf16, or E4M3
// codes with a power-of-two scale per 16-token block and KV head), one kernel.
//
// For a row at position p: q and k heads n[i] = x[i] / sqrt(mean x^2 + eps) *
// g[i], then, if theta > 0, elements i and i + 64 turn by p * theta^(-2i/128);
// q goes to q_out, k and v to cache row page_table[p / page] * page + p % page.
// E4M3: s = the smallest power of two with amax <= 448 s over the block's new
// values; a block with earlier tokens keeps the larger of s and its old scale
// and rewrites their codes when it grows.  A power of two only moves E4M3's
// exponent, so nothing but values that become subnormal is rounded twice, and
// a floating-point code loses nothing to a scale that is not the exact maximum.
//
// Bound: bandwidth for prompts (per token 10 KiB in, 8 KiB + 2 KiB or 1 KiB out
// at 32 / 4 heads), latency for single tokens.  A CTA takes one block of one
// sequence (at most 16 tokens, the unit that shares a scale) and one KV head
// with its query heads, so that no scale needs a second kernel or an exchange
// between CTAs.  It finds its block by a scan of the sequences' block counts:
// the host does not know them.
#include "paged.cuh"

namespace flint {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;

// Blocks of its cache a sequence appends to.
__device__ __forceinline__ int blocks_of(const pg::Seq& q) {
  return q.n > 0 ? ((q.len - 1) >> 4) - (q.first >> 4) + 1 : 0;
}

// 4 bf16 (8 bytes) -> 4 fp32.
__device__ __forceinline__ void bf4(const uint2& w, float (&x)[4]) {
  x[0] = bf_lo(w.x);
  x[1] = bf_hi(w.x);
  x[2] = bf_lo(w.y);
  x[3] = bf_hi(w.y);
}
__device__ __forceinline__ float finite_max(const float (&x)[4]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float a = fabsf(x[j]);
    m = a <= 3.402823466e38f ? fmaxf(m, a) : m;
  }
  return m;
}

// Exponent of the smallest power of two whose 448-fold (1.75 * 2^8) is >= amax.
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, -40), 40);
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

}  // namespace

template <bool FP8>
__global__ void __launch_bounds__(THREADS) paged_append_kernel(const __grid_constant__ PagedAppendArgs a) {
  using namespace pg;
  __shared__ int s_warp[WARPS];
  __shared__ int s_seq, s_blk;
  __shared__ float2 s_cs[BLOCK][HD / 2];
  __shared__ float s_amax[2][WARPS];
  pdl_wait();  // the projection rows come from the preceding kernel
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, kvh = blockIdx.y;
  const PagedView& b = a.b;

  // Which sequence and block: thread s counts sequence s's blocks.
  Seq mine{};
  int cnt = 0;
  if (tid < b.n_seqs) {
    mine = load_seq(b, tid);
    cnt = blocks_of(mine);
  }
  int incl = cnt;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_warp[warp] = incl;
  if (tid == 0) s_seq = -1;
  __syncthreads();
  int before = incl - cnt;
  for (int w = 0; w < warp; ++w) before += s_warp[w];
  const int task = blockIdx.x;
  if (task >= before && task < before + cnt) {
    s_seq = tid;
    s_blk = task - before;
  }
  __syncthreads();
  const int s = s_seq;
  if (s < 0) return;
  const Seq q = load_seq(b, s);
  const int base = ((q.first >> 4) + s_blk) << 4;  // first position of the block
  const int lo = max(base, q.first), hi = min(base + BLOCK, q.len);
  const int n = hi - lo;                            // tokens of this CTA
  const int t0 = q.q0 + (lo - q.first);             // their first row
  // Blocks divide pages, so one look-up serves the block.
  const int row0 = base >= 0 ? cache_row(b, s, base) : -1;

  if (a.rope) {
    constexpr double INV_TWO_PI = 0.15915494309189535;  // 1 / (2 pi)
    constexpr double TWO_PI_HI = 6.283185307179586;     // 2 pi = HI + LO
    constexpr double TWO_PI_LO = 2.4492935982947064e-16;
    for (int i = tid; i < n * (HD / 2); i += THREADS) {
      const double ang = (double)(lo + (i >> 6)) * a.inv_freq[i & 63];
      const double k = rint(ang * INV_TWO_PI);
      const double r = fma(-k, TWO_PI_LO, fma(-k, TWO_PI_HI, ang));
      float sn, cs;
      sincosf((float)r, &sn, &cs);
      s_cs[i >> 6][i & 63] = make_float2(cs, sn);
    }
  }
  __syncthreads();

  const int nq = b.nkv * b.group;
  const size_t row_len = (size_t)(nq + 2 * b.nkv) * HD;
  // One head's row: lane l holds elements 4l .. 4l + 3, whose rotation partners
  // are lane l ^ 16's.
  auto normed = [&](const uint16_t* src, const uint16_t* gain, int tok, float (&x)[4]) {
    bf4(*reinterpret_cast<const uint2*>(src + 4 * lane), x);
    float g[4];
    bf4(*reinterpret_cast<const uint2*>(gain + 4 * lane), g);
    const float ss = warp_sum(fmaf(x[0], x[0], fmaf(x[1], x[1], fmaf(x[2], x[2], x[3] * x[3]))));
    const float inv = 1.0f / sqrtf(ss / (float)HD + a.eps);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = x[j] * inv * g[j];
    if (a.rope) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float other = __shfl_xor_sync(0xffffffffu, x[j], 16);
        const float2 cs = s_cs[tok][(lane & 15) * 4 + j];
        x[j] = x[j] * cs.x + (lane < 16 ? -other : other) * cs.y;
      }
    }
  };

  // Keys and values: warp w has tokens w and w + 8.
  constexpr int TPW = BLOCK / WARPS;
  float k[TPW][4], v[TPW][4];
  float mk = 0.0f, mv = 0.0f;
#pragma unroll
  for (int i = 0; i < TPW; ++i) {
    const int tok = warp + i * WARPS;
    if (tok < n) {
      const uint16_t* row = a.qkv + (size_t)(t0 + tok) * row_len;
      normed(row + (size_t)(nq + kvh) * HD, a.k_norm, tok, k[i]);
      bf4(*reinterpret_cast<const uint2*>(row + (size_t)(nq + b.nkv + kvh) * HD + 4 * lane), v[i]);
      mk = fmaxf(mk, finite_max(k[i]));
      mv = fmaxf(mv, finite_max(v[i]));
    }
  }
  if constexpr (FP8) {
    mk = warp_max(mk);
    mv = warp_max(mv);
    if (lane == 0) {
      s_amax[0][warp] = mk;
      s_amax[1][warp] = mv;
    }
    __syncthreads();
    if (row0 >= 0) {
      const size_t sc = (size_t)(row0 >> 4) * b.nkv + kvh;
      const int kept = lo - base;  // earlier tokens of the block
      const float old_k = kept > 0 ? a.k_scale[sc] : 0.0f;
      const float old_v = kept > 0 ? a.v_scale[sc] : 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        mk = fmaxf(mk, s_amax[0][w]);
        mv = fmaxf(mv, s_amax[1][w]);
      }
      const float new_k = fmaxf(exp2i(scale_exp(mk)), old_k);
      const float new_v = fmaxf(exp2i(scale_exp(mv)), old_v);
      uint8_t* kc = static_cast<uint8_t*>(a.k_cache);
      uint8_t* vc = static_cast<uint8_t*>(a.v_cache);
      auto rewrite = [&](uint8_t* cache, float ratio) {
        for (int r = warp; r < kept; r += WARPS) {
          uint32_t* p = reinterpret_cast<uint32_t*>(cache + ((size_t)(row0 + r) * b.nkv + kvh) * HD) + lane;
          const uint32_t w = *p;
          const float2 x = f16x2_to_f32(e4m3x2_to_f16x2(w & 0xffffu));
          const float2 y = f16x2_to_f32(e4m3x2_to_f16x2(w >> 16));
          *p = f32x2_to_e4m3x2(x.x * ratio, x.y * ratio) | f32x2_to_e4m3x2(y.x * ratio, y.y * ratio) << 16;
        }
      };
      if (kept > 0 && new_k > old_k) rewrite(kc, old_k / new_k);
      if (kept > 0 && new_v > old_v) rewrite(vc, old_v / new_v);
      __syncthreads();  // every thread has read the old scales
      if (tid == 0) {
        a.k_scale[sc] = new_k;
        a.v_scale[sc] = new_v;
      }
      const float ik = 1.0f / new_k, iv = 1.0f / new_v;  // powers of two: exact
#pragma unroll
      for (int i = 0; i < TPW; ++i) {
        const int tok = warp + i * WARPS;
        if (tok < n) {
          const size_t at = ((size_t)(row0 + (lo - base) + tok) * b.nkv + kvh) * HD + 4 * lane;
          *reinterpret_cast<uint32_t*>(kc + at) =
              f32x2_to_e4m3x2(k[i][0] * ik, k[i][1] * ik) | f32x2_to_e4m3x2(k[i][2] * ik, k[i][3] * ik) << 16;
          *reinterpret_cast<uint32_t*>(vc + at) =
              f32x2_to_e4m3x2(v[i][0] * iv, v[i][1] * iv) | f32x2_to_e4m3x2(v[i][2] * iv, v[i][3] * iv) << 16;
        }
      }
    }
  } else if (row0 >= 0) {
    uint16_t* kc = static_cast<uint16_t*>(a.k_cache);
    uint16_t* vc = static_cast<uint16_t*>(a.v_cache);
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      const int tok = warp + i * WARPS;
      if (tok < n) {
        const size_t at = ((size_t)(row0 + (lo - base) + tok) * b.nkv + kvh) * HD + 4 * lane;
        *reinterpret_cast<uint2*>(kc + at) = make_uint2(pack_bf2(k[i][0], k[i][1]), pack_bf2(k[i][2], k[i][3]));
        // bf16 values widened and narrowed again: bit for bit the input but for
        // a NaN's payload, so the words are copied instead.
        *reinterpret_cast<uint2*>(vc + at) = *reinterpret_cast<const uint2*>(
            a.qkv + (size_t)(t0 + tok) * row_len + (size_t)(nq + b.nkv + kvh) * HD + 4 * lane);
      }
    }
  }

  // The group's query heads.
  for (int i = warp; i < n * b.group; i += WARPS) {
    const int tok = i / b.group, h = kvh * b.group + i % b.group;
    float x[4];
    normed(a.qkv + (size_t)(t0 + tok) * row_len + (size_t)h * HD, a.q_norm, tok, x);
    *reinterpret_cast<uint2*>(a.q_out + ((size_t)(t0 + tok) * nq + h) * HD + 4 * lane) =
        make_uint2(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]));
  }
}

cudaError_t launch_paged_append(const PagedAppendArgs& a, bool fp8, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  // A sequence of n rows touches at most min(n, n / 16 + 2) blocks.
  const int most = a.b.n_tokens / pg::BLOCK + 2 * a.b.n_seqs;
  cfg.gridDim = dim3(a.b.n_tokens < most ? a.b.n_tokens : most, a.b.nkv, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return fp8 ? cudaLaunchKernelEx(&cfg, paged_append_kernel<true>, a)
             : cudaLaunchKernelEx(&cfg, paged_append_kernel<false>, a);
}

}  // namespace flint
