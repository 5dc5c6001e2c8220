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
// the host does not know them.  A head's row belongs to 16 lanes, and a lane
// loads five of its up to ten rows before it uses the first: two round trips to
// memory instead of ten, with room for four CTAs on an SM.  A whole block (16
// tokens) has one token a lane and no index arithmetic: 33 -> 28 us for 5.5K
// tokens into E4M3, and the angles from steps of 1, 2, 4 and 8 tokens instead of
// a sine each: 25 us, 4.2 TB/s (its bytes at the copy rate: 16 us).  2.2K tokens
// into bf16: 10.5 us, 4.1 TB/s.  What is left is latency: half the warps an SM
// has room for, waiting on shared memory, shuffles and their rows in turn.
#include <type_traits>

#include "paged.cuh"

namespace flint {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32, ROWS = THREADS / 16;
constexpr int MOST = (pg::MAX_GROUP + 2) * pg::BLOCK / ROWS;  // rows a 16-lane group has at most
constexpr int BATCH = MOST / 2;                               // of them loaded at a time

// Blocks of its cache a sequence appends to.
__device__ __forceinline__ int blocks_of(const pg::Seq& q) {
  return q.n > 0 ? ((q.len - 1) >> 4) - (q.first >> 4) + 1 : 0;
}

// A lane's share of a row: elements 4l .. 4l + 3 and 64 + 4l .. 64 + 4l + 3, so
// that a rotation's pairs meet in one lane.
struct Row {
  uint2 a, b;
};
__device__ __forceinline__ Row load_row(const uint16_t* p) {
  return Row{*reinterpret_cast<const uint2*>(p), *reinterpret_cast<const uint2*>(p + pg::HD / 2)};
}
__device__ __forceinline__ void widen(const Row& w, float (&x)[8]) {
  const uint32_t v[4] = {w.a.x, w.a.y, w.b.x, w.b.y};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = bf_lo(v[j]);
    x[2 * j + 1] = bf_hi(v[j]);
  }
}
__device__ __forceinline__ Row narrow(const float (&x)[8]) {
  return Row{make_uint2(pg::pack_bf16(x[0], x[1]), pg::pack_bf16(x[2], x[3])),
             make_uint2(pg::pack_bf16(x[4], x[5]), pg::pack_bf16(x[6], x[7]))};
}
__device__ __forceinline__ void store_row(uint16_t* p, const Row& w) {
  *reinterpret_cast<uint2*>(p) = w.a;
  *reinterpret_cast<uint2*>(p + pg::HD / 2) = w.b;
}
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&x)[8], float f) {
  *reinterpret_cast<uint32_t*>(p) =
      pg::f32x2_to_e4m3x2(x[0] * f, x[1] * f) | pg::f32x2_to_e4m3x2(x[2] * f, x[3] * f) << 16;
  *reinterpret_cast<uint32_t*>(p + pg::HD / 2) =
      pg::f32x2_to_e4m3x2(x[4] * f, x[5] * f) | pg::f32x2_to_e4m3x2(x[6] * f, x[7] * f) << 16;
}
// Largest finite magnitude of a row: over this lane's 8 elements, then 16 lanes.
__device__ __forceinline__ float finite_max(const float (&x)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float a = fabsf(x[j]);
    m = a <= 3.402823466e38f ? fmaxf(m, a) : m;
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
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
__global__ void __launch_bounds__(THREADS, 4) paged_append_kernel(const __grid_constant__ PagedAppendArgs a) {
  using namespace pg;
  __shared__ int s_warp[WARPS];
  __shared__ Seq s_seq;
  __shared__ int s_blk, s_which;
  __shared__ __align__(16) float s_cos[BLOCK][HD / 2];  // read four at a time
  __shared__ __align__(16) float s_sin[BLOCK][HD / 2];
  __shared__ float2 s_step[4][HD / 2];           // turns by 1, 2, 4 and 8 tokens
  __shared__ int s_amax[2];  // of the new keys and values, as bits
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
  int before = cnt;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) s_warp[warp] = before;
  before -= cnt;
  if (tid == 0) s_which = -1;
  if (tid < 2) s_amax[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WARPS; ++w)
    if (w < warp) before += s_warp[w];
  const int task = blockIdx.x;
  if (task >= before && task < before + cnt) {
    s_which = tid;
    s_seq = mine;
    s_blk = task - before;
  }
  __syncthreads();
  const int s = s_which;
  if (s < 0) return;
  const Seq q = s_seq;
  const int base = ((q.first >> 4) + s_blk) << 4;  // first position of the block
  const int lo = max(base, q.first), hi = min(base + BLOCK, q.len);
  const int n = hi - lo;                            // tokens of this CTA
  const int t0 = q.q0 + (lo - q.first);             // their first row
  const int nq = b.nkv * b.group;

  // Row i: token i % n of head i / n, the key, the value, then the queries.
  // This lane's rows are hw, hw + 16, ...: in a whole block all of one token.
  const int hw = tid >> 4, l = tid & 15, rows = n * (b.group + 2);
  const int recip = (65536 + n - 1) / n;  // i / n for i < 160
  auto head_of = [&](int i) { return (i * recip) >> 16; };
  const Row k_gain = load_row(a.k_norm + 4 * l), q_gain = load_row(a.q_norm + 4 * l);
  // Blocks divide pages, so one look-up serves the block.
  const int row0 = base >= 0 ? cache_row(b, s, base) : -1;
  const int kept = lo - base;  // earlier tokens of the block
  const size_t sc = (size_t)(max(row0, 0) >> 4) * b.nkv + kvh;
  float old_k = 0.0f, old_v = 0.0f;
  if (FP8 && row0 >= 0 && kept > 0) {
    old_k = a.k_scale[sc];
    old_v = a.v_scale[sc];
  }
  // The keys are among the lanes' first rows, the values among the first two;
  // E4M3 keeps them until the block's scale is known.
  float key[8];
  Row val[2];

  auto rows_of = [&](auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;  // n is 16: no index arithmetic
    const uint16_t* tok_row = a.qkv + (size_t)(t0 + hw) * (nq + 2 * b.nkv) * HD + 4 * l;
    auto src_of = [&](int k) {
      const int i = hw + ROWS * k, j = WHOLE ? k : head_of(i);
      const int head = j == 0 ? nq + kvh : j == 1 ? nq + b.nkv + kvh : kvh * b.group + j - 2;
      if constexpr (WHOLE) return tok_row + head * HD;
      return a.qkv + ((size_t)(t0 + i - j * n) * (nq + 2 * b.nkv) + head) * HD + 4 * l;
    };
    Row raw[BATCH];
    auto load_batch = [&](int first) {
#pragma unroll
      for (int k = 0; k < BATCH; ++k)
        raw[k] = hw + ROWS * (first + k) < rows ? load_row(src_of(first + k))
                                                : Row{make_uint2(0u, 0u), make_uint2(0u, 0u)};
    };
    load_batch(0);
    // The first token's angles in fp64 (a position of 2^18 times a frequency near
    // 1 would leave an fp32 angle 0.03 rad off), reduced to [-pi, pi]; the others
    // turn on from there by steps of 1, 2, 4 and 8 tokens, whose angles fp32 holds
    // to 2^-21, at most four products after one another.  So a thread takes one
    // or two sines instead of four, and fp64, at two operations a clock and SM,
    // stays off the other tokens.
    if (a.rope) {
      constexpr double INV_TWO_PI = 0.15915494309189535;  // 1 / (2 pi)
      constexpr double TWO_PI_HI = 6.283185307179586;     // 2 pi = HI + LO
      constexpr double TWO_PI_LO = 2.4492935982947064e-16;
      const int e = tid & 63, part = tid >> 6;  // frequency; bit of the step, then four tokens
      if (n > 1) {
        const float ang = (float)(1 << part) * (float)a.inv_freq[e];
        float sn, cs;
        sincosf(ang, &sn, &cs);
        s_step[part][e] = make_float2(cs, sn);
      }
      if (tid < HD / 2) {
        const double ang = (double)lo * a.inv_freq[tid];
        const double k = rint(ang * INV_TWO_PI);
        const double r = fma(-k, TWO_PI_LO, fma(-k, TWO_PI_HI, ang));
        float sn, cs;
        sincosf((float)r, &sn, &cs);
        s_cos[0][tid] = cs;
        s_sin[0][tid] = sn;
      }
      if (n > 1) {
        __syncthreads();
        auto on = [&](float2 x, int bit) {
          const float2 y = s_step[bit][e];
          return make_float2(x.x * y.x - x.y * y.y, x.y * y.x + x.x * y.y);
        };
        float2 at[4];
        at[0] = make_float2(s_cos[0][e], s_sin[0][e]);
        if (part & 1) at[0] = on(at[0], 2);
        if (part & 2) at[0] = on(at[0], 3);
        at[1] = on(at[0], 0);
        at[2] = on(at[0], 1);
        at[3] = on(at[2], 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (part || i) {  // the first is there, and others read it
            s_cos[4 * part + i][e] = at[i].x;
            s_sin[4 * part + i][e] = at[i].y;
          }
      }
    }
    __syncthreads();

    float4 c4, s4;  // the token's turn
    auto turn_of = [&](int tok) {
      c4 = *reinterpret_cast<const float4*>(&s_cos[tok][4 * l]);
      s4 = *reinterpret_cast<const float4*>(&s_sin[tok][4 * l]);
    };
    if (WHOLE) turn_of(hw);
    // Norm and rotation of a row.
    auto turned = [&](const Row& w, const Row& gain, float (&x)[8]) {
      widen(w, x);
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = rsqrtf(ss / (float)HD + a.eps);
      float g[8];
      widen(gain, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = x[j] * inv * g[j];
      if (a.rope) {
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float lo = x[j], hi = x[4 + j];
          x[j] = lo * c[j] - hi * sn[j];
          x[4 + j] = hi * c[j] + lo * sn[j];
        }
      }
    };
#pragma unroll
    for (int k = 0; k < MOST; ++k) {
      const int i = hw + ROWS * k;
      if (WHOLE ? k >= b.group + 2 : !__any_sync(0xffffffffu, i < rows)) break;  // shuffles need the whole warp
      if (k == BATCH) load_batch(BATCH);
      const bool live = WHOLE || i < rows;
      const int j = WHOLE ? k : live ? head_of(i) : 2, tok = WHOLE ? hw : live ? i - j * n : 0;
      const Row w = raw[k % BATCH];
      float x[8];
      if (!WHOLE) turn_of(tok);
      if (!WHOLE || k != 1) turned(w, j == 0 ? k_gain : q_gain, x);
      if (k < 2 && (WHOLE || __any_sync(0xffffffffu, j < 2))) {
        if constexpr (FP8) {
          float v[8];
          widen(w, v);
          val[k] = w;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (k == 0) key[e] = x[e];
            if (j == 1) x[e] = v[e];
          }
          const float m = finite_max(x);
          if (j < 2 && l == 0) atomicMax(&s_amax[j], __float_as_int(m));
        } else if (j < 2 && row0 >= 0) {
          store_row(static_cast<uint16_t*>(j ? a.v_cache : a.k_cache) +
                        ((size_t)(row0 + kept + tok) * b.nkv + kvh) * HD + 4 * l,
                    j ? w : narrow(x));  // a value as it came, bit for bit
        }
      }
      if (live && j >= 2)
        store_row(a.q_out + ((size_t)(t0 + tok) * nq + kvh * b.group + j - 2) * HD + 4 * l, narrow(x));
    }
  };
  if (n == BLOCK)
    rows_of(std::true_type{});
  else
    rows_of(std::false_type{});
  if constexpr (FP8) {
    __syncthreads();
    if (row0 < 0) return;
    const float new_k = fmaxf(exp2i(scale_exp(__int_as_float(s_amax[0]))), old_k);
    const float new_v = fmaxf(exp2i(scale_exp(__int_as_float(s_amax[1]))), old_v);
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
    if (tid == 0) {
      a.k_scale[sc] = new_k;
      a.v_scale[sc] = new_v;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = hw + ROWS * k, j = i < rows ? head_of(i) : 2;
      if (j < 2) {  // 1 / a power of two: exact
        float x[8];
        widen(val[k], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = j ? x[e] : key[e];
        store_codes((j ? vc : kc) + ((size_t)(row0 + kept + i - j * n) * b.nkv + kvh) * HD + 4 * l, x,
                    1.0f / (j ? new_v : new_k));
      }
    }
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
