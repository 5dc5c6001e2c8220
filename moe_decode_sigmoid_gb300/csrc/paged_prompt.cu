// paged_prompt.cu — attention of prompts and drafts (several query rows a
// sequence) over a paged KV cache, on the tensor cores' tcgen05 path.
//
// The query heads that share a KV head are rows of one matrix: a tile is
// 128 / group tokens x group heads = 128 rows of one sequence, against tiles of
// 128 keys.  Per tile, with a running maximum m and sum l a row (2^x
// throughout, the scale carrying log2 e):
//   S = Q K^T (128 x 128 x 128),  p = 2^(S ks + lv - m),  O += P V
// E4M3: K and V are the codes as f16 (exact); a 16-key block's ks multiplies
// its scores, its vs enters the exponent as lv = log2 vs, and l gets p / vs, so
// P is held in f16 relative to the largest contribution whatever the blocks'
// scales.  Q is f16 too, each row scaled by a power of two (its largest element
// in [2^14, 2^15): a bf16 element stays exact down to 2^-31 of it).  bf16: Q, K
// and V as they are, P rounded to bf16, half a step 2^-8, as the output itself;
// l sums the weights before that rounding.
//
// Bound: the tensor cores for prompts (4 * 128 operations a query-key pair
// against 512 or 256 bytes a key), the cache's bytes for a few drafted tokens.
// One CTA per SM takes two tiles A and B at a time: while one tile's scores are
// with its softmax warps, the other's products run.  A and B are neighbouring
// tiles of a prompt (they share the keys they load), or, where a sequence
// brings no more than one tile, the even and the odd key tiles of that one.
//   warps 0-3, 4-7: softmax of A, of B; a thread has a row (TMEM lane)
//   warps 8-11:     bring K and V tiles into a ring in the operands' layout
//                   (cp.async; E4M3 codes by a staging ring, widened to f16);
//                   rows that no query of the item sees are zeroed there
//   warp 12:        one thread issues every mma
// TMEM: S_A, S_B, O_A, O_B, 128 columns each; P takes its S's place.  O is
// rescaled only when a row's maximum grows by more than 2^8.
//
// Work: items (tile pair of a sequence, KV head) of so many key tiles, laid end
// to end and cut into equal shares, as the next-token kernel cuts its rows; cut
// items are joined through the workspace by the CTA that arrives last.
#include "nv_util.cuh"
#include "paged.cuh"
#include "paged_work.cuh"
#include "tcgen05.cuh"

namespace flint {
namespace {

using namespace pg;

constexpr int THREADS = 512;
constexpr int TILE = 128;              // rows of a tile, keys of a tile
constexpr int OPER = TILE * HD * 2;    // bytes of an operand tile (16-bit): 2 blocks of 64 columns
constexpr int HALF = OPER / 2;
constexpr int STAGE = TILE * HD;       // bytes of a tile of codes
constexpr int MAX_ITEMS = 512;         // tile pairs: tokens / (tokens a pair) + sequences
constexpr int INFO = 8;                // tiles whose block scales are kept

template <bool FP8>
struct Cfg {
  static constexpr int RING = FP8 ? 3 : 4;     // operand tiles
  static constexpr int STAGES = FP8 ? 3 : 0;   // tiles of codes on their way
  static constexpr int AHEAD = 2;              // tiles copied ahead of the one handed over
  static constexpr int SMEM = 2 * OPER + RING * OPER + STAGES * STAGE + 1024;
};

struct Shared {
  uint64_t full[8], empty[8];        // ring slots: brought, used
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], drained;
  uint32_t tmem;
  int fail, last, cut[2], first, n_items;
  int scan[16];
  int pre[MAX_ITEMS + 1];            // key tiles (of all heads) before each item
  int4 item[MAX_ITEMS];              // {sequence, pair, first key tile, key tiles}
  int qpre[MAX_SEQS + 1];            // items before each sequence
  int4 seq[MAX_SEQS];                // {first row, rows, first position, -}
  float ks[INFO][8], lv[INFO][8], iv[INFO][8];   // a key tile's blocks
  int row[16][8];                    // a key tile's blocks: cache rows
};

static_assert(Cfg<true>::SMEM + sizeof(Shared) <= 227 * 1024, "fits");
static_assert(Cfg<false>::SMEM + sizeof(Shared) <= 227 * 1024, "fits");

// One share's part of an item.
struct Item {
  int seq, kvh, kt0, n;     // first key tile of this part, key tiles
  int tok0, tokens, pos0;   // first token row, tokens of the item, position of the first
  int q_row;                // row of q / out of tok0
  bool split;               // one tile: A has the even key tiles, B the odd ones
  int c0, c1;               // CTAs that share the item (c0 == c1: it is whole here)
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// a * k + d of two floats at once, and a + b.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t k, uint64_t d) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(k), "l"(d));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Two weights as the second product takes them (the first in the low half).
template <bool FP8>
__device__ __forceinline__ uint32_t pack_p(float lo, float hi) {
  uint32_t r;
  if constexpr (FP8)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Registers a thread of the calling warpgroup: 2 * 128 * 192 + 2 * 128 * 64 are
// the 512 * 128 the block starts with.
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const uint8_t* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Waits for a phase, a second at most; a wait that runs out (in any warp) ends
// every other one too.
__device__ __forceinline__ bool wait(Shared& sh, uint64_t& bar, uint32_t parity) {
  const uint32_t b = smem_addr(&bar);
  if (mbar_try_wait(b, parity)) return true;
  const uint64_t deadline = globaltimer_ns() + 1000000000ull;
  while (!mbar_try_wait(b, parity)) {
    if (*reinterpret_cast<volatile int*>(&sh.fail) != 0) return false;
    if (globaltimer_ns() > deadline) {
      *reinterpret_cast<volatile int*>(&sh.fail) = 1;
      return false;
    }
  }
  return true;
}

// The same for a whole warp, which goes on converged.
__device__ __forceinline__ bool warp_wait(Shared& sh, uint64_t& bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(sh, bar, parity));
}

}  // namespace

template <bool FP8>
__global__ void __launch_bounds__(THREADS, 1)
    paged_prompt_kernel(const __grid_constant__ PagedAttnArgs a) {
  using C = Cfg<FP8>;
  extern __shared__ uint8_t s_raw[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedView& b = a.b;
  const int nq = b.nkv * b.group;
  const int gshift = 31 - __clz(b.group);       // group is a power of two
  const int tile_toks = TILE >> gshift;         // tokens of a tile
  const uint32_t base = (smem_addr(s_raw) + 1023u) & ~1023u;
  const uint32_t q_smem = base, ring = base + 2 * OPER, stages = ring + C::RING * OPER;

  if (tid == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(smem_addr(&sh.full[i]), 128);
      mbar_init(smem_addr(&sh.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sh.q_full[i]), 128);
      mbar_init(smem_addr(&sh.s_full[i]), 1);
      mbar_init(smem_addr(&sh.p_full[i]), 128);
      mbar_init(smem_addr(&sh.o_full[i]), 1);
      sh.cut[i] = -1;
    }
    mbar_init(smem_addr(&sh.drained), 1);
    sh.fail = 0;
    fence_mbar_init();
  }
  if (warp == 12) tc::alloc512(smem_addr(&sh.tmem));
  pdl_wait();
  pdl_trigger();

  // ---- the items: sequences cut into tile pairs -------------------------------
  int cnt = 0, pre = 0;
  if (tid < MAX_SEQS) {
    if (tid < b.n_seqs) {
      const Seq q = load_seq(b, tid);
      sh.seq[tid] = make_int4(q.q0, q.n, q.first, 0);
      cnt = (q.n + 2 * tile_toks - 1) / (2 * tile_toks);
    }
    pre = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += v;
    }
    if (lane == 31) sh.scan[warp] = pre;
  }
  __syncthreads();
  if (tid < MAX_SEQS) {
    for (int w = 0; w < warp; ++w) pre += sh.scan[w];
    sh.qpre[tid + 1] = pre;
    if (tid == 0) sh.qpre[0] = 0;
  }
  __syncthreads();
  // Offsets that overlap could ask for more items than a call has tokens.
  const int n_items = min(sh.qpre[b.n_seqs], MAX_ITEMS);
  int4 info = make_int4(0, 0, 0, 0);
  cnt = 0;
  if (tid < n_items) {
    int lo = 0, hi = b.n_seqs;  // the sequence whose items include tid
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      (sh.qpre[mid] <= tid ? lo : hi) = mid;
    }
    const int4 sq = sh.seq[lo];
    const int pair = tid - sh.qpre[lo], tok = pair * 2 * tile_toks;
    const int first = sq.z + tok, last = sq.z + min(sq.y, tok + 2 * tile_toks) - 1;
    const int k0 = (a.window > 0 ? max(0, first - a.window + 1) : 0) >> 7;
    info = make_int4(lo, pair, k0, last >= 0 ? (last >> 7) + 1 - k0 : 0);
    sh.item[tid] = info;
    cnt = info.w * b.nkv;
  }
  pre = cnt;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, pre, o);
    if (lane >= o) pre += v;
  }
  if (lane == 31) sh.scan[warp] = pre;
  pre -= cnt;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) pre += total;
    total += sh.scan[w];
  }
  const int share = max((total + (int)gridDim.x - 1) / (int)gridDim.x, PR_MIN_SHARE);
  const int margin = share >> 4;
  if (tid < n_items) {
    sh.pre[tid + 1] = pre + cnt;
    if (tid == 0) sh.pre[0] = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long x = (long long)share * (blockIdx.x + k);
      if (pre <= x && x < pre + cnt) {  // this item holds the cut: move it to a near end
        const int off = (int)(x - pre) % info.w, rest = info.w - off;
        const int near = min(off, rest);
        sh.cut[k] = (int)x + (info.w <= PR_WHOLE || near <= margin ? (off <= rest ? -off : rest) : 0);
        if (k == 0) sh.first = tid;
      }
    }
    // Rows that see nothing: zeros.
    if (info.w == 0 && tid % gridDim.x == blockIdx.x) {
      const int4 sq = sh.seq[info.x];
      const int t0 = info.y * 2 * tile_toks, t1 = min(sq.y, t0 + 2 * tile_toks);
      uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)(sq.x + t0) * nq * HD);
      for (int i = 0; i < (t1 - t0) * nq * HD / 8; ++i) o[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sh.tmem;
  const int begin = sh.cut[0] < 0 ? total : sh.cut[0], end = sh.cut[1] < 0 ? total : sh.cut[1];

  // The part of an item at place `cur` of this CTA's share; it: its list entry.
  auto part = [&](int cur, int& it) {
    while (cur >= sh.pre[it + 1]) ++it;
    const int4 e = sh.item[it];
    const int4 sq = sh.seq[e.x];
    Item p;
    const int rel = cur - sh.pre[it];
    p.kvh = rel / e.w;
    const int off = rel - p.kvh * e.w;
    p.seq = e.x;
    p.kt0 = e.z + off;
    p.n = min(e.w - off, end - cur);
    p.tok0 = e.y * 2 * tile_toks;
    p.tokens = min(sq.y - p.tok0, 2 * tile_toks);
    p.pos0 = sq.z + p.tok0;
    p.q_row = sq.x + p.tok0;
    p.split = p.tokens <= tile_toks;
    const int row0 = cur - off;
    const int cut0 = (row0 + margin) / share + 1, cut1 = (row0 + e.w - margin - 1) / share;
    const bool whole = e.w <= PR_WHOLE || cut0 > cut1;
    p.c0 = whole ? 0 : cut0 - 1;
    p.c1 = whole ? 0 : cut1;
    return p;
  };

  if (warp < 8) {
    // ===== softmax, and the item's queries and outputs ===========================
    more_registers<192>();
    const int x = warp >> 2;               // tile A or B
    const int r = tid & 127;               // row of the tile
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_tm = tmem + lanes + 128 * x, o_tm = tmem + lanes + 256 + 128 * x;
    uint32_t s_phase = 0, o_phase = 0;
    const int head_in_group = r & (b.group - 1), tok_in_tile = r >> gshift;
    int tiles_before = 0;                  // key tiles this CTA has been through (INFO ring)
    // After a wait that ran out the items are only walked through: the other
    // tile's warps count on this one's arrivals at the joint barriers.
    bool ok = true;
    for (int cur = begin, it = sh.first; cur < end;) {
      const Item p = part(cur, it);
      cur += p.n;
      const int tok = tok_in_tile + (p.split ? 0 : x * tile_toks);
      const bool live = tok < p.tokens;
      const int pos = p.pos0 + min(tok, p.tokens - 1);
      const int head = p.kvh * b.group + head_in_group;

      // -- queries: this thread's row into the A operand's layout
      float qs = a.scale_log2;
      {
        const uint8_t* src = reinterpret_cast<const uint8_t*>(
            a.q + ((size_t)(p.q_row + (live ? tok : 0)) * nq + head) * HD);
        float up = 1.0f;
        if constexpr (FP8) {
          float mx = 0.0f;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const uint4 w = *reinterpret_cast<const uint4*>(src + 16 * c);
            const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) mx = fmaxf(mx, fmaxf(fabsf(bf_lo(v[j])), fabsf(bf_hi(v[j]))));
          }
          const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 127);
          up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
          qs *= __uint_as_float((uint32_t)(127 - 14 + e) << 23);
        }
        if (!p.split || x == 0) {
          const uint32_t dst = q_smem + x * OPER + r * 128;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            uint4 w = live ? *reinterpret_cast<const uint4*>(src + 16 * c) : make_uint4(0u, 0u, 0u, 0u);
            if constexpr (FP8) {
              w.x = nvu::f16x2_of(bf_lo(w.x) * up, bf_hi(w.x) * up);
              w.y = nvu::f16x2_of(bf_lo(w.y) * up, bf_hi(w.y) * up);
              w.z = nvu::f16x2_of(bf_lo(w.z) * up, bf_hi(w.z) * up);
              w.w = nvu::f16x2_of(bf_lo(w.w) * up, bf_hi(w.w) * up);
            }
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                             dst + (c >> 3) * HALF + (((c & 7) ^ (r & 7)) << 4)),
                         "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w)
                         : "memory");
          }
          tc::fence_smem_to_mma();
          mbar_arrive(smem_addr(&sh.q_full[x]));
        }
      }

      // -- the key tiles
      const int hi = pos, lo = a.window > 0 ? pos - a.window + 1 : 0;
      // the warp's rows see a tile whole if its first and its last row do
      const int hi_all = __shfl_sync(0xffffffffu, hi, 0), lo_all = __shfl_sync(0xffffffffu, lo, 31);
      float m = -INFINITY, l = 0.0f;
      const int step = p.split ? 2 : 1;
      bool any = false;
      for (int j = p.split ? x : 0; ok && j < p.n; j += step) {
        if (!(ok = warp_wait(sh, sh.s_full[x], s_phase))) break;
        s_phase ^= 1;
        tc::fence_after();
        const int slot = (tiles_before + j) & (INFO - 1);
        const int key0 = (p.kt0 + j) << 7;
        const bool masked = key0 + TILE - 1 > hi_all || key0 < lo_all;
        // What a block's scores are multiplied by; not 0, lest a masked score
        // becomes NaN (a query of zeros, a scale of 0).
        auto factor = [&](int blk) {
          return fmaxf(FP8 ? qs * sh.ks[slot][blk] : qs, 1.17549435e-38f);
        };
        uint32_t v[4][32];  // the row's scores, then its weights
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::ld32(s_tm + 32 * c, v[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::wait_ld(v[c]);
        if (masked) {  // columns outside [mlo, mhi] are not seen
          const int mlo = lo - key0, mhi = hi - key0;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * c + i < mlo || 32 * c + i > mhi) v[c][i] = 0xff800000u;  // -infinity
        }
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // a block of 16 keys
            float b4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b4[i] = __uint_as_float(v[c][16 * h + i]);
#pragma unroll
            for (int i = 4; i < 16; ++i) b4[i & 3] = fmaxf(b4[i & 3], __uint_as_float(v[c][16 * h + i]));
            const float bm = fmaxf(fmaxf(b4[0], b4[1]), fmaxf(b4[2], b4[3]));
            const float k = factor(2 * c + h);
            mx = fmaxf(mx, fmaf(bm, k, sh.lv[slot][2 * c + h]));
          }
        const bool grow = mx > m + 8.0f;
        if (__any_sync(0xffffffffu, grow)) {
          const float mn = fmaxf(m, mx);
          const float f = m > -INFINITY ? ex2(m - mn) : 0.0f;
          l *= f;
          m = mn;
          if (any) {  // the products so far
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              uint32_t w[16];
              tc::ld16(o_tm + 16 * c, w);
              tc::wait_ld(w);
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
              tc::st16(o_tm + 16 * c, w);
            }
          }
        }
        any = true;
        const float mu = m > -INFINITY ? m : 0.0f;
        uint64_t sums[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float k = factor(2 * c + h), d = sh.lv[slot][2 * c + h] - mu;
            const uint64_t k2 = pair(k, k), d2 = pair(d, d);
            if constexpr (FP8) sums[0] = sums[1] = 0ull;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float y0, y1;
              unpair(fma2(pair(__uint_as_float(v[c][16 * h + 2 * i]),
                               __uint_as_float(v[c][16 * h + 2 * i + 1])), k2, d2), y0, y1);
              y0 = ex2(y0);
              y1 = ex2(y1);
              sums[i & 1] = add2(sums[i & 1], pair(y0, y1));
              w[8 * h + i] = pack_p<FP8>(y0, y1);
            }
            if constexpr (FP8) {
              float y0, y1;
              unpair(add2(sums[0], sums[1]), y0, y1);
              l = fmaf(y0 + y1, sh.iv[slot][2 * c + h], l);
            }
          }
          tc::st16(s_tm + 16 * c, w);
        }
        if constexpr (!FP8) {
          float y0, y1;
          unpair(add2(sums[0], sums[1]), y0, y1);
          l += y0 + y1;
        }
        tc::wait_st();
        tc::fence_before();
        mbar_arrive(smem_addr(&sh.p_full[x]));
      }
      tiles_before += p.n;

      // -- the outputs
      if (ok && any) {
        ok = warp_wait(sh, sh.o_full[x], o_phase);
        o_phase ^= 1;
        tc::fence_after();
      }
      const bool whole = p.c0 == p.c1;
      uint16_t* out = a.out + ((size_t)(p.q_row + tok) * nq + head) * HD;
      if (whole && !p.split) {
        const float inv = row_factor(a, head, m, l);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tc::ld32(o_tm + 32 * c, v);
          tc::wait_ld(v);
          if (live) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 w;
              w.x = pack_bf2(__uint_as_float(v[8 * i]) * inv, __uint_as_float(v[8 * i + 1]) * inv);
              w.y = pack_bf2(__uint_as_float(v[8 * i + 2]) * inv, __uint_as_float(v[8 * i + 3]) * inv);
              w.z = pack_bf2(__uint_as_float(v[8 * i + 4]) * inv, __uint_as_float(v[8 * i + 5]) * inv);
              w.w = pack_bf2(__uint_as_float(v[8 * i + 6]) * inv, __uint_as_float(v[8 * i + 7]) * inv);
              *reinterpret_cast<uint4*>(out + 32 * c + 8 * i) = w;
            }
          }
        }
        continue;
      }
      // Partial: maxima, sums and unscaled outputs of this tile, [4 columns][row].
      {
        float* slot = pr_slot(a.ws, blockIdx.x, whole || (int)blockIdx.x == p.c0, x);
        __stcg(slot + r, m);
        __stcg(slot + TILE + r, any ? l : 0.0f);
        float4* o4 = reinterpret_cast<float4*>(slot + 2 * TILE);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          if (any) {
            tc::ld32(o_tm + 32 * c, v);
            tc::wait_ld(v);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            __stcg(o4 + (8 * c + i) * TILE + r,
                   any ? make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                     __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]))
                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f));
        }
      }
      __threadfence();
      named_sync(1, 256);
      if (!whole) {
        if (tid == 0) {
          uint32_t* ticket = ws_tickets(a.ws) + p.c0;
          const bool last = atomicAdd(ticket, 1u) == (uint32_t)(p.c1 - p.c0);
          if (last) *ticket = 0u;  // ready for the next call
          __threadfence();
          sh.last = last;
        }
        named_sync(1, 256);
        const bool last = sh.last != 0;
        named_sync(1, 256);  // sh.last is read before the next item sets it
        if (!last) continue;
      }
      // Join: a pair's tile each; a split tile's two halves of the columns.
      const int segs = whole ? 1 : p.c1 - p.c0 + 1, halves = p.split ? 2 : 1;
      auto slot_of = [&](int k, int h) {
        return pr_slot(a.ws, whole ? blockIdx.x : p.c0 + k, whole || k == 0, p.split ? h : x);
      };
      float mm = -INFINITY, ll = 0.0f;
      for (int k = 0; k < segs; ++k)
        for (int h = 0; h < halves; ++h) mm = fmaxf(mm, __ldcg(slot_of(k, h) + r));
      for (int k = 0; k < segs; ++k)
        for (int h = 0; h < halves; ++h) {
          const float* s = slot_of(k, h);
          const float mk = __ldcg(s + r);
          ll = fmaf(__ldcg(s + TILE + r), mk > -INFINITY ? ex2(mk - mm) : 0.0f, ll);
        }
      const float inv = row_factor(a, head, mm, ll);
      for (int c = p.split ? 4 * x : 0; c < (p.split ? 4 * x + 4 : 8); ++c) {  // 16 columns
        float o[16] = {};
        for (int k = 0; k < segs; ++k)
          for (int h = 0; h < halves; ++h) {
            const float* s = slot_of(k, h);
            const float mk = __ldcg(s + r), f = mk > -INFINITY ? ex2(mk - mm) : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 w = __ldcg(reinterpret_cast<const float4*>(s + 2 * TILE) + (4 * c + i) * TILE + r);
              o[4 * i] = fmaf(w.x, f, o[4 * i]);
              o[4 * i + 1] = fmaf(w.y, f, o[4 * i + 1]);
              o[4 * i + 2] = fmaf(w.z, f, o[4 * i + 2]);
              o[4 * i + 3] = fmaf(w.w, f, o[4 * i + 3]);
            }
          }
        if (live) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint4 w;
            w.x = pack_bf2(o[8 * i] * inv, o[8 * i + 1] * inv);
            w.y = pack_bf2(o[8 * i + 2] * inv, o[8 * i + 3] * inv);
            w.z = pack_bf2(o[8 * i + 4] * inv, o[8 * i + 5] * inv);
            w.w = pack_bf2(o[8 * i + 6] * inv, o[8 * i + 7] * inv);
            *reinterpret_cast<uint4*>(out + 16 * c + 8 * i) = w;
          }
        }
      }
      // Slots that a later item of this CTA writes are read by now.
      named_sync(1, 256);
    }
  } else if (warp < 12) {
    // ===== K and V tiles ===========================================================
    fewer_registers<64>();
    const int w4 = warp - 8;   // this warp brings keys 32 w4 .. + 31 of every tile
    constexpr int ES = FP8 ? 1 : 2;
    const size_t tok_bytes = (size_t)b.nkv * HD * ES;
    int u = 0;                 // tiles handed over (K and V alike)
    int tiles_before = 0;
    bool ok = true;
    for (int cur = begin, it = sh.first; ok && cur < end;) {
      const Item p = part(cur, it);
      cur += p.n;
      // Keys some query of the item sees; anything else is zeroed.
      const int see_hi = p.pos0 + p.tokens - 1;
      const int see_lo = a.window > 0 ? max(0, p.pos0 - a.window + 1) : 0;
      const int lead = p.split ? 2 : 1, loads = 2 * p.n;
      // Load i of the item: K of the first `lead` tiles, then V_j, K_(j + lead)
      // in turn; {tile, V?}.
      auto which = [&](int i) {
        const int ld = min(lead, p.n);
        if (i < ld) return make_int2(i, 0);
        const int k = i - ld;
        if (k < 2 * (p.n - ld)) return make_int2((k >> 1) + (k & 1 ? ld : 0), k & 1 ? 0 : 1);
        return make_int2(k - (p.n - ld), 1);
      };
      // Where the blocks lie: lane l holds block 2 w4 + l % 2 of tile 16 batch + l / 2.
      int now_row = -1, next_row = -1, have = -1;
      float now_ks = 0.0f, now_vs = 1.0f;
      auto look_up = [&](int batch) {
        const int tile = 16 * batch + (lane >> 1);
        const int key = ((p.kt0 + tile) << 7) + 32 * w4 + 16 * (lane & 1);
        return tile < p.n && key <= see_hi ? cache_row(b, p.seq, key) : -1;
      };
      // Copies load i; K also leaves its tile's block table.
      auto issue = [&](int i) {
        if (i < loads) {
          const int2 kv = which(i);
          const int tile = kv.x;
          if (kv.y == 0) {
            if ((tile >> 4) != have) {
              now_row = have < 0 ? look_up(0) : next_row;
              have = tile >> 4;
              next_row = look_up(have + 1);
              if constexpr (FP8) {
                if (now_row >= 0) {
                  const size_t at = (size_t)(now_row >> 4) * b.nkv + p.kvh;
                  now_ks = __ldg(a.k_scale + at);
                  // A scale of zero would take a block's weights out of the sum: 2^-100.
                  now_vs = fmaxf(__ldg(a.v_scale + at), 7.8886090522101181e-31f);
                }
              }
            }
            const int src = 2 * (tile & 15) + (lane & 1);
            const int row = __shfl_sync(0xffffffffu, now_row, src);
            const float ks = FP8 ? __shfl_sync(0xffffffffu, now_ks, src) : 1.0f;
            const float vs = FP8 ? __shfl_sync(0xffffffffu, now_vs, src) : 1.0f;
            if (lane < 2) {
              const int slot = (tiles_before + tile) & (INFO - 1), blk = 2 * w4 + lane;
              sh.row[(tiles_before + tile) & 15][blk] = row;
              sh.ks[slot][blk] = row >= 0 ? ks : 0.0f;
              sh.lv[slot][blk] = row < 0 ? -INFINITY : FP8 ? log2f(vs) : 0.0f;
              sh.iv[slot][blk] = row >= 0 && FP8 ? 1.0f / vs : 1.0f;
            }
            __syncwarp();
          }
          const uint8_t* cache = static_cast<const uint8_t*>(kv.y ? a.v_cache : a.k_cache);
          const int key0 = ((p.kt0 + tile) << 7) + 32 * w4;
          constexpr int CH = FP8 ? 8 : 16;       // 16-byte chunks of a key
          constexpr int STEP = 32 / CH;          // keys copied at a time
          const int cr = lane / CH, cc = lane % CH;
          const uint32_t dst = FP8 ? stages + ((u + i) % (FP8 ? C::STAGES : 1)) * STAGE
                                   : ring + ((u + i) % C::RING) * OPER;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = sh.row[(tiles_before + tile) & 15][2 * w4 + h];
            const uint8_t* src = cache + (size_t)max(row, 0) * tok_bytes + (size_t)p.kvh * HD * ES + 16 * cc;
#pragma unroll
            for (int j = 0; j < 16 / STEP; ++j) {
              const int k = STEP * j + cr, r = 32 * w4 + 16 * h + k;  // row of the tile
              const int key = key0 + 16 * h + k;
              const bool live = row >= 0 && key >= see_lo && key <= see_hi;
              const uint32_t at = FP8 ? r * HD + ((cc ^ ((r & 1) << 2)) << 4)
                                      : (cc >> 3) * HALF + r * 128 + (((cc & 7) ^ (r & 7)) << 4);
              cp_async16(dst + at, src + (size_t)k * tok_bytes, live);
            }
          }
        }
        cp_commit();
      };
      auto free_slot = [&](int i) {  // the ring slot of load i
        const int n = u + i;
        return n < C::RING || warp_wait(sh, sh.empty[n % C::RING], ((n / C::RING) & 1) ^ 1);
      };
      if constexpr (FP8) {
        for (int i = 0; i < C::AHEAD; ++i) issue(i);
        for (int i = 0; i < loads; ++i) {
          issue(i + C::AHEAD);
          cp_wait<C::AHEAD>();
          __syncwarp();
          if (!(ok = free_slot(i))) break;
          const uint32_t src = stages + ((u + i) % C::STAGES) * STAGE, dst = ring + ((u + i) % C::RING) * OPER;
#pragma unroll
          for (int j = 0; j < 8; ++j) {  // 8 keys x 4 chunks of codes a time
            const int r = 32 * w4 + 8 * (j >> 1) + (lane >> 2), c = (lane & 3) + 4 * (j & 1);
            uint4 w;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                         : "r"(src + r * HD + ((c ^ ((r & 1) << 2)) << 4)));
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int ch = 2 * c + h;  // chunk of the operand row
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                               dst + (ch >> 3) * HALF + r * 128 + (((ch & 7) ^ (r & 7)) << 4)),
                           "r"(e4m3x2_to_f16x2(x[2 * h] & 0xffffu)), "r"(e4m3x2_to_f16x2(x[2 * h] >> 16)),
                           "r"(e4m3x2_to_f16x2(x[2 * h + 1] & 0xffffu)),
                           "r"(e4m3x2_to_f16x2(x[2 * h + 1] >> 16))
                           : "memory");
            }
          }
          __syncwarp();  // the stage is read before it is copied into again
          tc::fence_smem_to_mma();
          mbar_arrive(smem_addr(&sh.full[(u + i) % C::RING]));
        }
      } else {
        for (int i = 0; i < C::AHEAD && ok; ++i) {
          if (i < loads) ok = free_slot(i);
          if (ok) issue(i);
        }
        for (int i = 0; ok && i < loads; ++i) {
          if (i + C::AHEAD < loads && !(ok = free_slot(i + C::AHEAD))) break;
          issue(i + C::AHEAD);
          cp_wait<C::AHEAD>();
          tc::fence_smem_to_mma();
          mbar_arrive(smem_addr(&sh.full[(u + i) % C::RING]));
        }
      }
      cp_wait<0>();
      __syncwarp();
      u += loads;
      tiles_before += p.n;
    }
    cp_wait<0>();
  } else {
    // ===== the products: one warp, of which one thread issues ======================
    fewer_registers<64>();
    if (warp == 12) {
      constexpr uint32_t s_desc = tc::inst_desc(!FP8, false), o_desc = tc::inst_desc(!FP8, true);
      // Whatever steers the products is broadcast, so that it is uniform for
      // the compiler too.
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t q_lo = tc::desc_lo(q_smem, 16), k_lo = tc::desc_lo(ring, 16);
      const uint32_t v_lo = tc::desc_lo(ring, HALF);
      uint32_t q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
      int u = 0;
      bool ok = true;
      auto tile_in = [&](int n) { return warp_wait(sh, sh.full[n % C::RING], (n / C::RING) & 1); };
      auto scores = [&](int x, int q, int n) {  // S_x = Q_q (tile in slot n)^T
        const uint32_t slot = (uint32_t)(n % C::RING) * (OPER >> 4);
        if (tc::one_thread()) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t off = ((k >> 2) * HALF + (k & 3) * 32) >> 4;
            tc::mma_ss(tm + 128 * x, q_lo + q * (OPER >> 4) + off, k_lo + slot + off, s_desc, k > 0);
          }
          tc::commit(smem_addr(&sh.s_full[x]));
        }
        __syncwarp();
      };
      auto product = [&](int x, int n, bool add, bool last) {  // O_x += P_x (tile in slot n)
        const uint32_t slot = (uint32_t)(n % C::RING) * (OPER >> 4);
        if (tc::one_thread()) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc::mma_ts(tm + 256 + 128 * x, tm + 128 * x + 8 * k, v_lo + slot + k * (2048 >> 4), o_desc,
                       k > 0 ? 1u : (uint32_t)add);
          if (last) tc::commit(smem_addr(&sh.o_full[x]));
        }
        __syncwarp();
      };
      auto release = [&](int n) {
        if (tc::one_thread()) tc::commit(smem_addr(&sh.empty[n % C::RING]));
        __syncwarp();
      };
      for (int cur = begin, it = sh.first; ok && cur < end;) {
        const Item p = part(cur, it);
        cur += p.n;
        const int tiles = __shfl_sync(0xffffffffu, p.n, 0);
        const bool split = __shfl_sync(0xffffffffu, (int)p.split, 0) != 0;
        const int ld = min(split ? 2 : 1, tiles);
        // Places of K_j and V_j in the order of the loads.
        auto k_at = [&](int j) { return u + (j < ld ? j : ld + 2 * (j - ld) + 1); };
        auto v_at = [&](int j) { return u + (j < tiles - ld ? ld + 2 * j : tiles + j); };
        for (int q = 0; ok && q < (split ? 1 : 2); ++q) {
          ok = warp_wait(sh, sh.q_full[q], q_phase[q]);
          q_phase[q] ^= 1;
        }
        if (!split) {
          if (!ok || !(ok = tile_in(k_at(0)))) break;
          tc::fence_after();
          scores(0, 0, k_at(0));
          scores(1, 1, k_at(0));
          release(k_at(0));
          for (int j = 0; ok && j < tiles; ++j) {
            const bool more = j + 1 < tiles;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (!(ok = warp_wait(sh, sh.p_full[x], p_phase[x]))) break;
              p_phase[x] ^= 1;
              if (x == 0 && !(ok = tile_in(v_at(j)))) break;
              tc::fence_after();
              product(x, v_at(j), j > 0, !more);
              if (x == 1) release(v_at(j));
              if (more) {
                if (x == 0 && !(ok = tile_in(k_at(j + 1)))) break;
                tc::fence_after();
                scores(x, x, k_at(j + 1));
                if (x == 1) release(k_at(j + 1));
              }
            }
          }
        } else {
          for (int j = 0; ok && j < ld; ++j) {
            if (!(ok = tile_in(k_at(j)))) break;
            tc::fence_after();
            scores(j, 0, k_at(j));
            release(k_at(j));
          }
          for (int j = 0; ok && j < tiles; ++j) {
            const int x = j & 1;
            if (!(ok = warp_wait(sh, sh.p_full[x], p_phase[x]))) break;
            p_phase[x] ^= 1;
            if (!(ok = tile_in(v_at(j)))) break;
            tc::fence_after();
            product(x, v_at(j), j > 1, j + 2 >= tiles);
            release(v_at(j));
            if (j + 2 < tiles) {
              if (!(ok = tile_in(k_at(j + 2)))) break;
              tc::fence_after();
              scores(x, 0, k_at(j + 2));
              release(k_at(j + 2));
            }
          }
        }
        u += 2 * tiles;
      }
      // Every product is complete before the TMEM is given back.
      if (tc::one_thread()) tc::commit(smem_addr(&sh.drained));
      __syncwarp();
      mbar_wait(smem_addr(&sh.drained), 0, globaltimer_ns() + 1000000000ull);
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (tid == 0 && sh.fail != 0) ws_error(a.ws);
  if (warp == 12) {
    tc::fence_after();
    tc::dealloc512(tmem);
  }
}

cudaError_t launch_paged_prompt(const PagedAttnArgs& a, bool fp8, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done[2];
  const int smem = fp8 ? Cfg<true>::SMEM : Cfg<false>::SMEM;
  const cudaError_t e = fp8 ? set_smem_limit_once(paged_prompt_kernel<true>, smem, done[1])
                            : set_smem_limit_once(paged_prompt_kernel<false>, smem, done[0]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms < MAX_CTAS ? sms : MAX_CTAS, 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return fp8 ? cudaLaunchKernelEx(&cfg, paged_prompt_kernel<true>, a)
             : cudaLaunchKernelEx(&cfg, paged_prompt_kernel<false>, a);
}

}  // namespace flint
