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
//   warp 13:        looks pages up and copies K and V tiles by TMA, a box a page
//                   (16 to 128 keys): bf16 into the operand ring, E4M3 codes into
//                   a staging ring; a page that is not there is a box beyond the
//                   cache, which fills with zeros
//   warps 8-11:     widen the codes to f16 into the operand ring (E4M3), and zero
//                   the rows of V that no query of the item sees: whatever bits
//                   lie there must not meet a zero weight
//   warp 12:        issues every mma
// TMEM: S_A, S_B, O_A, O_B, 128 columns each; P takes its S's place.  O is
// rescaled only when a row's maximum grows by more than 2^8.
//
// Work: items (tile pair of a sequence, KV head) of so many key tiles, laid end
// to end and cut into equal shares, as the next-token kernel cuts its rows; cut
// items are joined through the workspace by the CTA that arrives last.
#include <type_traits>

#include "nv_util.cuh"
#include "paged.cuh"
#include "paged_work.cuh"
#include "tcgen05.cuh"
#include "tmap.h"

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
  // Warps that hand a tile over: all four widen, one looks after bf16's edges.
  static constexpr int HANDS = FP8 ? 4 : 1;
  static constexpr int SMEM = 2 * OPER + RING * OPER + STAGES * STAGE + 1024;
};

struct Shared {
  uint64_t landed[4], taken[4];      // copies: into a stage (bf16: ring slot), out of a stage
  uint64_t full[4], empty[4];        // ring slots: ready, used
  uint64_t q_full[2], s_full[2], p_half[2], p_full[2], o_full[2], drained;
  uint32_t tmem;
  int fail, last, cut[2], first, n_items;
  int scan[16];
  int pre[MAX_ITEMS + 1];            // key tiles (of all heads) before each item
  int4 item[MAX_ITEMS];              // {sequence, pair, first key tile, key tiles}
  int qpre[MAX_SEQS + 1];            // items before each sequence
  int4 seq[MAX_SEQS];                // {first row, rows, first position, -}
  alignas(16) float ks[INFO][8], lv[INFO][8], iv[INFO][8];  // a key tile's blocks (read four at a time)
  int row[16][8];                    // a key tile's blocks: cache rows
};

static_assert(Cfg<true>::SMEM + sizeof(Shared) <= 227 * 1024, "fits");
static_assert(Cfg<false>::SMEM + sizeof(Shared) <= 227 * 1024, "fits");

// The caches as (elements of a token, token rows), boxes of 128 bytes x a page's
// keys (at most a tile's).
struct Maps {
  CUtensorMap k, v;
};

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
__device__ __forceinline__ float as_f(uint32_t v) { return __uint_as_float(v); }
__device__ __forceinline__ float as_f(float v) { return v; }
template <class A, class B, class C>
__device__ __forceinline__ float max3(A a, B b, C c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(as_f(a)), "f"(as_f(b)), "f"(as_f(c)));
  return r;
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
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

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
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
    paged_prompt_kernel(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ Maps maps) {
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
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_addr(&sh.landed[i]), 1);
      mbar_init(smem_addr(&sh.taken[i]), C::HANDS);
      mbar_init(smem_addr(&sh.full[i]), C::HANDS);
      mbar_init(smem_addr(&sh.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sh.q_full[i]), 128);
      mbar_init(smem_addr(&sh.s_full[i]), 1);
      mbar_init(smem_addr(&sh.p_half[i]), 4);
      mbar_init(smem_addr(&sh.p_full[i]), 4);
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

  // Load i of an item's part: K of the first tiles (one; two where A and B have a
  // tile each), then V_j and K_(j + that many) in turn; {tile, V?}.
  auto load_of = [&](const Item& p, int i) {
    const int ld = min(p.split ? 2 : 1, p.n);
    if (i < ld) return make_int2(i, 0);
    const int k = i - ld;
    if (k < 2 * (p.n - ld)) return make_int2((k >> 1) + (k & 1 ? ld : 0), k & 1 ? 0 : 1);
    return make_int2(k - (p.n - ld), 1);
  };

  if (warp < 8)
    more_registers<192>();
  else
    fewer_registers<64>();

  if (warp < 8) {
    // ===== softmax, and the item's queries and outputs ===========================
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
        uint4 w[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) w[c] = *reinterpret_cast<const uint4*>(src + 16 * c);
        if constexpr (FP8) {
          float mx = 0.0f;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const uint32_t v[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) mx = fmaxf(mx, fmaxf(fabsf(bf_lo(v[j])), fabsf(bf_hi(v[j]))));
          }
          const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 127);
          const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
          qs *= __uint_as_float((uint32_t)(127 - 14 + e) << 23);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            w[c].x = nvu::f16x2_of(bf_lo(w[c].x) * up, bf_hi(w[c].x) * up);
            w[c].y = nvu::f16x2_of(bf_lo(w[c].y) * up, bf_hi(w[c].y) * up);
            w[c].z = nvu::f16x2_of(bf_lo(w[c].z) * up, bf_hi(w[c].z) * up);
            w[c].w = nvu::f16x2_of(bf_lo(w[c].w) * up, bf_hi(w[c].w) * up);
          }
        }
        if (!p.split || x == 0) {
          const uint32_t dst = q_smem + x * OPER + r * 128;
#pragma unroll
          for (int c = 0; c < 16; ++c)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                             dst + (c >> 3) * HALF + (((c & 7) ^ (r & 7)) << 4)),
                         "r"(w[c].x), "r"(w[c].y), "r"(w[c].z), "r"(w[c].w)
                         : "memory");
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
        // Two copies of the code, so that a tile that is seen whole pays nothing
        // for the mask.
        auto weigh = [&](auto edge) {
          constexpr bool MASK = decltype(edge)::value;
          // What the blocks' scores are multiplied by (not 0, lest a masked score
          // becomes NaN: a query of zeros, a scale of 0) and what is added.
          float kf[FP8 ? 8 : 1], lv[8];
          load8(sh.lv[slot], lv);
          if constexpr (FP8) {
            load8(sh.ks[slot], kf);
#pragma unroll
            for (int i = 0; i < 8; ++i) kf[i] = fmaxf(qs * kf[i], 1.17549435e-38f);
          } else {
            kf[0] = fmaxf(qs, 1.17549435e-38f);
          }
          // The row's scores twice, 32 columns at a time with the next ones on their
          // way: for the maximum, then for the weights.  (All 128 in registers at
          // once: spills, and 8 % slower.)
          const int mlo = lo - key0, mhi = hi - key0;  // columns seen
          auto mask = [&](int c, uint32_t (&v)[32]) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * c + i < mlo || 32 * c + i > mhi) v[i] = 0xff800000u;  // -infinity
          };
          uint32_t v[2][32];
          float mx = -INFINITY;
          tc::ld32(s_tm, v[0]);
          tc::wait_ld(v[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t(&y)[32] = v[c & 1];
            tc::ld32(s_tm + 32 * ((c + 1) & 3), v[(c + 1) & 1]);
            if constexpr (MASK) mask(c, y);
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // a block of 16 keys
              float b4[5];
#pragma unroll
              for (int i = 0; i < 5; ++i)
                b4[i] = max3(y[16 * h + 3 * i], y[16 * h + 3 * i + 1], y[16 * h + 3 * i + 2]);
              const float bm = fmaxf(max3(b4[0], b4[1], b4[2]), max3(b4[3], b4[4], y[16 * h + 15]));
              mx = fmaxf(mx, fmaf(bm, kf[FP8 ? 2 * c + h : 0], lv[2 * c + h]));
            }
            tc::wait_ld(v[(c + 1) & 1]);
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
          float iv[8];
          if constexpr (FP8) load8(sh.iv[slot], iv);
          uint64_t sums[2] = {0ull, 0ull};
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // columns 32c .. are in v[c & 1]
            uint32_t(&y)[32] = v[c & 1];
            if (c < 3) tc::ld32(s_tm + 32 * (c + 1), v[(c + 1) & 1]);
            if constexpr (MASK) mask(c, y);
            uint32_t w[16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int blk = 2 * c + h;
              const float d = lv[blk] - mu;
              const uint64_t k2 = pair(kf[FP8 ? blk : 0], kf[FP8 ? blk : 0]), d2 = pair(d, d);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float y0, y1;
                unpair(fma2(pair(as_f(y[16 * h + 2 * i]), as_f(y[16 * h + 2 * i + 1])), k2, d2), y0, y1);
                y0 = ex2(y0);
                y1 = ex2(y1);
                sums[i & 1] = FP8 && i < 2 ? pair(y0, y1) : add2(sums[i & 1], pair(y0, y1));
                w[8 * h + i] = pack_p<FP8>(y0, y1);
              }
              if constexpr (FP8) {
                float y0, y1;
                unpair(add2(sums[0], sums[1]), y0, y1);
                l = fmaf(y0 + y1, iv[blk], l);
              }
            }
            tc::st16(s_tm + 16 * c, w);
            if (c == 1) {  // the second product may begin
              tc::wait_st();
              tc::fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_addr(&sh.p_half[x]));
            }
            if (c < 3) tc::wait_ld(v[(c + 1) & 1]);
          }
          tc::wait_st();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[x]));
          if constexpr (!FP8) {
            float y0, y1;
            unpair(add2(sums[0], sums[1]), y0, y1);
            l += y0 + y1;
          }
        };
        if (masked)
          weigh(std::true_type{});
        else
          weigh(std::false_type{});
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
    // ===== tiles from copies to operands =============================================
    const int w4 = warp - 8;
    int u = 0;  // tiles handed over (K and V alike)
    bool ok = warp - 8 < C::HANDS;
    for (int cur = begin, it = sh.first; ok && cur < end;) {
      const Item p = part(cur, it);
      cur += p.n;
      const int see_hi = p.pos0 + p.tokens - 1;
      const int see_lo = a.window > 0 ? max(0, p.pos0 - a.window + 1) : 0;
      for (int i = 0; i < 2 * p.n; ++i, ++u) {
        const int2 kv = load_of(p, i);
        const int key0 = (p.kt0 + kv.x) << 7;
        const uint32_t dst = ring + (u % C::RING) * OPER;
        if constexpr (FP8) {
          const int st = u % C::STAGES, slot = u % C::RING;
          if (!(ok = warp_wait(sh, sh.landed[st], (u / C::STAGES) & 1))) break;
          uint4 w[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {  // 4 keys a time, a chunk of 16 codes a lane
            const int r = 32 * w4 + 4 * j + (lane >> 3), c = lane & 7;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[j].x), "=r"(w[j].y), "=r"(w[j].z), "=r"(w[j].w)
                         : "r"(stages + st * STAGE + r * HD + ((c ^ (r & 7)) << 4)));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.taken[st]));
          if (u >= C::RING && !(ok = warp_wait(sh, sh.empty[slot], ((u / C::RING) & 1) ^ 1))) break;
          const bool edge = key0 < see_lo || key0 + TILE - 1 > see_hi;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int r = 32 * w4 + 4 * j + (lane >> 3), c = lane & 7;
            if (edge && (key0 + r < see_lo || key0 + r > see_hi)) w[j] = make_uint4(0u, 0u, 0u, 0u);
            // Operand chunks 2c and 2c + 1; the upper lanes store the odd one
            // first, so that the eight lanes of a phase fall into distinct banks.
            const bool odd = (c & 4) != 0;
            uint32_t x[8] = {e4m3x2_to_f16x2(w[j].x & 0xffffu), e4m3x2_to_f16x2(w[j].x >> 16),
                             e4m3x2_to_f16x2(w[j].y & 0xffffu), e4m3x2_to_f16x2(w[j].y >> 16),
                             e4m3x2_to_f16x2(w[j].z & 0xffffu), e4m3x2_to_f16x2(w[j].z >> 16),
                             e4m3x2_to_f16x2(w[j].w & 0xffffu), e4m3x2_to_f16x2(w[j].w >> 16)};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int ch = 2 * c + (odd ? 1 - h : h);
              uint32_t y[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) y[k] = odd ? x[4 * (1 - h) + k] : x[4 * h + k];
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                               dst + (ch >> 3) * HALF + r * 128 + (((ch & 7) ^ (r & 7)) << 4)),
                           "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                           : "memory");
            }
          }
          tc::fence_smem_to_mma();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.full[slot]));
        } else {
          const int slot = u % C::RING;
          if (!(ok = warp_wait(sh, sh.landed[slot], (u / C::RING) & 1))) break;
          if (kv.y && (key0 < see_lo || key0 + TILE - 1 > see_hi)) {
            for (int r = lane >> 4; r < TILE; r += 2)
              if (key0 + r < see_lo || key0 + r > see_hi) {
                const int c = lane & 15;
                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                 dst + (c >> 3) * HALF + r * 128 + ((c & 7) << 4)),
                             "r"(0u)
                             : "memory");
              }
            tc::fence_smem_to_mma();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(smem_addr(&sh.full[slot]));
        }
      }
    }
  } else if (warp == 13) {
    // ===== K and V tiles, copied ======================================================
    const int box_keys = min(1 << b.page_shift, TILE), boxes = TILE / box_keys;
    const int n_rows = b.n_pages << b.page_shift;
    int u = 0;             // tiles copied (K and V alike)
    int tiles_before = 0;
    bool ok = true;
    for (int cur = begin, it = sh.first; ok && cur < end;) {
      const Item p = part(cur, it);
      cur += p.n;
      // Keys some query of the item sees.
      const int see_hi = p.pos0 + p.tokens - 1;
      const int see_lo = a.window > 0 ? max(0, p.pos0 - a.window + 1) : 0;
      // Where the 16-key blocks lie: lane l holds block l % 8 of tile 4 batch +
      // l / 8; the rows two batches and the scales one batch ahead of their use.
      auto rows_of = [&](int batch) {
        const int tile = 4 * batch + (lane >> 3);
        const int key = ((p.kt0 + tile) << 7) + 16 * (lane & 7);
        const int box = key & ~(box_keys - 1);
        return tile < p.n && box <= see_hi && box + box_keys - 1 >= see_lo ? cache_row(b, p.seq, key) : -1;
      };
      int row[3] = {-1, -1, -1};
      float ks[2] = {0.0f, 0.0f}, vs[2] = {1.0f, 1.0f};
      auto scales_of = [&](int i) {
        if constexpr (FP8) {
          if (row[i] >= 0) {
            const size_t at = (size_t)(row[i] >> 4) * b.nkv + p.kvh;
            ks[i] = __ldg(a.k_scale + at);
            vs[i] = __ldg(a.v_scale + at);
          }
        }
      };
      row[1] = rows_of(0);
      row[2] = rows_of(1);
      scales_of(1);
      for (int i = 0; i < 2 * p.n; ++i, ++u) {
        const int2 kv = load_of(p, i);
        const int tile = kv.x;
        if (kv.y == 0 && (tile & 3) == 0) {
          row[0] = row[1];
          ks[0] = ks[1];
          vs[0] = vs[1];
          row[1] = row[2];
          scales_of(1);
          row[2] = rows_of((tile >> 2) + 2);
        }
        constexpr int SLOTS = FP8 ? C::STAGES : C::RING;
        const int slot = u % SLOTS;
        if (u >= SLOTS && !(ok = warp_wait(sh, FP8 ? sh.taken[slot] : sh.empty[slot],
                                           ((u / SLOTS) & 1) ^ 1)))
          break;
        const uint32_t bar = smem_addr(&sh.landed[slot]);
        const uint32_t dst = FP8 ? stages + slot * STAGE : ring + slot * OPER;
        const int blk = 8 * (tile & 3) + (lane & 7);  // the lane with this lane's block
        int at = __shfl_sync(0xffffffffu, row[0], blk);
        if (kv.y == 0) {
          if (lane < 8) sh.row[(tiles_before + tile) & 15][lane] = at;
        } else {
          at = sh.row[(tiles_before + tile) & 15][lane & 7];
        }
        // Box i of the tile starts at its block i * box_keys / 16.
        const int box = FP8 ? lane : lane >> 1, half = FP8 ? 0 : lane & 1;
        int y = __shfl_sync(0xffffffffu, at, (box * (box_keys >> 4)) & 7);
        if (y < 0) y = n_rows;
        if (box < boxes)
          tma_box(dst + half * HALF + box * box_keys * 128, kv.y ? &maps.v : &maps.k,
                  p.kvh * HD + 64 * half, y, bar);
        if (kv.y == 0) {  // the tile's block table
          const float k = FP8 ? __shfl_sync(0xffffffffu, ks[0], blk) : 1.0f;
          // A scale of zero would take a block's weights out of the sum: 2^-100.
          const float v = FP8 ? fmaxf(__shfl_sync(0xffffffffu, vs[0], blk), 7.8886090522101181e-31f) : 1.0f;
          if (lane < 8) {
            const int info = (tiles_before + tile) & (INFO - 1);
            const int key = ((p.kt0 + tile) << 7) + 16 * lane;
            // A block that nothing sees may have any scale.
            const bool live = at >= 0 && key <= see_hi && key + BLOCK - 1 >= see_lo;
            sh.ks[info][lane] = live ? k : 0.0f;
            sh.lv[info][lane] = live ? (FP8 ? log2f(v) : 0.0f) : -INFINITY;
            sh.iv[info][lane] = live && FP8 ? 1.0f / v : 1.0f;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_expect_tx(bar, FP8 ? STAGE : OPER);
      }
      tiles_before += p.n;
    }
    if (!ok) {  // nothing may land after the CTA has left
      constexpr int SLOTS = FP8 ? C::STAGES : C::RING;
      const uint64_t deadline = globaltimer_ns() + 1000000000ull;
      for (int n = max(0, u - SLOTS); n < u; ++n)
        mbar_wait(smem_addr(&sh.landed[n % SLOTS]), (n / SLOTS) & 1, deadline);
    }
  } else {
    // ===== the products: one warp, of which one thread issues ======================
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
      // O_x += P_x (tile in slot n), the weights of keys 0-63 and 64-127 as they come.
      auto product = [&](int x, int n, bool add, bool last) {
        const uint32_t slot = (uint32_t)(n % C::RING) * (OPER >> 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!(ok = warp_wait(sh, h ? sh.p_full[x] : sh.p_half[x], p_phase[x]))) return false;
          tc::fence_after();
          if (tc::one_thread()) {
#pragma unroll
            for (int k = 4 * h; k < 4 * h + 4; ++k)
              tc::mma_ts(tm + 256 + 128 * x, tm + 128 * x + 8 * k, v_lo + slot + k * (2048 >> 4), o_desc,
                         k > 0 ? 1u : (uint32_t)add);
            if (h && last) tc::commit(smem_addr(&sh.o_full[x]));
          }
          __syncwarp();
        }
        p_phase[x] ^= 1;
        return true;
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
              if (x == 0 && !(ok = tile_in(v_at(j)))) break;
              if (!product(x, v_at(j), j > 0, !more)) break;
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
            if (!(ok = tile_in(v_at(j)))) break;
            if (!product(x, v_at(j), j > 1, j + 2 >= tiles)) break;
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

namespace {
bool encode_cache(CUtensorMap* map, const PagedAttnArgs& a, const void* base, bool fp8) {
  const EncodeTiledFn enc = encode_tiled();
  if (enc == nullptr) return false;
  const int es = fp8 ? 1 : 2, page = 1 << a.b.page_shift;
  const cuuint64_t dims[2] = {(cuuint64_t)a.b.nkv * HD, (cuuint64_t)a.b.n_pages << a.b.page_shift};
  const cuuint64_t strides[1] = {(cuuint64_t)a.b.nkv * HD * es};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / es), (cuuint32_t)(page < TILE ? page : TILE)};
  const cuuint32_t elem[2] = {1, 1};
  return enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
             const_cast<void*>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace

cudaError_t launch_paged_prompt(const PagedAttnArgs& a, bool fp8, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done[2];
  const int smem = fp8 ? Cfg<true>::SMEM : Cfg<false>::SMEM;
  const cudaError_t e = fp8 ? set_smem_limit_once(paged_prompt_kernel<true>, smem, done[1])
                            : set_smem_limit_once(paged_prompt_kernel<false>, smem, done[0]);
  if (e != cudaSuccess) return e;
  Maps maps;
  if (!encode_cache(&maps.k, a, a.k_cache, fp8) || !encode_cache(&maps.v, a, a.v_cache, fp8))
    return cudaErrorInvalidValue;
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
  return fp8 ? cudaLaunchKernelEx(&cfg, paged_prompt_kernel<true>, a, maps)
             : cudaLaunchKernelEx(&cfg, paged_prompt_kernel<false>, a, maps);
}

}  // namespace flint
