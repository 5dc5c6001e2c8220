// paged_prompt.cu — attention of prompts and drafts (several query rows a
// sequence) over a paged KV cache, on the tensor cores' tcgen05 path.
//
// The query heads that share a KV head are rows of one matrix: a tile is
// 128 / group tokens x group heads = 128 rows of one sequence, against tiles of
// 128 keys.  Per tile, with a running maximum m and sum l a row (2^x
// throughout, the scale carrying log2 e):
//   S = Q K^T (128 x 128 x 128),  p = 2^(S ks + lv - m),  O += P V
// E4M3: a 16-key block's ks multiplies its scores, its vs enters the exponent
// as lv = log2 vs, and l gets p / vs.  K's codes are an operand as they lie in
// the cache; a query row, scaled by a power of two to a largest element in
// [224, 448], is the sum of two E4M3 rows, hi + lo, exact down to 2^-18 of that
// element (bf16 has 8 significant bits, each half 4), so S = hi K^T + lo K^T at
// E4M3's double rate costs what one product of 16-bit operands does.  V's codes
// are widened to f16 (exact) and P is f16, 11 bits down to 2^-21 of the largest
// contribution and steps of 2^-31 of it below, whatever the blocks' scales: P in
// E4M3 would lose the small weights of a long context.  bf16: Q, K and V as they are,
// P rounded to bf16, half a step 2^-8, as the output itself; l sums the weights
// before rounding.
//
// Bound: the tensor cores for prompts (4 * 128 operations a query-key pair
// against 512 or 256 bytes a key), the cache's bytes for a few drafted tokens.
// One CTA per SM takes two tiles A and B at a time: while one tile's scores are
// with its softmax warps, the other's products run.  A and B are neighbouring
// tiles of a prompt (they share the keys they load), or, where a sequence
// brings no more than one tile, every other key tile of that one.
//   warps 0-3, 4-7: softmax of A, of B; a thread has a row (TMEM lane)
//   warps 13, 15:   look pages up and copy K, V tiles by TMA, a box a page (16 to
//                   128 keys), V's codes into a staging ring; a page that is not
//                   there is a box beyond the cache, which fills with zeros
//   warps 8-11:     widen V's codes to f16, and zero the rows of V that no query
//                   of the item sees: whatever bits lie there must not meet a
//                   zero weight
//   warps 12, 14:   issue the products of A, of B
// TMEM: S_A, S_B, O_A, O_B, 128 columns each; P takes its S's place.  O is
// rescaled only when a row's maximum grows by more than 2^8 (conditional rescaling
// of an online softmax, a published method).
//
// Work: items (tile pair of a sequence, KV head) of so many key tiles, cut as the
// next-token kernel's rows; cut items are joined through the workspace by the
// CTAs that arrive last.
//
// Measured: a chunk of 2048 tokens over 8192, 32 / 4 heads, 211 us in bf16, 1.14
// PFLOP/s (of 1.92 measured for a plain product), 230 us in E4M3; four drafted
// tokens for 8 sequences of 30K E4M3 54 us (25 of bytes).  A step of two tiles takes
// 3200-3600 cycles where its products need 2056 and its softmax alone ~1750: the
// chain scores -> softmax -> product of each tile, half hidden by the other tile, and
// an item's start and end (~6 us: queries, first keys, first maximum, outputs).
// Tried, and not faster: all 128 scores of a row in registers, tokens that keep the
// two product warps in turn (2-4 %, not kept for their waits), the next item's
// queries loaded ahead (into registers: 6 % slower; into L2: no change), the halves
// of a split item joined through shared memory (slower: registers).
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
constexpr int CODES = TILE * HD;       // bytes of a tile of codes
constexpr int MAX_ITEMS = 512;         // tile pairs: tokens / (tokens a pair) + sequences
static_assert(MAX_ITEMS >= MAX_TOKENS / (2 * TILE / MAX_GROUP) + MAX_SEQS, "room for every item");
constexpr int INFO = 8;                // tiles whose block tables are kept

template <bool FP8>
struct Cfg {
  static constexpr int KB = FP8 ? CODES : OPER;  // bytes of a K tile
  static constexpr int KR = 2;                   // K tiles
  static constexpr int KS = FP8 ? 4 : 2;         // of a split item: E4M3 has two more in tile B's queries' place
  static constexpr int VR = 2;                   // V tiles as operands, and as codes
  // Warps that hand a V tile over: all four widen, one looks after bf16's edges.
  static constexpr int HANDS = FP8 ? 4 : 1;
  static constexpr int SMEM = 2 * OPER + KR * KB + VR * OPER + (FP8 ? VR * CODES : 0) + 1024;
};

struct Shared {
  uint64_t k_in[4], k_out[4];        // K tiles: copied, used
  uint64_t v_in[2], v_taken[2];      // V tiles: copied; codes read
  uint64_t v_full[2], v_out[2];      // V operands: ready, used
  uint64_t q_full[2], s_full[2], p_half[2], p_full[2], o_full[2], b_free, drained, never;
  uint32_t tmem;
  int fail, last, cut[2], first;
  int scan[16];
  int pre[MAX_ITEMS + 1];            // weight (of all heads) before each item
  int4 item[MAX_ITEMS];              // {sequence, pair, first key tile, key tiles}
  int qpre[MAX_SEQS + 1];            // items before each sequence
  int4 seq[MAX_SEQS];                // {first row, rows, first position, -}
  alignas(16) float ks[INFO][8], lv[INFO][8], iv[INFO][8];  // a key tile's blocks (read four at a time)
  int plain[INFO];                   // all of them are there
  float qs[2][TILE];                 // E4M3: what the query rows were divided by
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
  int seq, kvh, kt0, n;  // first key tile of this part, key tiles
  int tokens, pos0;      // tokens of the item, position of the first
  int q_row;             // its row of q / out
  int row0, all;         // where the whole item begins, its key tiles
  int next;              // where the share goes on
  bool split;            // one tile: A and B have every other key tile
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
// The same, and pair(), of registers that a TMEM load filled: volatile, so that
// they stay behind the wait for it.
template <class A, class B, class C>
__device__ __forceinline__ float max3_tm(A a, B b, C c) {
  float r;
  asm volatile("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(as_f(a)), "f"(as_f(b)), "f"(as_f(c)));
  return r;
}
__device__ __forceinline__ uint64_t pair_tm(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm volatile("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
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

// How often a ring's slots have been used, as parities, over items whose number
// of slots may differ: tile j of an item uses slot j % slots.  Every warp counts
// every slot, its own use or not.
struct Turns {
  uint32_t parity = 0, used = 0;  // a bit a slot
  // Parity of the phase in which tile j of the current item is in its slot.
  __device__ __forceinline__ uint32_t of(int slot, int j, int shift) const {
    return ((parity >> slot) ^ (uint32_t)(j >> shift)) & 1u;
  }
  __device__ __forceinline__ bool fresh(int slot, int j, int shift) const {
    return (j >> shift) == 0 && ((used >> slot) & 1u) == 0;
  }
  __device__ __forceinline__ void item(int n, int shift) {  // n tiles in 1 << shift slots
    for (int s = 0; s < (1 << shift); ++s) {
      const int uses = (n - s + (1 << shift) - 1) >> shift;
      parity ^= (uint32_t)(uses & 1) << s;
      used |= (uint32_t)(uses > 0) << s;
    }
  }
};

// Where 16-byte chunk c of a 256-byte row lies in an operand tile.
__device__ __forceinline__ uint32_t row_chunk(int r, int c) {
  return (c >> 3) * HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4);
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

// DRAFTS: no sequence brings more than a tile, so that every item is split.
template <bool FP8, bool DRAFTS>
__global__ void __launch_bounds__(THREADS, 1)
    paged_prompt_kernel(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ Maps maps) {
  using C = Cfg<FP8>;
  using Cuts = PrCut<DRAFTS>;
  constexpr float LIFT = weight_lift<FP8>;
  extern __shared__ uint8_t s_raw[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedView& b = a.b;
  const int nq = b.nkv * b.group;
  const int gshift = 31 - __clz(b.group);       // group is a power of two
  const int tile_toks = TILE >> gshift;         // tokens of a tile
  const uint32_t base = (smem_addr(s_raw) + 1023u) & ~1023u;
  const uint32_t q_smem = base, k_smem = base + 2 * OPER, v_smem = k_smem + C::KR * C::KB;
  const uint32_t v_codes = v_smem + C::VR * OPER;

  if (tid == 0) {
    for (int i = 0; i < C::KS; ++i) {
      mbar_init(smem_addr(&sh.k_in[i]), 1);
      mbar_init(smem_addr(&sh.k_out[i]), 2);
    }
    for (int i = 0; i < C::VR; ++i) {
      mbar_init(smem_addr(&sh.v_in[i]), 1);
      mbar_init(smem_addr(&sh.v_taken[i]), C::HANDS);
      mbar_init(smem_addr(&sh.v_full[i]), C::HANDS);
      mbar_init(smem_addr(&sh.v_out[i]), 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sh.q_full[i]), 128);
      mbar_init(smem_addr(&sh.s_full[i]), 1);
      mbar_init(smem_addr(&sh.p_half[i]), 4);
      mbar_init(smem_addr(&sh.p_full[i]), 4);
      mbar_init(smem_addr(&sh.o_full[i]), 1);
      sh.cut[i] = -1;
    }
    mbar_init(smem_addr(&sh.b_free), 4);
    mbar_init(smem_addr(&sh.drained), 2);
    mbar_init(smem_addr(&sh.never), 1);
    sh.fail = 0;
    fence_mbar_init();
  }
  // (No other kernel that uses TMEM finds room beside this one's shared memory, so
  // none that this launch waits for is held up by the allocation.)
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
    cnt = Cuts::weight(info.w) * b.nkv;
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
  const Cuts cuts(total, gridDim.x);
  if (tid < n_items) {
    sh.pre[tid + 1] = pre + cnt;
    if (tid == 0) sh.pre[0] = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long x = (long long)cuts.share * (blockIdx.x + k);
      if (pre <= x && x < pre + cnt) {  // this item holds the cut
        sh.cut[k] = cuts.at((int)x, pre, info.w);
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
    const int weight = Cuts::weight(e.w);
    p.row0 = sh.pre[it];
    p.kvh = 0;
    while (cur >= p.row0 + weight) {
      p.row0 += weight;
      ++p.kvh;
    }
    int from, to;
    cuts.part(cur, end, p.row0, e.w, from, to);
    p.next = min(end, p.row0 + weight);
    p.seq = e.x;
    p.kt0 = e.z + from;
    p.n = to - from;
    p.all = e.w;
    const int tok0 = e.y * 2 * tile_toks;
    p.tokens = min(sq.y - tok0, 2 * tile_toks);
    p.pos0 = sq.z + tok0;
    p.q_row = sq.x + tok0;
    p.split = DRAFTS || p.tokens <= tile_toks;
    return p;
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
    int tiles_before = 0;                  // key tiles this CTA has been through
    // After a wait that ran out the items are only walked through: the other
    // tile's warps count on this one's arrivals at the joint barriers.
    bool ok = true;
    for (int cur = begin, it = sh.first; cur < end;) {
      const Item p = part(cur, it);
      cur = p.next;
      const int tok = tok_in_tile + (p.split ? 0 : x * tile_toks);
      const int pos = p.pos0 + min(tok, p.tokens - 1);
      const int head = p.kvh * b.group + head_in_group;

      // -- queries into the A operand's layout: the warp's 32 rows, two at a time
      if (!p.split || x == 0) {
        const uint32_t dst = q_smem + x * OPER;
        const int c = lane & 15;  // 16-byte chunk of the row
#pragma unroll 1
        for (int i0 = 0; i0 < 16; i0 += 8) {
          uint4 w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = 32 * (warp & 3) + 2 * (i0 + i) + (lane >> 4);
            const int tk = (rr >> gshift) + x * tile_toks;
            const size_t head = (size_t)(p.q_row + tk) * nq + p.kvh * b.group + (rr & (b.group - 1));
            w[i] = tk < p.tokens ? *reinterpret_cast<const uint4*>(a.q + head * HD + 8 * c)
                                 : make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = 32 * (warp & 3) + 2 * (i0 + i) + (lane >> 4);
            if constexpr (FP8) {
              float q[8] = {bf_lo(w[i].x), bf_hi(w[i].x), bf_lo(w[i].y), bf_hi(w[i].y),
                            bf_lo(w[i].z), bf_hi(w[i].z), bf_lo(w[i].w), bf_hi(w[i].w)};
              float mx = 0.0f;
#pragma unroll
              for (int j = 0; j < 8; j += 2) mx = max3(mx, fabsf(q[j]), fabsf(q[j + 1]));
#pragma unroll
              for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              // The power of two that brings it to (224, 448] = (0.875, 1.75] 2^8
              // (NaN for a row with an infinity, which E4M3 would turn into 448).
              const uint32_t bits = __float_as_uint(mx);
              const int e = min(max((int)(bits >> 23) - 127 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0), -100), 127);
              const float up = __uint_as_float(bits >= 0x7f800000u ? 0x7fffffffu : (uint32_t)(127 + 8 - e) << 23);
              if (c == 0) sh.qs[x][rr] = __uint_as_float((uint32_t)(127 - 8 + e) << 23);
              uint32_t hi[2], lo[2];
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const float q0 = q[4 * j] * up, q1 = q[4 * j + 1] * up, q2 = q[4 * j + 2] * up, q3 = q[4 * j + 3] * up;
                const uint32_t h0 = f32x2_to_e4m3x2(q0, q1), h1 = f32x2_to_e4m3x2(q2, q3);
                const float2 g0 = f16x2_to_f32(e4m3x2_to_f16x2(h0)), g1 = f16x2_to_f32(e4m3x2_to_f16x2(h1));
                hi[j] = h0 | h1 << 16;
                lo[j] = f32x2_to_e4m3x2(q0 - g0.x, q1 - g0.y) | f32x2_to_e4m3x2(q2 - g1.x, q3 - g1.y) << 16;
              }
              const uint32_t at = dst + rr * 128 + (((c >> 1) ^ (rr & 7)) << 4) + (c & 1) * 8;
              asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(hi[0]), "r"(hi[1]) : "memory");
              asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at + CODES), "r"(lo[0]), "r"(lo[1]) : "memory");
            } else {
              sts128(dst + row_chunk(rr, c), w[i].x, w[i].y, w[i].z, w[i].w);
            }
          }
        }
        tc::fence_smem_to_mma();
        mbar_arrive(smem_addr(&sh.q_full[x]));
        // B's products take them too, if B has key tiles: without any, nothing waits
        // for B's product warp to have seen this phase.  The phase before has to be
        // complete and seen as well, and may be one of B's own arrivals: behind a
        // split item its join orders them (B's last products come before B's part of
        // it), behind a pair, which may have none, A waits for B here.  The rings hold
        // A up only from an item's third key tile.  (At the item's start this barrier
        // cost E4M3 registers: 2048 over 8192 233 us instead of 230.)
        if (p.split && p.n > 1) {
          if (!DRAFTS) named_sync(1, 256);
          mbar_arrive(smem_addr(&sh.q_full[1]));
        }
      }
      if (!DRAFTS && p.split && x == 1 && p.n > 1) named_sync(1, 256);  // as above
      if (C::KS > 2 && p.split && x == 1) {  // B's queries' place is free for keys
        tc::fence_smem_to_mma();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.b_free));
      }
      float qs = a.scale_log2;

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
        if (FP8 && !any) qs *= sh.qs[p.split ? 0 : x][r];
        const int slot = (tiles_before + j) & (INFO - 1);
        const int key0 = (p.kt0 + j) << 7;
        // Two copies of the code, so that a tile that is seen whole, of pages that
        // are all there, pays nothing for the mask.
        auto weigh = [&](auto edge) {
          constexpr bool MASK = decltype(edge)::value;
          constexpr bool BLOCKS = FP8 || MASK;  // blocks differ in scale or presence
          // What a block's scores are multiplied by (not 0, lest a masked score
          // becomes NaN: a query of zeros, a scale of 0), and what is added.
          auto factor = [&](int blk) {
            return FP8 ? fmaxf(qs * sh.ks[slot][blk], 1.17549435e-38f) : fmaxf(qs, 1.17549435e-38f);
          };
          auto offset = [&](int blk) { return BLOCKS ? sh.lv[slot][blk] : 0.0f; };
          // Columns 32c .. of the row: not seen is -infinity; the highest of each block.
          auto mask = [&](int c, uint32_t (&v)[32]) {
            const int k0 = key0 + 32 * c;
            if (MASK && (k0 < lo_all || k0 + 31 > hi_all)) {
              const int mlo = lo - k0, mhi = hi - k0;
              tc::arrived(v);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (i < mlo || i > mhi) v[i] = 0xff800000u;
            }
          };
          auto highest = [&](int c, const uint32_t (&v)[32]) {
            float bm[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t* y = v + 16 * h;
              const float a0 = max3_tm(y[0], y[1], y[2]), a1 = max3_tm(y[3], y[4], y[5]);
              const float a2 = max3_tm(y[6], y[7], y[8]), a3 = max3_tm(y[9], y[10], y[11]);
              const float a4 = max3_tm(y[12], y[13], y[14]), a5 = max3_tm(a3, a4, y[15]);
              bm[h] = fmaxf(max3(a0, a1, a2), a5);
              if constexpr (BLOCKS) bm[h] = fmaf(bm[h], factor(2 * c + h), offset(2 * c + h));
            }
            return fmaxf(bm[0], bm[1]);
          };
          // The weights of 32 columns, relative to 2^m.
          uint64_t s0 = 0, s1 = 0;
          float sum = 0.0f;
          auto weights = [&](int c, const uint32_t (&v)[32], uint32_t (&w)[16]) {
            const float mu = m > -INFINITY ? m : 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int blk = 2 * c + h;
              const float k = factor(blk), d = offset(blk) - mu;
              const uint64_t k2 = pair(k, k), d2 = pair(d, d);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                float y0, y1;
                unpair(fma2(pair_tm(v[16 * h + 2 * i], v[16 * h + 2 * i + 1]), k2, d2), y0, y1);
                y0 = ex2(y0);
                y1 = ex2(y1);
                const uint64_t y = pair(y0, y1);
                const bool first = i < 2 && (FP8 || blk == 0);
                if (i & 1)
                  s1 = first ? y : add2(s1, y);
                else
                  s0 = first ? y : add2(s0, y);
                w[8 * h + i] = pack_p<FP8>(y0, y1);
              }
              if constexpr (FP8) {
                float y0, y1;
                unpair(add2(s0, s1), y0, y1);
                sum = blk == 0 ? (y0 + y1) * sh.iv[slot][0] : fmaf(y0 + y1, sh.iv[slot][blk], sum);
              }
            }
          };
          // The maximum moves only when it grows by more than 2^8 (or from
          // nothing), so the first half's exponentials start from the old one,
          // before the new one is known, and are taken again, from scores still in
          // TMEM, in the few tiles where it moves.
          uint32_t va[32], vb[32], vc[32], w0[16], w1[16];
          tc::ld32(s_tm, va);
          tc::ld32(s_tm + 32, vb);
          tc::wait_ld();
          tc::ld32(s_tm + 64, vc);
          mask(0, va);
          float mx = highest(0, va);
          weights(0, va, w0);
          tc::ld32(s_tm + 96, va);
          mask(1, vb);
          mx = fmaxf(mx, highest(1, vb));
          weights(1, vb, w1);
          tc::wait_ld();
          mask(2, vc);
          mask(3, va);
          mx = max3(mx, highest(2, vc), highest(3, va));
          if constexpr (!BLOCKS) mx *= factor(0);
          if (__any_sync(0xffffffffu, mx > m + LIFT + 8.0f)) {
            const float mn = fmaxf(m, mx - LIFT);
            const float f = m > -INFINITY ? ex2(m - mn) : 0.0f;
            l *= f;
            m = mn;
            if (any) {  // the products so far
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                tc::ld16(o_tm + 16 * c, w0);
                tc::wait_ld();
                tc::arrived(w0);
#pragma unroll
                for (int i = 0; i < 16; ++i) w0[i] = __float_as_uint(as_f(w0[i]) * f);
                tc::st16(o_tm + 16 * c, w0);
              }
            }
            tc::ld32(s_tm, vb);
            tc::wait_ld();
            mask(0, vb);
            weights(0, vb, w0);
            tc::ld32(s_tm + 32, vb);
            tc::wait_ld();
            mask(1, vb);
            weights(1, vb, w1);
          }
          any = true;
          auto hand_over = [&](uint64_t& bar) {
            tc::wait_st();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&bar));
          };
          tc::st16(s_tm, w0);
          tc::st16(s_tm + 16, w1);
          hand_over(sh.p_half[x]);  // the second product may begin
          weights(2, vc, w0);
          tc::st16(s_tm + 32, w0);
          weights(3, va, w1);
          tc::st16(s_tm + 48, w1);
          hand_over(sh.p_full[x]);
          if constexpr (!FP8) {
            float y0, y1;
            unpair(add2(s0, s1), y0, y1);
            sum = y0 + y1;
          }
          l += sum;
        };
        if (key0 + TILE - 1 > hi_all || key0 < lo_all || (!FP8 && !sh.plain[slot]))
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
      int c0, c1;  // the CTAs that share the item
      const bool whole = !cuts.shared(p.row0, p.all, c0, c1);
      // A finished row goes out by way of the query tile's place, which is free:
      // a thread writes chunks of its row there, and the warp takes its 32 rows
      // out two at a time, whole lines instead of 16 bytes of 32 rows.
      // (A split item's two halves of the columns share A's: B's may hold keys.)
      const uint32_t stage = q_smem + (p.split ? 0 : x * OPER);
      auto put = [&](int row, int c, const float* o, float f) {  // 8 columns
        sts128(stage + row_chunk(row, c), pack_bf16(o[0] * f, o[1] * f), pack_bf16(o[2] * f, o[3] * f),
               pack_bf16(o[4] * f, o[5] * f), pack_bf16(o[6] * f, o[7] * f));
      };
      auto send = [&](int row, int chunks, int first) {  // `chunks` (a power of two) of 32 rows' chunks
        __syncwarp();
        const int per = 32 / chunks, c = first + (lane & (chunks - 1));
#pragma unroll 4
        for (int i = 0; i < 32; i += per) {
          const int rr = row + i + lane / chunks;
          const int tk = (rr >> gshift) + (p.split ? 0 : x * tile_toks);
          uint4 w;
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                       : "r"(stage + row_chunk(rr, c)));
          if (tk < p.tokens)
            *reinterpret_cast<uint4*>(
                a.out + ((size_t)(p.q_row + tk) * nq + p.kvh * b.group + (rr & (b.group - 1))) * HD + 8 * c) = w;
        }
        __syncwarp();
      };
      if (whole && !p.split) {
        const float inv = row_factor(a, head, m, l);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tc::ld32(o_tm + 32 * c, v);
          tc::wait_ld();
          tc::arrived(v);
#pragma unroll
          for (int i = 0; i < 4; ++i) put(r, 4 * c + i, reinterpret_cast<const float*>(v) + 8 * i, inv);
        }
        send(r & ~31, 16, 0);
        continue;
      }
      // Partial: maxima, sums and unscaled outputs of this tile, [4 columns][row],
      // of the warps that have a row.
      if (__any_sync(0xffffffffu, tok < p.tokens)) {
        float* slot = pr_slot(a.ws, blockIdx.x, whole || (int)blockIdx.x == c0, x);
        __stcg(slot + r, m);
        __stcg(slot + TILE + r, any ? l : 0.0f);
        float4* o4 = reinterpret_cast<float4*>(slot + 2 * TILE);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[32];
          tc::ld32(o_tm + 32 * c, v);
          tc::wait_ld();
          tc::arrived(v);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            __stcg(o4 + (8 * c + i) * TILE + r,
                   any ? make_float4(as_f(v[4 * i]), as_f(v[4 * i + 1]), as_f(v[4 * i + 2]), as_f(v[4 * i + 3]))
                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f));
        }
      }
      // Join, in the order of the keys: a pair's warps have their own rows; a split
      // tile's 32-row blocks (a power of two of them) are shared by all eight warps,
      // a part of the columns each.
      const int rows = p.tokens << gshift;
      const int blocks = !p.split ? 8 : rows <= 32 ? 1 : rows <= 64 ? 2 : 4, share = 4 * blocks;
      const int row = !p.split ? r : 32 * (warp & (blocks - 1)) + lane, col = (warp / blocks) * share;  // of 32
      const int h0 = p.split ? 0 : x, row_tok = (row >> gshift) + h0 * tile_toks;
      const int row_head = p.kvh * b.group + (row & (b.group - 1));
      int halves = p.split ? 2 : 1;
      Join jn(blockIdx.x, whole ? (int)blockIdx.x : c0, whole ? (int)blockIdx.x : c1);
      for (;; jn.up(), halves = 1) {
        __threadfence();
        named_sync(1, 256);
        if (!whole) {
          if (tid == 0) sh.last = jn.arrive(a.ws);
          named_sync(1, 256);
          const bool last = sh.last != 0;
          named_sync(1, 256);  // sh.last is read before it is set again
          if (!last) break;
        }
        const int parts = jn.n * halves;
        auto slot_of = [&](int q) {
          const int k = halves == 2 ? q >> 1 : q, h = halves == 2 ? q & 1 : h0;
          return pr_slot(a.ws, jn.cta(k), jn.begins(k), h);
        };
        float* to = slot_of(0);
        const bool live = __any_sync(0xffffffffu, row_tok < p.tokens);
        float mm = -INFINITY, ll = 0.0f;
        if (live) {
#pragma unroll 4
          for (int q = 0; q < parts; ++q) mm = fmaxf(mm, __ldcg(slot_of(q) + row));
#pragma unroll 4
          for (int q = 0; q < parts; ++q) {
            const float* s = slot_of(q);
            const float mk = __ldcg(s + row), lk = __ldcg(s + TILE + row);
            ll = fmaf(lk, mk > -INFINITY ? ex2(mk - mm) : 0.0f, ll);
          }
          const float inv = row_factor(a, row_head, mm, ll);
#pragma unroll 1
          for (int c = col; c < col + share; c += 4) {  // 16 columns at a time
            float o[16] = {};
#pragma unroll 4
            for (int q = 0; q < parts; ++q) {
              const float* s = slot_of(q);
              const float4* o4 = reinterpret_cast<const float4*>(s + 2 * TILE) + c * TILE + row;
              const float mk = __ldcg(s + row), f = mk > -INFINITY ? ex2(mk - mm) : 0.0f;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 w = __ldcg(o4 + i * TILE);
                o[4 * i] = fmaf(w.x, f, o[4 * i]);
                o[4 * i + 1] = fmaf(w.y, f, o[4 * i + 1]);
                o[4 * i + 2] = fmaf(w.z, f, o[4 * i + 2]);
                o[4 * i + 3] = fmaf(w.w, f, o[4 * i + 3]);
              }
            }
            if (jn.top) {
              put(row, c >> 1, o, inv);
              put(row, (c >> 1) + 1, o + 8, inv);
            } else {  // in place: no other thread reads these
              float4* o4 = reinterpret_cast<float4*>(to + 2 * TILE) + c * TILE + row;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                __stcg(o4 + i * TILE, make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
            }
          }
          if (jn.top) send(row & ~31, share >> 1, col >> 1);
        }
        if (jn.top) break;
        named_sync(1, 256);  // the maxima and sums have been read
        if (live && col == 0) {
          __stcg(to + row, mm);
          __stcg(to + TILE + row, ll);
        }
      }
      // Slots that a later item of this CTA writes are read by now.
      named_sync(1, 256);
    }
  } else if (warp < 12) {
    // ===== V tiles from copies to operands ==========================================
    const int w4 = warp - 8;
    Turns turns;
    bool ok = w4 < C::HANDS;
    for (int cur = begin, it = sh.first; ok && cur < end;) {
      const Item p = part(cur, it);
      cur = p.next;
      const int see_hi = p.pos0 + p.tokens - 1;
      const int see_lo = a.window > 0 ? max(0, p.pos0 - a.window + 1) : 0;
#pragma unroll 1
      for (int j = 0; j < p.n; ++j) {
        const int s = j & 1, key0 = (p.kt0 + j) << 7;
        const uint32_t phase = turns.of(s, j, 1), dst = v_smem + s * OPER;
        const bool edge = key0 < see_lo || key0 + TILE - 1 > see_hi;
        if (!(ok = warp_wait(sh, sh.v_in[s], phase))) break;
        if constexpr (FP8) {
          uint4 w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {  // 4 keys a time, a chunk of 16 codes a lane
            const int r = 32 * w4 + 4 * i + (lane >> 3), c = lane & 7;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                         : "r"(v_codes + s * CODES + r * HD + ((c ^ (r & 7)) << 4)));
          }
          if (edge) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int key = key0 + 32 * w4 + 4 * i + (lane >> 3);
              if (key < see_lo || key > see_hi) w[i] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.v_taken[s]));
          if (!turns.fresh(s, j, 1) && !(ok = warp_wait(sh, sh.v_out[s], phase ^ 1))) break;
          // Operand chunks 2c and 2c + 1; the upper lanes store the odd one first,
          // so that the eight lanes of a phase fall into distinct banks.
          const int c = lane & 7, odd = (lane >> 2) & 1;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 32 * w4 + 4 * i + (lane >> 3);
            const uint32_t row = dst + (c >> 2) * HALF + r * 128;
            const uint32_t x0 = odd ? w[i].z : w[i].x, x1 = odd ? w[i].w : w[i].y;
            const uint32_t y0 = odd ? w[i].x : w[i].z, y1 = odd ? w[i].y : w[i].w;
            const int first = (2 * c + odd) & 7;
            sts128(row + ((first ^ (r & 7)) << 4), e4m3x2_to_f16x2(x0 & 0xffffu), e4m3x2_to_f16x2(x0 >> 16),
                   e4m3x2_to_f16x2(x1 & 0xffffu), e4m3x2_to_f16x2(x1 >> 16));
            sts128(row + ((first ^ 1 ^ (r & 7)) << 4), e4m3x2_to_f16x2(y0 & 0xffffu),
                   e4m3x2_to_f16x2(y0 >> 16), e4m3x2_to_f16x2(y1 & 0xffffu), e4m3x2_to_f16x2(y1 >> 16));
          }
          tc::fence_smem_to_mma();
          __syncwarp();
        } else if (edge) {
          for (int r = lane >> 4; r < TILE; r += 2)
            if (key0 + r < see_lo || key0 + r > see_hi)
              sts128(dst + ((lane & 15) >> 3) * HALF + r * 128 + ((lane & 7) << 4), 0u, 0u, 0u, 0u);
          tc::fence_smem_to_mma();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(smem_addr(&sh.v_full[s]));
      }
      turns.item(p.n, 1);
    }
  } else if (warp == 13 || warp == 15) {
    // ===== K tiles, V tiles, copied: a warp each ======================================
    const bool v = warp == 15;
    const int box_keys = min(1 << b.page_shift, TILE), boxes = TILE / box_keys;
    const int n_rows = b.n_pages << b.page_shift;
    static_assert(C::KR == 2 && C::VR == 2, "a shift of 1");
    uint64_t *in = v ? sh.v_in : sh.k_in, *out = !v ? sh.k_out : FP8 ? sh.v_taken : sh.v_out;
    const int bytes = FP8 ? CODES : OPER;
    const uint32_t ring = !v ? k_smem : FP8 ? v_codes : v_smem;
    const CUtensorMap* map = v ? &maps.v : &maps.k;
    int t = 0;  // tiles copied
    Turns turns;
    uint32_t flying = 0, flying_parity = 0;  // the slots' last copies
    uint32_t b_phase = 0;
    bool ok = true;
    for (int cur = begin, it = sh.first; ok && cur < end;) {
      const Item p = part(cur, it);
      cur = p.next;
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
      int row0 = -1, row1 = rows_of(0), row2 = rows_of(1);
      float ks0 = 0.0f, vs0 = 1.0f, ks1 = 0.0f, vs1 = 1.0f;
      auto scales = [&]() {
        if (FP8 && !v && row1 >= 0) {
          const size_t at = (size_t)(row1 >> 4) * b.nkv + p.kvh;
          ks1 = a.k_scale[at];
          vs1 = a.v_scale[at];
        }
      };
      scales();
      const int shift = !v && p.split && C::KS == 4 ? 2 : 1;
#pragma unroll 1
      for (int j = 0; j < p.n; ++j, ++t) {
        if ((j & 3) == 0) {
          row0 = row1;
          ks0 = ks1;
          vs0 = vs1;
          row1 = row2;
          scales();
          row2 = rows_of((j >> 2) + 2);
        }
        const int lane0 = 8 * (j & 3);  // the lanes with this tile's blocks
        // All that can be done before the slot is free: the boxes' rows (a shuffle,
        // an election and a barrier for each copy took 200 cycles apiece) and the
        // tile's block table.
        int y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[i] = __shfl_sync(0xffffffffu, row0, lane0 + ((i * (box_keys >> 4)) & 7));
          y[i] = y[i] < 0 ? n_rows : y[i];
        }
        if (!v) {
          const int blk = lane0 + (lane & 7), info = t & (INFO - 1);
          const int at = __shfl_sync(0xffffffffu, row0, blk);
          const float k = FP8 ? __shfl_sync(0xffffffffu, ks0, blk) : 1.0f;
          const float z = FP8 ? fmaxf(__shfl_sync(0xffffffffu, vs0, blk), LEAST_SCALE) : 1.0f;
          const int key = ((p.kt0 + j) << 7) + 16 * (lane & 7);
          // A block that nothing sees may have any scale.
          const bool live = at >= 0 && key <= see_hi && key + BLOCK - 1 >= see_lo;
          const bool plain = __all_sync(0xffffffffu, at >= 0);
          if (lane < 8) {
            sh.ks[info][lane] = live ? k : 0.0f;
            sh.lv[info][lane] = live ? (FP8 ? log2f(z) : 0.0f) : -INFINITY;
            sh.iv[info][lane] = live && FP8 ? 1.0f / z : 1.0f;
            if (lane == 0) sh.plain[info] = plain;
          }
          __syncwarp();
        }
        const int slot = j & ((1 << shift) - 1);
        const uint32_t phase = turns.of(slot, j, shift);
        if (shift == 2 && j == min(2, p.n - 1)) {  // tile B is through with its last item's outputs
          if (!(ok = warp_wait(sh, sh.b_free, b_phase))) break;
          b_phase ^= 1;
        }
        if (!turns.fresh(slot, j, shift) && !(ok = warp_wait(sh, out[slot], phase ^ 1))) break;
        const uint32_t bar = smem_addr(&in[slot]);
        const uint32_t dst = slot < 2 ? ring + slot * bytes : q_smem + OPER + (slot - 2) * bytes;
        if (tc::one_thread()) {
          mbar_expect_tx(bar, bytes);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i < boxes) {
              tma_box(dst + i * box_keys * 128, map, p.kvh * HD, y[i], bar);
              if constexpr (!FP8) tma_box(dst + HALF + i * box_keys * 128, map, p.kvh * HD + 64, y[i], bar);
            }
        }
        __syncwarp();
        flying |= 1u << slot;
        flying_parity = (flying_parity & ~(1u << slot)) | phase << slot;
      }
      turns.item(p.n, shift);
    }
    // Nothing may land after the CTA has left, whichever warp's wait ran out.
    const uint64_t deadline = globaltimer_ns() + 1000000000ull;
    for (int s = 0; s < C::KS; ++s)
      if ((flying >> s) & 1u) mbar_wait(smem_addr(&in[s]), (flying_parity >> s) & 1u, deadline);
  } else if (warp == 12 || warp == 14) {
    // ===== the products of tile A, of tile B: a warp each, of which one thread issues ===
    // Issue blocks while the tensor core is busy, and the tensor core idles while
    // its issuer waits on barriers (~60 cycles each, four a tile): with one warp
    // for both tiles it idled a third of the time.
    constexpr uint32_t s_desc = FP8 ? tc::inst_desc_e4m3() : tc::inst_desc(true, false);
    constexpr uint32_t o_desc = tc::inst_desc(!FP8, true);
    const int x = warp == 14;
    // Whatever steers the products is broadcast, so that it is uniform for the
    // compiler too.
    const uint32_t s_at = __shfl_sync(0xffffffffu, tmem + 128 * x, 0), o_at = s_at + 256;
    const uint32_t q_lo = tc::desc_lo(q_smem, 16), k_lo = tc::desc_lo(k_smem, 16);
    const uint32_t v_lo = tc::desc_lo(v_smem, HALF);
    uint32_t q_phase = 0, p_phase = 0;
    Turns k_turns, v_turns;
    bool ok = true;
    // The test hook, in the CTA that has the first item (its queries arrive later).
    if (x == 0 && begin == 0 && end > 0 && __ldcg(ws_stall(a.ws)) != 0) {
      if (lane == 0) *ws_stall(a.ws) = 0;
      ok = warp_wait(sh, sh.never, 0);
    }
    for (int cur = begin, it = sh.first; ok && cur < end;) {
      const Item p = part(cur, it);
      cur = p.next;
      const int tiles = __shfl_sync(0xffffffffu, p.n, 0);
      const bool split = DRAFTS || __shfl_sync(0xffffffffu, (int)p.split, 0) != 0;
      // Of a split item A has the even key tiles and B the odd ones (a ring slot
      // is then one warp's throughout the item); both share A's queries, and a
      // key tile has one user, which counts for both.
      const int step = split ? 2 : 1, first = split ? x : 0, shift = split && C::KS == 4 ? 2 : 1;
      const uint32_t qt = q_lo + (split ? 0 : x) * (OPER >> 4);
      if (first < tiles) {
        if (!(ok = warp_wait(sh, sh.q_full[x], q_phase))) break;
        q_phase ^= 1;
      }
#pragma unroll 1
      for (int j = first - step; j < tiles; j += step) {
        const int next = j + step;
        const int sv = j & 1, sk = next & ((1 << shift) - 1);
        if (j >= 0) {  // O += P V_j, the weights of keys 0-63 and 64-127 as they come
          if (!(ok = warp_wait(sh, sh.v_full[sv], v_turns.of(sv, j, 1)))) break;
          const uint32_t vt = v_lo + sv * (OPER >> 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!(ok = warp_wait(sh, h ? sh.p_full[x] : sh.p_half[x], p_phase))) break;
            tc::fence_after();
            if (tc::one_thread()) {
#pragma unroll
              for (int k = 4 * h; k < 4 * h + 4; ++k)
                tc::mma_ts(o_at, s_at + 8 * k, vt + k * (2048 >> 4), o_desc, k > 0 ? 1u : (uint32_t)(j > first));
              if (h) {
                tc::commit(smem_addr(&sh.v_out[sv]));
                if (split) tc::commit(smem_addr(&sh.v_out[sv]));
                if (next >= tiles) tc::commit(smem_addr(&sh.o_full[x]));
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          p_phase ^= 1;
        }
        if (next < tiles) {  // S = Q K_next^T
          const uint32_t kt = sk < 2 ? k_lo + sk * (C::KB >> 4) : q_lo + (OPER >> 4) + (sk - 2) * (C::KB >> 4);
          if (!(ok = warp_wait(sh, sh.k_in[sk], k_turns.of(sk, next, shift)))) break;
          tc::fence_after();
          if (tc::one_thread()) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if constexpr (FP8)  // hi, then lo: 32 elements a step
                tc::mma_ss<true>(s_at, qt + ((k >> 2) * CODES + (k & 3) * 32 >> 4), kt + ((k & 3) * 32 >> 4),
                                 s_desc, k > 0);
              else
                tc::mma_ss<false>(s_at, qt + ((k >> 2) * HALF + (k & 3) * 32 >> 4),
                                  kt + ((k >> 2) * HALF + (k & 3) * 32 >> 4), s_desc, k > 0);
            }
            tc::commit(smem_addr(&sh.s_full[x]));
            tc::commit(smem_addr(&sh.k_out[sk]));
            if (split) tc::commit(smem_addr(&sh.k_out[sk]));
          }
          __syncwarp();
        }
      }
      k_turns.item(tiles, shift);
      v_turns.item(tiles, 1);
    }
    // Every product is complete before the TMEM is given back.
    if (tc::one_thread()) tc::commit(smem_addr(&sh.drained));
    __syncwarp();
    mbar_wait(smem_addr(&sh.drained), 0, globaltimer_ns() + 1000000000ull);
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

namespace {
template <bool FP8, bool DRAFTS>
cudaError_t launch(const PagedAttnArgs& a, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done;
  const int smem = Cfg<FP8>::SMEM;
  const cudaError_t e = set_smem_limit_once(paged_prompt_kernel<FP8, DRAFTS>, smem, done);
  if (e != cudaSuccess) return e;
  Maps maps;
  if (!encode_cache(&maps.k, a, a.k_cache, FP8) || !encode_cache(&maps.v, a, a.v_cache, FP8))
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
  return cudaLaunchKernelEx(&cfg, paged_prompt_kernel<FP8, DRAFTS>, a, maps);
}
}  // namespace

cudaError_t launch_paged_prompt(const PagedAttnArgs& a, bool fp8, int sms, cudaStream_t stream) {
  if (a.b.max_q <= TILE / a.b.group)
    return fp8 ? launch<true, true>(a, sms, stream) : launch<false, true>(a, sms, stream);
  return fp8 ? launch<true, false>(a, sms, stream) : launch<false, false>(a, sms, stream);
}

}  // namespace flint
