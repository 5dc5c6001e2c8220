// linear_tiles.cu — matrix products of many rows, plain or grouped, on the tensor
// cores' tcgen05 path.
//
// D^T = W X^T: the weights' rows are the M side of the product (128 a CTA, TMEM
// lanes) and the rows of x the N side, 32 to 256 of them (TMEM columns), so that a
// group of few rows costs few columns and its weights are read once.  With CG = 2 a
// cluster of two CTAs works on one tile of 256 weight rows (cta_group::2): each loads
// its 128 weight rows and half the rows of x.  SwiGLU: a CTA's 128 weight rows are
// blocks of 16 gate and the 16 up rows of the same outputs (one 5-dimensional tensor
// copy), so that a warp of the epilogue has both in its 32 lanes.
//
// One CTA per SM, persistent:
//   warp 0      issues the products (of the pair: the first CTA's)
//   warps 1-3, 12-14  copy W and X, 64 k a stage, a stage each (or two) in turn (TMA,
//               128-byte swizzle); X as boxes of rows, or four rows an instruction where an index
//               says which
//   warps 4-11  epilogue: bias, activation and residual on fragments of 16 outputs x
//               8 rows, transposed to rows through shared memory 8 x 8 at a time
// TMEM holds two accumulators: a tile's epilogue runs beside the next one's products.
// The layer's products: gate/up leaves h as pairs of bf16 (PAIR_OUT), down takes them, hi and
// lo on the same weights of a stage, and leaves f16 with a scale for every 32 outputs, which a
// warp of the epilogue has (PAIR_IN).
//
// Groups: the tiles' costs (their rows, and COST_TILE for what a tile costs besides) are
// laid end to end and cut into equal shares, a tile belonging to the share where it
// begins.  Plain products, tiles of one cost, are dealt out in turn; few tiles have k cut
// over a cluster of CTAs (SPLIT), whose sums are joined in their order.
//
// Bound: the tensor pipe for many rows of few matrices (8192 x 2048 -> SwiGLU 4096: 142 us,
// 1.94 PFLOP/s, in short runs; 163 at the power limit; 8192 x 2048 -> 4096 74 us, with SiLU 76,
// with GELU, whose erfc the epilogue takes longer for than the products, 115), HBM for groups
// (4200 rows, 512 -> 2048, 256 groups 90 us, 6.2 TB/s; 49152 rows, 2048 -> SwiGLU 512 214-222 us,
// 5.3 TB/s: a tile of 256 weight rows takes 9.7 us and 11 ns a row, 15.2 tiles a pair), latencies
// for few tiles (33 x 4096 -> 2048 9.0 us; 128 x 2048 -> 5120 12.6).  The down product of pairs
// (57344 rows, 512 -> 1024) takes 111 us: 553 MB at 5.0 TB/s beside a tensor pipe 51 % busy,
// 13.2 K cycles a tile of 192 rows, of which its products are 6.7.
// Tried, and not faster: L2 prefetches of the next tile's weights (285 -> 436 us for the
// gathered gate/up: 78 MB ahead of use, L2 lost its x), the next rows' accumulators loaded
// ahead in the epilogue, a last share weighed by where its weights come from; tiles of groups
// dealt to the pairs from a counter instead of shares (49152 rows 211 -> 205 us, but 4200 rows
// 87 -> 92, and 2000 tokens' layer 297 -> 305: a pair's own tiles, one after another, read HBM
// faster).
#include <cuda_fp16.h>

#include "linear.cuh"
#include "tcgen05.cuh"
#include "tmap.h"

namespace flint {
namespace {

using namespace lin;

constexpr int THREADS = 480, WARPS = THREADS / 32;
constexpr int EPI0 = 4, EPI_WARPS = 8;     // warps of the epilogue, two a quarter of TMEM's lanes
constexpr int COPY_WARPS = 6;             // warps 1, 2, 3, 12, 13, 14: alone or in twos, a stage each in turn
constexpr int KS = 64;                    // k of a stage: a 128-byte row
constexpr int A_BYTES = 128 * KS * 2;
constexpr int MAX_STAGES = 12;
constexpr int STAGE_AREA = 192 * 1024;
constexpr int EPI_BYTES = 32 * 80;        // a warp's 32 rows of 32 outputs, padded
constexpr int SMEM = STAGE_AREA + EPI_WARPS * EPI_BYTES + 1024;
constexpr int NT_MAX = 256, NT_MAX_F32 = 128;
static_assert(NT_MAX_F32 == 4 * 32, "two chunks of rows a warp of the epilogue");
constexpr int SEGMENT = 8;                // fp32 outputs: stages that are summed in TMEM
constexpr int MAX_SPLITS = 8;             // parts of k: a portable cluster
constexpr int PART_BYTES = 4096;          // 32 rows x 32 weight rows of sums
// What a tile of a group costs besides its rows, in rows: its weights' copies, whether
// they come from HBM or, as those of a group's further tiles of rows, from L2.  Measured for
// k = 2048: 9.7 us and 11 ns a row.  (512, 896, 1504, 2496 rows, 49152 rows of the gate/up:
// 211, 207, 208, 210 us; at k = 512 they do not differ.)
constexpr int COST_TILE = 896;
constexpr int STRIP = 8;                  // tiles of weights that share their rows of x in L2

// What a kernel's outputs are, and x: bf16 of bf16, fp32, pairs, and scaled f16 of pairs.
enum Form { BF16, FP32, PAIR_OUT, PAIR_IN };

struct Shared {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES], acc_full[2], acc_empty[2], drained, never;
  uint32_t tmem;
  int fail;
  long long warp_tot[WARPS];
  long long pre[GROUP_LIMIT + 2];          // cost of all tiles before a group's
};
static_assert(SMEM + sizeof(Shared) <= 227 * 1024, "fits");

// Tensor maps: the weights (all groups but a last one of its own, and that one), x, and
// x for that last group, whose rows are x's in order.
struct Maps {
  CUtensorMap w, w_last, x, x_last;
};

// Divisions by a number the host knows, of values below 2^24 by divisors below 2^16: a
// kernel's start is a chain of them, ~200 cycles each (33 x 4096 -> 2048 10.0 -> 9.5 us).
struct Divisor {
  uint64_t magic;  // 2^40 / d, rounded up
  int d;
  explicit Divisor(int d_ = 1) : magic(((1ull << 40) + d_ - 1) / d_), d(d_) {}
  __device__ __forceinline__ int div(int x) const { return (int)(((uint64_t)(uint32_t)x * magic) >> 40); }
};

struct Plan {
  int nt;          // most rows of a tile, a multiple of 32 (groups: a power of two)
  int nt_shift;    // its logarithm, for groups
  int stages, stage_bytes;
  int x_bytes;     // of a stage's rows of x (a pair's lo: as many behind them)
  int n_m;         // tiles of weight rows of a group
  int k_steps;
  int box_rows;    // rows of a box of x; 0: four rows an instruction by index
  int box_shift;   // logarithm of a copy's rows, for groups
  int n_main;      // groups whose weights are in the first map
  int splits;      // CTAs that share a tile's k
  int part_bytes;  // room for their sums, behind the ring
  int team_shift;  // copying warps a stage: 2^1 where rows are gathered, 2^0
  int checked;     // rows whose index is out of range are not stored
  int tiles;       // plain: tiles; rows' tiles of a strip of STRIP of weights, a last strip's
  Divisor strip, last;
};

struct Tile {
  int g, m, r0, n, rows;  // group, tile of weight rows, first row, rows rounded up, rows
};

// `begin`: at a kernel's start, where nothing but barriers' initialisation is published,
// which has a fence of its own.
__device__ __forceinline__ void cluster_begin() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

template <int CG>
struct Ops {
  static __device__ __forceinline__ void alloc(uint32_t word) {
    if constexpr (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(word) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tc::alloc512(word);
    }
  }
  static __device__ __forceinline__ void dealloc(uint32_t t) {
    if constexpr (CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(t) : "memory");
    else
      tc::dealloc512(t);
  }
  static __device__ __forceinline__ void mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t add) {
    if constexpr (CG == 2)
      asm volatile(
          "{ .reg .pred p; .reg .b64 a, b; setp.ne.b32 p, %4, 0;\n"
          "  mov.b64 a, {%1, %5}; mov.b64 b, {%2, %5};\n"
          "  tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p; }" ::"r"(d),
          "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(add), "r"(tc::DESC_HI)
          : "memory");
    else
      tc::mma_ss<false>(d, a_lo, b_lo, idesc, add);
  }
  // One arrival on `bar` of every CTA of the tile once all earlier products are complete.
  static __device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (CG == 2)
      asm volatile(
          "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
          "h"((uint16_t)3)
          : "memory");
    else
      tc::commit(bar);
  }
  // The address of the first CTA's barrier, for the copies and arrivals of both.
  static __device__ __forceinline__ uint32_t leader(uint32_t bar) {
    if constexpr (CG == 2) {
      uint32_t r;
      asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(bar));
      return r;
    }
    return bar;
  }
  // Relaxed: neither arrival publishes a write of the thread's, and with the default
  // release each cost ~1000 cycles behind the copies (stores) the thread had under way:
  // 33 x 4096 -> 2048 54 us with it, 24 without, 8192 x 2048 -> 2 x 4096 381, 178.
  static __device__ __forceinline__ void expect(uint32_t leader_bar, uint32_t bytes) {
    if constexpr (CG == 2)
      asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(leader_bar), "r"(bytes)
                   : "memory");
    else
      asm volatile("mbarrier.arrive.expect_tx.relaxed.cta.shared::cta.b64 _, [%0], %1;" ::"r"(leader_bar), "r"(bytes)
                   : "memory");
  }
  static __device__ __forceinline__ void arrive(uint32_t leader_bar) {
    if constexpr (CG == 2)
      asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(leader_bar) : "memory");
    else
      asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(leader_bar) : "memory");
  }
  static __device__ __forceinline__ void sync_all() {
    if constexpr (CG == 2) cluster_sync();
    else __syncthreads();
  }
#define FLINT_GROUP_COPY(DIM, MODE, COORDS, ...)                                                                       \
  if constexpr (CG == 2)                                                                                               \
    asm volatile("cp.async.bulk.tensor." DIM ".shared::cluster.global." MODE                                           \
                 ".mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint [%0], [%1, " COORDS "], [%2], %3;" ::      \
                     "r"(dst), "l"(map), "r"(bar), "l"(policy), __VA_ARGS__                                            \
                 : "memory");                                                                                          \
  else                                                                                                                 \
    asm volatile("cp.async.bulk.tensor." DIM ".shared::cluster.global." MODE                                           \
                 ".mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, " COORDS "], [%2], %3;" ::"r"(dst),          \
                 "l"(map), "r"(bar), "l"(policy), __VA_ARGS__                                                          \
                 : "memory")
  static __device__ __forceinline__ void copy2(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar,
                                               uint64_t policy) {
    FLINT_GROUP_COPY("2d", "tile", "{%4, %5}", "r"(x), "r"(y));
  }
  static __device__ __forceinline__ void copy3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar,
                                               uint64_t policy) {
    FLINT_GROUP_COPY("3d", "tile", "{%4, %5, %6}", "r"(x), "r"(y), "r"(z));
  }
  static __device__ __forceinline__ void copy5(uint32_t dst, const CUtensorMap* map, int x, int block, int g,
                                               uint32_t bar, uint64_t policy) {
    FLINT_GROUP_COPY("5d", "tile", "{%4, %7, %7, %5, %6}", "r"(x), "r"(block), "r"(g), "r"(0));
  }
  static __device__ __forceinline__ void gather4(uint32_t dst, const CUtensorMap* map, int x, const int (&y)[4],
                                                 uint32_t bar, uint64_t policy) {
    FLINT_GROUP_COPY("2d", "tile::gather4", "{%4, %5, %6, %7, %8}", "r"(x), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]));
  }
#undef FLINT_GROUP_COPY
};

// 32 columns of 16 TMEM lanes: register 4 j + i of lane 4 r + c is row r + 8 (i / 2),
// column 8 j + 2 c + i % 2.
__device__ __forceinline__ void ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Four 8 x 8 blocks of 16-bit elements, transposed on the way; lane l has the address
// of row l % 8 of block l / 8.
__device__ __forceinline__ void st_blocks(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void ld_blocks(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void st_shared16(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ void st_cluster16(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void st_shared4(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Waits for a phase, a second at most, by a whole warp, which goes on converged; a
// wait that runs out (in any warp) ends every other one of the CTA too.
__device__ __forceinline__ bool warp_wait(Shared& sh, uint64_t& bar, uint32_t parity) {
  const uint32_t b = smem_addr(&bar);
  bool ok = mbar_try_wait(b, parity);
  if (!ok) {
    const uint64_t deadline = globaltimer_ns() + 1000000000ull;
    while (!(ok = mbar_try_wait(b, parity))) {
      if (*reinterpret_cast<volatile int*>(&sh.fail) != 0) break;
      if (globaltimer_ns() > deadline) {
        *reinterpret_cast<volatile int*>(&sh.fail) = 1;
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// The tiles of one CTA (pair), in order.
struct Walk {
  const LinearArgs& a;
  const Plan& p;
  const Shared& sh;
  int unit, units;              // this pair, pairs
  // plain: the tile's number; groups: where the share goes on and ends
  int t;
  long long at, end;
  int g, m, n, count, cost, size;  // group, tile in it (weights, rows), tiles of rows, a tile's cost, rows
  Rows rows;

  __device__ __forceinline__ Walk(const LinearArgs& a_, const Plan& p_, const Shared& sh_, int unit_, int units_)
      : a(a_), p(p_), sh(sh_), unit(unit_), units(units_) {
    if (a.start == nullptr) {
      t = unit;
    } else {
      const long long total = sh.pre[a.n_groups];
      at = total * unit / units;
      end = total * (unit + 1) / units;
      if (at < end) {
        enter();
        // the first tile that begins here
        const int i = (int)((at - sh.pre[g] + cost - 1) / cost);
        m = i / count;
        n = i - m * count;
        settle();
      }
    }
  }
  // The group that the place `at` (before the end of all) falls in.
  __device__ __forceinline__ void enter() {
    int lo = 0, hi = a.n_groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sh.pre[mid + 1] > at) hi = mid;
      else lo = mid + 1;
    }
    g = lo;
    m = n = 0;
    rows = group_rows(a, g);
    count = max((rows.n + p.nt - 1) >> p.nt_shift, 1);
    size = tile_rows(rows.n, count);
    cost = size + COST_TILE;
  }
  // A group's tiles of rows in turn on the same weights, which L2 then has.
  __device__ __forceinline__ void settle() {
    if (n >= count) {
      n = 0;
      ++m;
    }
    at = sh.pre[g] + (long long)(m * count + n) * cost;
    if (m >= p.n_m && at < end) enter();
  }
  // Rows of a group's tiles: of `count` tiles, alike but for the last.
  static __device__ __forceinline__ int tile_rows(int n, int count) {
    return ((count == 1 ? n : (n + count - 1) / count) + 31) & ~31;
  }
  __device__ __forceinline__ bool more() const { return a.start == nullptr ? t < p.tiles : at < end; }
  __device__ __forceinline__ Tile get() const {
    Tile o;
    if (a.start == nullptr) {
      const int strip = p.strip.div(t), in = t - strip * p.strip.d;
      const bool whole = (strip + 1) * STRIP <= p.n_m;
      const int n = whole ? in / STRIP : p.last.div(in);
      o.g = 0;
      o.m = strip * STRIP + in - n * (whole ? STRIP : p.last.d);
      o.r0 = n * p.nt;
      o.n = p.nt;
      o.rows = min(p.nt, a.n_rows - o.r0);
    } else {
      o.g = g;
      o.m = m;
      o.r0 = rows.r0 + n * size;
      // the last tile of a group may have fewer rows, or (rounding) none
      o.rows = max(min(size, rows.n - n * size), 0);
      o.n = max((o.rows + 31) & ~31, 32);
    }
    return o;
  }
  __device__ __forceinline__ void next() {
    if (a.start == nullptr) {
      t += units;
    } else {
      ++n;
      settle();
    }
  }
};

// silu of an output that is rounded to bf16 or a pair, as activate() takes it: exponential and
// quotient of the fast kind, off by ~|v| + 4 units of fp32's last place (2^-17 of the value at
// v = -87), against a rounding of 2^-9 or 2^-17.
__device__ __forceinline__ float silu_bf16(float v) {
  const float e = __expf(-fabsf(v));
  return __fdividef(v < 0.0f ? v * e : v, 1.0f + e);
}

// Where a lane's row of the epilogue's four 8 x 8 blocks lies.
template <bool SWIGLU>
__device__ __forceinline__ uint32_t block_row(uint32_t stage, int lane) {
  return SWIGLU ? stage + ((lane >> 4) * 8 + (lane & 7)) * 48 + ((lane >> 3) & 1) * 16
                : stage + (lane & 7) * 80 + (lane >> 3) * 16;
}

// Bias of a lane's rows of the fragments.
template <bool SWIGLU>
__device__ __forceinline__ void load_bias(const LinearArgs& a, int g, int f0, float (&bias)[4]) {
  const int r = (threadIdx.x & 31) >> 2;
  const float* src = a.bias + (size_t)g * a.n_out * (SWIGLU ? 2 : 1);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int f = SWIGLU ? f0 + r + 8 * (i & 1) : f0 + r + 8 * i;
    bias[i] = a.bias != nullptr && f < a.n_out ? src[f + (SWIGLU && i >= 2 ? a.n_out : 0)] : 0.0f;
  }
}

// The epilogue of 32 rows (from row0, `left` of them there) and a warp's weight rows, whose
// sums are in lo, hi once land() has returned: bias, activation, residual, rounding, and
// the outputs f0 .. in whole 16-byte parts of rows (fp32: sectors).
template <bool SWIGLU, Form FORM, class Land>
__device__ __forceinline__ void finish(const LinearArgs& a, const Plan& p, uint32_t stage, uint32_t block, int f0, int row0,
                                       int left, const float (&bias)[4], uint32_t (&lo)[16], uint32_t (&hi)[16], Land land) {
  constexpr bool F32 = FORM == FP32;
  constexpr int WF = SWIGLU ? 16 : 32;    // outputs of a warp
  constexpr int ROW = WF * 2 + 16;        // bytes of a row of the transposition
  constexpr int PARTS = WF / 8;           // 16-byte parts of a row: a lane has as many of 32 rows
  constexpr int HALVES = SWIGLU ? 1 : 2;  // 16 outputs a lane at a time: of 32 rows (SwiGLU), of 16
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  // This lane's parts of the rows, whether they are stored, and the residual there.
  bool store[PARTS];
  if constexpr (!F32) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const int u = lane + 32 * i, tok = u / PARTS, f = f0 + 8 * (u % PARTS);
      store[i] = tok < left && f < a.n_out;
      if (p.checked && store[i]) store[i] = (unsigned)a.index[row0 + tok] < (unsigned)a.n_x;
    }
    if (a.residual != nullptr) {
#pragma unroll
      for (int i = 0; i < PARTS; ++i) {
        const int u = lane + 32 * i, tok = u / PARTS, f = f0 + 8 * (u % PARTS);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (store[i])
          v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.residual) +
                                              (size_t)(row0 + tok) * a.n_out + f);
        st_shared16(stage + tok * ROW + (u % PARTS) * 16, v);
      }
      __syncwarp();
    }
  }
  land();
#pragma unroll
  for (int h = 0; h < HALVES; ++h) {
    // Outputs r, r + 8 (of 16 of the first lanes' rows; not SwiGLU: v[8 ..] those of
    // the others') of rows 8 j + 2 c, + 1.
    float v[16];
#pragma unroll
    for (int i = 0; i < 16 / HALVES; ++i) {
      const float x = __uint_as_float(lo[8 * h + i]) + bias[(i >> 1) & 1];
      const float y = __uint_as_float(hi[8 * h + i]) + bias[2 + ((i >> 1) & 1)];
      if constexpr (SWIGLU) {
        v[i] = (F32 ? activate(x, ACT_SILU) : silu_bf16(x)) * y;
      } else {
        v[i] = x;
        v[8 + i] = y;
      }
    }
    if constexpr (!SWIGLU) {
      if (a.act == ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = F32 ? activate(v[i], ACT_SILU) : silu_bf16(v[i]);
      } else if (a.act == ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = activate(v[i], ACT_GELU);
      }
    }
    if constexpr (F32) {
      // Rows of these outputs (as many bytes as FROW holds) through shared memory.
      constexpr int FROW = WF * 4 + 16, FROWS = SWIGLU ? 32 : 16;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int in = SWIGLU ? i : i & 7;
        const int tok = 8 * (in >> 2) + 2 * c + (i & 1), f = r + 8 * ((i >> 1) & 1) + (SWIGLU || i < 8 ? 0 : 16);
        st_shared4(stage + tok * FROW + f * 4, v[i]);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        constexpr int FPARTS = WF / 4;
        const int u = lane + 32 * i, tok = 16 * h + u / FPARTS, f = f0 + 4 * (u % FPARTS);
        static_assert(FROWS * FPARTS == 128, "4 parts a lane");
        if (tok < left && f < a.n_out) {
          const int row = row0 + tok;
          if (!p.checked || (unsigned)a.index[row] < (unsigned)a.n_x) {
            const size_t at = (size_t)row * a.n_out + f;
            uint4 o = ld_shared16(stage + (u / FPARTS) * FROW + (u % FPARTS) * 16);
            if (a.residual != nullptr) {
              const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.residual) + at);
              o = make_uint4(__float_as_uint(__uint_as_float(o.x) + x.x), __float_as_uint(__uint_as_float(o.y) + x.y),
                             __float_as_uint(__uint_as_float(o.z) + x.z), __float_as_uint(__uint_as_float(o.w) + x.w));
            }
            *reinterpret_cast<uint4*>(static_cast<float*>(a.out) + at) = o;
          }
        }
      }
      __syncwarp();
    } else {
      // Block q of the four that move at a time: outputs 8 q .. of rows 8 j .. (SwiGLU:
      // outputs 8 (q % 2) .. of rows 8 (2 j + q / 2) ..); the register of its first row.
      auto reg = [](int j, int q) {
        return SWIGLU ? 4 * (2 * j + (q >> 1)) + 2 * (q & 1) : 4 * j + 2 * (q & 1) + 8 * (q >> 1);
      };
      if constexpr (FORM == PAIR_OUT) {
        static_assert(SWIGLU, "v holds the warp's outputs");
#pragma unroll
        for (int lo_part = 0; lo_part < 2; ++lo_part) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t x[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float &u0 = v[reg(j, q)], &u1 = v[reg(j, q) + 1];
              x[q] = pack_bf2(u0, u1);
              u0 -= bf_lo(x[q]);
              u1 -= bf_hi(x[q]);
            }
            st_blocks(block + 16 * j * ROW, x[0], x[1], x[2], x[3]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < PARTS; ++i) {
            const int u = lane + 32 * i, tok = u / PARTS, f = f0 + 8 * (u % PARTS);
            const uint4 o = ld_shared16(stage + tok * ROW + (u % PARTS) * 16);
            if (store[i])
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) +
                                        ((size_t)(row0 + tok) * 2 + lo_part) * a.n_out + f) = o;
          }
          __syncwarp();
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t at = block + (SWIGLU ? 16 * j : 16 * h + 8 * j) * ROW;
          uint32_t x[4];
          if (a.residual != nullptr) {
            ld_blocks(at, x);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              v[reg(j, q)] += bf_lo(x[q]);
              v[reg(j, q) + 1] += bf_hi(x[q]);
            }
          }
          if constexpr (FORM == PAIR_IN) {
            // The largest of the 32 outputs of rows 2 c and 2 c + 1 of these: four a lane,
            // eight lanes.
            static_assert(WF == SCALED, "a warp's outputs have one scale");
            float big[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float size = fabsf(v[reg(j, i >> 1) + (i & 1)]);
              if (size < __int_as_float(0x7f800000)) big[i & 1] = fmaxf(big[i & 1], size);
            }
            float inv[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) big[i] = fmaxf(big[i], __shfl_xor_sync(0xffffffffu, big[i], o));
              const int e = max((int)(__float_as_uint(big[i]) >> 23) - 14, 1);
              inv[i] = __uint_as_float((uint32_t)(254 - e) << 23);
              const int tok = 16 * h + 8 * j + 2 * c + i;
              if (r == 0 && tok < left && f0 < a.n_out)
                a.scale[(size_t)(row0 + tok) * (a.n_out / SCALED) + f0 / SCALED] = (uint8_t)e;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const __half2 two = __floats2half2_rn(v[reg(j, q)] * inv[0], v[reg(j, q) + 1] * inv[1]);
              x[q] = *reinterpret_cast<const uint32_t*>(&two);
            }
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) x[q] = pack_bf2(v[reg(j, q)], v[reg(j, q) + 1]);
          }
          st_blocks(at, x[0], x[1], x[2], x[3]);
        }
      }
    }
  }
  if constexpr (FORM == BF16 || FORM == PAIR_IN) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const int u = lane + 32 * i, tok = u / PARTS, f = f0 + 8 * (u % PARTS);
      const uint4 o = ld_shared16(stage + tok * ROW + (u % PARTS) * 16);
      if (store[i])
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (size_t)(row0 + tok) * a.n_out + f) = o;
    }
    __syncwarp();
  }
}

// SPLIT: one tile a cluster of `splits` CTAs, each of which has a part of k.
template <int CG, bool SWIGLU, Form FORM, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
    linear_tiles_kernel(const __grid_constant__ LinearArgs a, const __grid_constant__ Plan p,
                        const __grid_constant__ Maps maps) {
  using O = Ops<CG>;
  constexpr bool F32 = FORM == FP32;
  constexpr int X_PARTS = FORM == PAIR_IN ? 2 : 1;
  constexpr int FE = SWIGLU ? 64 : 128;   // outputs of a CTA's tile
  constexpr int WF = FE / 4;              // of a warp
  extern __shared__ uint8_t s_raw[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = CG == 2 ? blockIdx.x & 1 : 0;
  const int splits = SPLIT ? p.splits : 1, part = SPLIT ? blockIdx.x % splits : 0;   // of k
  const int unit = blockIdx.x / (CG * splits), units = gridDim.x / (CG * splits);
  // Steps of k of a tile, the first of which is k0.
  const int k0 = SPLIT ? p.k_steps * part / splits : 0;
  const int k_steps = SPLIT ? p.k_steps * (part + 1) / splits - k0 : p.k_steps;
  const uint32_t smem = (smem_addr(s_raw) + 1023u) & ~1023u;
  const uint32_t parts = smem + STAGE_AREA - p.part_bytes;   // SPLIT: other CTAs write here

  if (tid == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(smem_addr(&sh.full[i]), CG << p.team_shift);
      mbar_init(smem_addr(&sh.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&sh.acc_full[i]), 1);
      mbar_init(smem_addr(&sh.acc_empty[i]), EPI_WARPS * CG);
    }
    mbar_init(smem_addr(&sh.drained), 1);
    mbar_init(smem_addr(&sh.never), 1);
    sh.fail = 0;
    fence_mbar_init();
  }
  if (warp == 3) O::alloc(smem_addr(&sh.tmem));
  pdl_wait();
  pdl_trigger();

  if (a.start != nullptr) {
    // Costs before each group: a thread sums a few neighbouring groups, then a scan.
    const int per = (a.n_groups + THREADS - 1) / THREADS, g0 = min(tid * per, a.n_groups), g1 = min(g0 + per, a.n_groups);
    long long sum = 0;
    for (int g = g0; g < g1; ++g) {
      const int n = group_rows(a, g).n;
      sh.pre[g] = sum;
      const int count = (n + p.nt - 1) >> p.nt_shift;
      if (n > 0) sum += (long long)count * p.n_m * (Walk::tile_rows(n, count) + COST_TILE);
    }
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sh.warp_tot[warp] = incl;
    __syncthreads();
    long long base = incl - sum, all = 0;
    for (int i = 0; i < WARPS; ++i) {
      if (i < warp) base += sh.warp_tot[i];
      all += sh.warp_tot[i];
    }
    for (int g = g0; g < g1; ++g) sh.pre[g] += base;
    if (tid == 0) sh.pre[a.n_groups] = all;
  }
  tc::fence_before();
  __syncthreads();
  if constexpr (CG == 2) {
    cluster_begin();
    cluster_wait();
  }
  // (Nobody writes to a CTA of the cluster that has not begun.)
  if constexpr (SPLIT) cluster_begin();
  tc::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sh.tmem);

  const int copier = warp >= EPI0 + EPI_WARPS ? warp - EPI0 - EPI_WARPS + 3 : warp - 1;
  // No more teams than stages: a warp waits for a slot's last use but one to be over,
  // and parities tell it from the one before only if the warp's own last stage is within
  // a round of the ring.
  const int teams = min(COPY_WARPS >> p.team_shift, p.stages), team = copier >> p.team_shift;
  const int mate = copier - (team << p.team_shift);
  if (warp > 0 && (warp < EPI0 || warp >= EPI0 + EPI_WARPS) && team < teams) {
    // ===== copies: a team every teams-th stage =====================================
    int s = team, turn = team, step = 0;   // stage, step and the tile's first step, of all tiles
    uint32_t phase = 1;
    bool ok = true;
    // x, which every tile of weights reads, stays in L2; weights that no other tile reads
    // leave it (49152 rows of gate/up 294 -> 277 us for this, 229 -> 224 for that).
    uint64_t keep, normal;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
    for (Walk walk(a, p, sh, unit, units); ok && walk.more(); walk.next(), step += k_steps) {
      if (turn >= step + k_steps) continue;
      const Tile t = walk.get();
      const bool main = t.g < p.n_main;
      const CUtensorMap* wm = main ? &maps.w : &maps.w_last;
      const int wg = main ? t.g : 0;
      const int f = (t.m * CG + rank) * FE;
      const int rows_b = t.n / CG, row0 = t.r0 + rank * rows_b;
      // The last group of its own has the rows of x in order: boxes, also where the others
      // gather (four rows an instruction take ~22 cycles, 704 a stage of 256 rows).
      static_assert(32 / CG == 1 << (6 - CG), "32 rows, or 16 each");
      const int box_rows = main ? p.box_rows : 32 / CG;
      const CUtensorMap* xm = main ? &maps.x : &maps.x_last;
      const uint32_t bytes = (box_rows > 0 ? box_rows : 4) * KS * 2;   // of a copy of X
      const int all = a.start == nullptr ? 1 : rows_b >> (main ? p.box_shift : 6 - CG);
      const int copies = (all - mate + (1 << p.team_shift) - 1) >> p.team_shift;
      const int box = (lane << p.team_shift) + mate;   // of this lane
      const uint64_t policy = a.start != nullptr && walk.rows.n <= p.nt ? l2_evict_first() : normal;
      int y[4] = {};
      if (box_rows > 0) {
        y[0] = row0 + box * box_rows - (main || a.index == nullptr ? 0 : walk.rows.r0);
      } else if (lane < copies) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // A row of no index is not stored: any row will do.
          const int r = row0 + 4 * box + j;
          if (r < a.n_rows) y[j] = a.index[r];
          if ((unsigned)y[j] >= (unsigned)a.n_x) y[j] = 0;
        }
      }
      for (; turn < step + k_steps; turn += teams) {
        if (!(ok = warp_wait(sh, sh.empty[s], phase))) break;
        const uint32_t bar = O::leader(smem_addr(&sh.full[s])), dst = smem + s * p.stage_bytes;
        const int k = (k0 + turn - step) * KS;
        if (tc::one_thread()) {
          O::expect(bar, (mate == 0 ? A_BYTES : 0) + X_PARTS * copies * bytes);
          if (mate == 0) {
            if constexpr (SWIGLU) O::copy5(dst, wm, k, f / 16, wg, bar, policy);
            else O::copy3(dst, wm, k, f, wg, bar, policy);
          }
        }
        __syncwarp();
        if (lane < copies) {
          if (box_rows > 0) O::copy2(dst + A_BYTES + box * bytes, xm, k, y[0], bar, keep);
          else O::gather4(dst + A_BYTES + box * bytes, xm, k, y, bar, keep);
          if constexpr (FORM == PAIR_IN)
            O::copy2(dst + A_BYTES + p.x_bytes + box * bytes, xm, a.n_in + k, y[0], bar, keep);
        }
        __syncwarp();
        if ((s += teams) >= p.stages) {
          s -= p.stages;
          phase ^= 1;
        }
      }
    }
    // A wait ran out: what was asked for lands long before this.
    if (*reinterpret_cast<volatile int*>(&sh.fail) != 0)
      for (const uint64_t until = globaltimer_ns() + 50000000ull; globaltimer_ns() < until;) {}
  } else if (warp == 0 && rank == 0) {
    // ===== products ================================================================
    const uint32_t d0 = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t x16 = p.x_bytes >> 4;   // of a matrix descriptor's address
    int s = 0, it = 0;
    uint32_t phase = 0;
    bool ok = true;
    if (unit == 0 && __ldcg(reinterpret_cast<const int*>(static_cast<const char*>(a.ws) + WS_STALL)) != 0) {
      if (lane == 0) *reinterpret_cast<int*>(static_cast<char*>(a.ws) + WS_STALL) = 0;   // the test hook
      ok = warp_wait(sh, sh.never, 0);
    }
    for (Walk walk(a, p, sh, unit, units); ok && walk.more(); walk.next()) {
      const int n = __shfl_sync(0xffffffffu, walk.get().n, 0);
      const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)(n >> 3) << 17 | (uint32_t)(128 * CG >> 4) << 24;
      int b = 0;
      uint32_t d = 0;
      // Two stages at a time: a wait (~150 cycles) and a stage's issue (~200) run one behind
      // the other, and a stage of 192 rows executes in 384.
      for (int k = 0; k < k_steps; k += 2) {
        const bool two = k + 1 < k_steps;
        const bool first = F32 ? k % SEGMENT == 0 : k == 0;
        const bool last = k + 2 >= k_steps || (F32 && (k + 2) % SEGMENT == 0);
        if (first) {
          b = it & 1;
          d = d0 + b * NT_MAX;
          if (!(ok = warp_wait(sh, sh.acc_empty[b], ((it >> 1) & 1) ^ 1))) break;
          tc::fence_after();
          ++it;
        }
        int s1 = s + 1;
        uint32_t phase1 = phase;
        if (s1 == p.stages) {
          s1 = 0;
          phase1 ^= 1;
        }
        if (!(ok = warp_wait(sh, sh.full[s], phase))) break;
        if (two && !(ok = warp_wait(sh, sh.full[s1], phase1))) break;
        tc::fence_after();
        const uint32_t at = smem + s * p.stage_bytes, at1 = smem + s1 * p.stage_bytes;
        const uint32_t a_lo = tc::desc_lo(at, 16), b_lo = tc::desc_lo(at + A_BYTES, 16);
        const uint32_t a1_lo = tc::desc_lo(at1, 16), b1_lo = tc::desc_lo(at1 + A_BYTES, 16);
        if (tc::one_thread()) {
#pragma unroll
          for (int j = 0; j < KS / 16; ++j) O::mma(d, a_lo + 2 * j, b_lo + 2 * j, idesc, !first || j > 0);
          if constexpr (FORM == PAIR_IN)
#pragma unroll
            for (int j = 0; j < KS / 16; ++j) O::mma(d, a_lo + 2 * j, b_lo + x16 + 2 * j, idesc, 1);
          O::commit(smem_addr(&sh.empty[s]));
          if (two) {
#pragma unroll
            for (int j = 0; j < KS / 16; ++j) O::mma(d, a1_lo + 2 * j, b1_lo + 2 * j, idesc, 1);
            if constexpr (FORM == PAIR_IN)
#pragma unroll
              for (int j = 0; j < KS / 16; ++j) O::mma(d, a1_lo + 2 * j, b1_lo + x16 + 2 * j, idesc, 1);
            O::commit(smem_addr(&sh.empty[s1]));
          }
          if (last) O::commit(smem_addr(&sh.acc_full[b]));
        }
        __syncwarp();
        s = s1;
        phase = phase1;
        if (two && ++s == p.stages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    // Every product is complete before the TMEM is given back (and has arrived in both CTAs
    // before they leave).
    if (tc::one_thread()) O::commit(smem_addr(&sh.drained));
    __syncwarp();
    mbar_wait(smem_addr(&sh.drained), 0, globaltimer_ns() + 1000000000ull);
  } else if (warp >= EPI0 && warp < EPI0 + EPI_WARPS) {
    // ===== epilogue ================================================================
    const int w = warp & 3, half = (warp - EPI0) >> 2;
    const uint32_t stage = smem + STAGE_AREA + (warp - EPI0) * EPI_BYTES;
    const uint32_t t0 = tmem + ((uint32_t)(32 * w) << 16);
    const uint32_t block = block_row<SWIGLU>(stage, lane);
    if constexpr (SPLIT) cluster_wait();
    bool ok = true;
    int it = 0;
    for (Walk walk(a, p, sh, unit, units); ok && walk.more(); walk.next()) {
      const Tile t = walk.get();
      const int f0 = (t.m * CG + rank) * FE + WF * w;
      float bias[4];
      if constexpr (!SPLIT) load_bias<SWIGLU>(a, t.g, f0, bias);
      const int chunks = t.n / 32;
      // This CTA's part of the sums of 32 rows, to the CTA that finishes these 32 x 32.
      const auto push = [&](int ch, const uint32_t (&lo)[16], const uint32_t (&hi)[16]) {
        const int u = 4 * ch + w;
        uint32_t at;
        asm("mapa.shared::cluster.u32 %0, %1, %2;"
            : "=r"(at)
            : "r"(parts + (u / splits * splits + part) * PART_BYTES + lane * 16), "r"(u % splits));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          st_cluster16(at + i * 512, lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
          st_cluster16(at + 2048 + i * 512, hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
        }
      };
      if constexpr (F32) {
        // fp32 outputs: the tensor core cuts what it adds to its sums, a bias of up to half
        // a unit a step (rel. error 1e-6 at k = 2048, growing with k); so TMEM sums no more
        // than SEGMENT stages, and registers, which round, the segments.
        uint32_t lo[2][16] = {}, hi[2][16] = {};
        for (int k = 0; k < k_steps; k += SEGMENT, ++it) {
          const int b = it & 1;
          if (!(ok = warp_wait(sh, sh.acc_full[b], (it >> 1) & 1))) break;
          tc::fence_after();
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (half + 2 * i < chunks) {
              uint32_t x[16], y[16];
              ld_frag(t0 + b * NT_MAX + 32 * (half + 2 * i), x);
              ld_frag(t0 + b * NT_MAX + 32 * (half + 2 * i) + (16u << 16), y);
              tc::wait_ld();
              tc::arrived(x);
              tc::arrived(y);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                lo[i][j] = __float_as_uint(__uint_as_float(lo[i][j]) + __uint_as_float(x[j]));
                hi[i][j] = __float_as_uint(__uint_as_float(hi[i][j]) + __uint_as_float(y[j]));
              }
            }
          tc::fence_before();
          __syncwarp();
          if (lane == 0) O::arrive(O::leader(smem_addr(&sh.acc_empty[b])));
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int ch = half + 2 * i;
          if (ch < chunks) {
            if constexpr (SPLIT) push(ch, lo[i], hi[i]);
            else finish<SWIGLU, FORM>(a, p, stage, block, f0, t.r0 + 32 * ch, t.rows - 32 * ch, bias, lo[i], hi[i], [] {});
          }
        }
      } else {
        const int b = it & 1;
        if (!(ok = warp_wait(sh, sh.acc_full[b], (it >> 1) & 1))) break;
        ++it;
        tc::fence_after();
        if (half >= chunks && lane == 0) O::arrive(O::leader(smem_addr(&sh.acc_empty[b])));
        // Two warps have the same lanes; each takes every other 32 rows.
        for (int ch = half; ch < chunks; ch += 2) {
          uint32_t lo[16], hi[16];
          ld_frag(t0 + b * NT_MAX + 32 * ch, lo);
          ld_frag(t0 + b * NT_MAX + 32 * ch + (16u << 16), hi);
          const auto land = [&] {
            tc::wait_ld();
            tc::arrived(lo);
            tc::arrived(hi);
            if (ch + 2 >= chunks) {
              tc::fence_before();
              __syncwarp();
              if (lane == 0) O::arrive(O::leader(smem_addr(&sh.acc_empty[b])));
            }
          };
          if constexpr (SPLIT) {
            land();
            push(ch, lo, hi);
          } else {
            finish<SWIGLU, FORM>(a, p, stage, block, f0, t.r0 + 32 * ch, t.rows - 32 * ch, bias, lo, hi, land);
          }
        }
      }
    }
  }
  if constexpr (SPLIT) {
    // ===== the parts of all CTAs of the cluster, joined in their order: 32 rows x 32
    // weight rows a warp, dealt out over the CTAs.  (Each wrote them to where they are
    // read, which took 3 us less at 8 parts than to read them from one another.) ======
    const int e = warp - EPI0;
    __syncwarp();
    if (e < 0 || e >= EPI_WARPS) cluster_wait();
    cluster_sync();
    Walk walk(a, p, sh, unit, units);
    if (e >= 0 && e < EPI_WARPS && walk.more() && *reinterpret_cast<volatile int*>(&sh.fail) == 0) {
      const Tile t = walk.get();
      const uint32_t stage = smem + STAGE_AREA + e * EPI_BYTES;
      const uint32_t block = block_row<SWIGLU>(stage, lane);
      for (int u = part + splits * e; u < t.n / 8; u += splits * EPI_WARPS) {
        const int w = u & 3, ch = u >> 2, f0 = t.m * FE + WF * w;
        if (32 * ch >= t.rows) continue;
        float bias[4];
        load_bias<SWIGLU>(a, t.g, f0, bias);
        float sum[32] = {};
#pragma unroll 2
        for (int q = 0; q < splits; ++q) {
          const uint32_t at = parts + (u / splits * splits + q) * PART_BYTES + lane * 16;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 x = ld_shared16(at + i * 512);
            sum[4 * i] += __uint_as_float(x.x);
            sum[4 * i + 1] += __uint_as_float(x.y);
            sum[4 * i + 2] += __uint_as_float(x.z);
            sum[4 * i + 3] += __uint_as_float(x.w);
          }
        }
        uint32_t lo[16], hi[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          lo[i] = __float_as_uint(sum[i]);
          hi[i] = __float_as_uint(sum[16 + i]);
        }
        finish<SWIGLU, FORM>(a, p, stage, block, f0, t.r0 + 32 * ch, t.rows - 32 * ch, bias, lo, hi, [] {});
      }
    }
  }
  __syncwarp();
  tc::fence_before();
  O::sync_all();
  // The second CTA's share of the last arrival, which nothing else waits for.
  if (CG == 2 && rank == 1 && warp == 0) mbar_wait(smem_addr(&sh.drained), 0, globaltimer_ns() + 1000000000ull);
  __syncthreads();
  if (tid == 0 && sh.fail != 0) atomicCAS(reinterpret_cast<uint32_t*>(static_cast<char*>(a.ws) + WS_ERROR), DEV_OK, DEV_TIMEOUT);
  if (warp == 3) {
    tc::fence_after();
    O::dealloc(tmem);
  }
}

bool encode(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  const EncodeTiledFn enc = encode_tiled();
  const cuuint32_t elem[5] = {1, 1, 1, 1, 1};
  return enc != nullptr &&
         enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, elem,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_w(CUtensorMap* map, const LinearArgs& a, const void* base, int groups) {
  const cuuint64_t k = a.n_in, n = a.n_out, row = k * 2, all = a.w_rows > 0 ? a.w_rows : n;
  if (a.act == ACT_SWIGLU) {
    const cuuint64_t dims[5] = {k, 16, 2, n / 16, (cuuint64_t)groups};
    const cuuint64_t strides[4] = {row, n * row, 16 * row, 2 * n * row};
    const cuuint32_t box[5] = {KS, 16, 2, 4, 1};
    return encode(map, base, 5, dims, strides, box);
  }
  const cuuint64_t dims[3] = {k, n, (cuuint64_t)groups};
  const cuuint64_t strides[2] = {row, all * row};
  const cuuint32_t box[3] = {KS, 128, 1};
  return encode(map, base, 3, dims, strides, box);
}

bool encode_x(CUtensorMap* map, const LinearArgs& a, int rows) {
  const cuuint64_t k = (cuuint64_t)a.n_in * (a.pair_in ? 2 : 1);
  const cuuint64_t dims[2] = {k, (cuuint64_t)a.n_x};
  const cuuint64_t strides[1] = {k * 2};
  const cuuint32_t box[2] = {KS, (cuuint32_t)rows};
  return encode(map, a.x, 2, dims, strides, box);
}

template <int CG, bool SWIGLU, Form FORM, bool SPLIT>
cudaError_t launch(const LinearArgs& a, int nt, int splits, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done;
  const cudaError_t e = set_smem_limit_once(linear_tiles_kernel<CG, SWIGLU, FORM, SPLIT>, SMEM, done);
  if (e != cudaSuccess) return e;
  constexpr int FE = (SWIGLU ? 64 : 128) * CG;
  Plan p;
  p.nt = nt;
  p.x_bytes = nt / CG * KS * 2;
  p.stage_bytes = A_BYTES + p.x_bytes * (FORM == PAIR_IN ? 2 : 1);
  p.part_bytes = splits > 1 ? (nt / 8 + splits - 1) / splits * splits * PART_BYTES : 0;
  p.stages = (STAGE_AREA - p.part_bytes) / p.stage_bytes;
  if (p.stages > MAX_STAGES) p.stages = MAX_STAGES;
  p.n_m = (a.n_out + FE - 1) / FE;
  p.k_steps = (a.n_in + KS - 1) / KS;
  p.splits = splits;
  p.nt_shift = 0;
  while ((1 << p.nt_shift) < nt) ++p.nt_shift;
  p.box_rows = a.start == nullptr ? nt / CG : a.index == nullptr ? 32 / CG : 0;
  p.box_shift = p.box_rows > 0 ? 6 - CG : 2;
  p.team_shift = p.box_rows > 0 ? 0 : 1;
  const int tiles_n = (a.n_rows + nt - 1) / nt;
  p.tiles = tiles_n * p.n_m;
  p.strip = Divisor(STRIP * tiles_n);
  p.last = Divisor(p.n_m % STRIP != 0 ? p.n_m % STRIP : STRIP);
  p.n_main = a.w_last != nullptr ? a.n_groups - 1 : a.n_groups;
  // (the layer's own indices are in range)
  p.checked = a.index != nullptr && a.w_last == nullptr;
  Maps maps;
  if (!encode_w(&maps.w, a, a.w, p.n_main)) return cudaErrorInvalidValue;
  maps.w_last = maps.w;
  if (a.w_last != nullptr && !encode_w(&maps.w_last, a, a.w_last, 1)) return cudaErrorInvalidValue;
  if (!encode_x(&maps.x, a, p.box_rows > 0 ? p.box_rows : 1)) return cudaErrorInvalidValue;
  maps.x_last = maps.x;
  if (a.w_last != nullptr && a.index != nullptr && !encode_x(&maps.x_last, a, 32 / CG)) return cudaErrorInvalidValue;

  int units = sms / (CG * splits);
  if (a.start == nullptr) {
    if (p.tiles < units) units = p.tiles;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(units * CG * splits, 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG * splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG * splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, linear_tiles_kernel<CG, SWIGLU, FORM, SPLIT>, a, p, maps);
}

template <int CG, bool SPLIT>
cudaError_t launch_as(const LinearArgs& a, int nt, int splits, int sms, cudaStream_t stream) {
  if constexpr (!SPLIT) {
    if (a.pair_out) return launch<CG, true, PAIR_OUT, SPLIT>(a, nt, splits, sms, stream);
    if (a.pair_in) return launch<CG, false, PAIR_IN, SPLIT>(a, nt, splits, sms, stream);
  }
  if (a.act == ACT_SWIGLU)
    return a.out_f32 ? launch<CG, true, FP32, SPLIT>(a, nt, splits, sms, stream)
                     : launch<CG, true, BF16, SPLIT>(a, nt, splits, sms, stream);
  return a.out_f32 ? launch<CG, false, FP32, SPLIT>(a, nt, splits, sms, stream)
                   : launch<CG, false, BF16, SPLIT>(a, nt, splits, sms, stream);
}

// Clusters of so many CTAs that the device runs at once: GPCs have no whole number of
// them (of GB300's 152 SMs 8-CTA clusters take 120, 6-CTA ones 138).
int clusters(int splits, int sms) {
  static std::atomic<int> known[64][MAX_SPLITS + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev][splits].load(std::memory_order_relaxed);
  if (n == 0) {
    static std::atomic<uint64_t> done;
    const auto kernel = linear_tiles_kernel<1, false, BF16, true>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(splits * (sms / splits), 1, 1);
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (set_smem_limit_once(kernel, SMEM, done) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      n = 0;
    }
    known[dev][splits].store(n > 0 ? n : -1, std::memory_order_relaxed);
  }
  return n;
}

// How a plain product is cut: CTAs a tile, rows of a tile, parts of k.  Cycles, fitted to
// measured times: a stage of n rows takes 2 n (the products) and 96 (224 for one CTA, which
// reads more of x), 400 at least (its barriers and copies); a tile's epilogue 8 n, hidden
// but for the last tile's; a pair's start 700, joining parts 3000.  Over 90 sizes (24 to 6400
// rows, 512 to 8192 inputs) the choice is within 10 % of the best of all cuts.
struct Choice {
  int cg, nt, splits;
  long long cost;
};
Choice choose(const LinearArgs& a, int sms) {
  const int fe = a.act == ACT_SWIGLU ? 64 : 128, k_steps = (a.n_in + KS - 1) / KS;
  Choice best = {0, 0, 0, 0};
  const auto consider = [&](int cg, int n, int splits) {
    const long long tiles = (long long)((a.n_rows + n - 1) / n) * ((a.n_out + fe * cg - 1) / (fe * cg));
    const long long units = splits > 1 ? clusters(splits, sms) : sms / cg;
    if (units < 1 || tiles >= 1 << 24 || (splits > 1 && (tiles > units || k_steps < 4 * splits))) return;
    const int rows = 2 * n + (cg == 2 ? 96 : 224), step = rows > 400 ? rows : 400;
    const long long cost = (tiles + units - 1) / units * ((k_steps + splits - 1) / splits) * step +
                           8 * n / splits + (splits > 1 ? 3000 : cg == 2 ? 700 : 0);
    if (best.cg == 0 || cost < best.cost) best = {cg, n, splits, cost};
  };
  for (int n = a.out_f32 ? NT_MAX_F32 : NT_MAX; n >= 32; n -= 32) {
    consider(2, n, 1);
    consider(1, n, 1);
    // Three stages at least beside the parts.
    if (n <= 128)
      for (const int s : {2, 3, 4, 6, 8}) consider(1, n, s);
  }
  return best;
}

// The same for groups, as if they had equal numbers of rows (what they have is on the
// device).  Tiles of up to twice those rows: smaller ones leave the ring more stages (292
// rows of 24 groups 41.6 -> 37.2 us), larger ones few groups need.
Choice choose_grouped(const LinearArgs& a, int sms) {
  const int fe = a.act == ACT_SWIGLU ? 64 : 128, each = (a.n_rows + a.n_groups - 1) / a.n_groups;
  const int used = a.n_rows < a.n_groups ? a.n_rows : a.n_groups, k_steps = (a.n_in + KS - 1) / KS;
  int most = a.out_f32 ? NT_MAX_F32 : NT_MAX;
  while (most > 32 && most / 2 >= 2 * each) most /= 2;
  Choice best = {0, 0, 0, 0};
  for (int n = most; n >= 32; n /= 2)
    for (int cg = 2; cg >= 1; --cg) {
      // (two stages of pairs are all that one CTA has room for)
      if (a.pair_in && cg == 1 && n == NT_MAX) continue;
      const long long k = (each + n - 1) / n, units = sms / cg;
      const long long tiles = k * used * ((a.n_out + fe * cg - 1) / (fe * cg));
      const int rows = (int)((each + k - 1) / k), full = (a.pair_in ? 4 : 2) * rows + (cg == 2 ? 96 : 224), least = cg == 2 ? 400 : 440;
      const long long cost = (tiles + units - 1) / units * k_steps * (full > least ? full : least) +
                             8 * ((rows + 31) & ~31) + (cg == 2 ? 700 : 0);
      if (best.cg == 0 || cost < best.cost) best = {cg, n, 1, cost};
    }
  return best;
}

}  // namespace

cudaError_t launch_linear_tiles(const LinearArgs& a, int sms, cudaStream_t stream) {
  // (Weighing the cuts takes a microsecond: a thread remembers its last calls' sizes.)
  struct Known {
    int rows, groups, in, out, act, form, sms;
    Choice c;
  };
  static thread_local Known known[16] = {};
  const int groups = a.start != nullptr ? a.n_groups : 0, form = a.out_f32 + 2 * a.pair_out + 4 * a.pair_in;
  Known& k = known[(a.n_rows + 3 * a.n_in / 8 + 5 * a.n_out / 8 + groups) & 15];
  if (k.rows != a.n_rows || k.groups != groups || k.in != a.n_in || k.out != a.n_out || k.act != a.act ||
      k.form != form || k.sms != sms)
    k = {a.n_rows, groups, a.n_in, a.n_out, a.act, form, sms, groups > 0 ? choose_grouped(a, sms) : choose(a, sms)};
  const Choice c = k.c;
  if (c.splits > 1) return launch_as<1, true>(a, c.nt, c.splits, sms, stream);
  return c.cg == 2 ? launch_as<2, false>(a, c.nt, 1, sms, stream) : launch_as<1, false>(a, c.nt, 1, sms, stream);
}

}  // namespace flint
