// paged_decode.cu — attention of next tokens and short drafts (up to 16 query rows,
// tokens x the `group` heads that share a KV head) over a paged KV cache, bf16 or
// E4M3 with a scale per 16-token block and KV head.
//
// For a query row, and the keys of its KV head: scores s_j =
// scale q.k_j, o = sum_j e^{s_j} v_j / (sum_j e^{s_j} + e^sink), in one pass
// over the keys with a running maximum m, sum l and output o (2^x throughout,
// the scale carrying log2 e).  E4M3: k_j = kc_j ks and v_j = vc_j vs with one
// ks and vs a 16-key block, so ks multiplies the block's scores and vs enters
// the exponent: p'_j = 2^(s_j + log2 vs - m) is the weight of the codes, and
// l gets p'_j / vs.  A weight is thus held as f16 relative to the largest
// contribution, whatever the scales of its block; m is kept 7 below the largest
// exponent, so that weights use f16's range up to 2^15 and its steps end at 2^-31
// of the largest contribution: 2^23 keys of less than half of one are 2^-9 of it.
//
// Bound: the cache bytes.  16 (E4M3) or 8 (bf16) operations a byte at 8 query
// heads a KV head are far below the tensor cores' ridge but above the CUDA
// cores', so both products run on mma.sync m16n8k16:
//   S = Q K^T:     A = 8 or 16 query rows (of 8, the upper half is zero), B = 8 keys
//   O^T = V^T P^T: A = V^T (16 elements x 16 keys), B = P^T: the score tile's
//                  accumulator registers are its operand registers.
// 16 rows is where it ends: an SM quarter issues such a product every 16 cycles or
// so, and 32 rows of E4M3 (64 products a granule) ran at 3.7 TB/s, the tcgen05
// kernel at 5.0.  At 16 rows (8 x 30K, 2 drafts) 62 us here, 84 there.
// The order of the 128 elements inside a dot product and of the outputs is
// free, so a lane's 16-byte shared-memory loads are its operand words, and only
// V's keys have to be paired (one byte permute per two codes).  What a
// streaming kernel lives on is loads in flight: every warp copies its granules
// (16 keys: 4 KiB of codes, 8 KiB of bf16) into a ring of its own with cp.async,
// two to five of them on the way at any time, ~190 KiB an SM, with no barrier
// between warps.  (With the granule on its way in registers instead, 64 KiB an
// SM, 32 x 100K E4M3 took 440 us, 5.0 TB/s.)
// Work: the (sequence, KV head) rows of 16-key granules laid end to end and cut
// into equal shares, one per CTA (one per SM); a share's warps take its
// granules in turn, and start on the next row's while this row's results are put
// together.  A row cut between CTAs leaves partial results in the workspace, and
// the CTAs that arrive last join them in the order of the keys, so the bits do not
// depend on timing.  The lengths are on the device: every CTA computes the cuts
// itself, by a scan over the sequences.
// Measured: 8 x 100K bf16 249-256 us, 6.4-6.6 TB/s; 32 x 100K E4M3 338-342 us, 6.4-6.5
// (the copy rate: 6.7).  A single 100K E4M3 sequence: 31 us against 15 of bytes;
// the rest is the launch, three dependent look-ups before the first key (~3 us),
// and the joins (two tickets and reads through L2, ~4 us).
#include "nv_util.cuh"
#include "paged.cuh"
#include "paged_work.cuh"

namespace flint {
namespace {

using namespace pg;

// NT: groups of 8 rows.
template <bool FP8, int NT>
struct Cfg {
  // (E4M3, 32 x 100K: 16 warps of 3 slots 355 us, 12 of 4 342, 8 of 6 416: what a
  // warp holds in registers against warps that hide each other's latency.)
  static constexpr int WARPS = FP8 && NT == 1 ? 12 : 8;
  static constexpr int SLOTS = FP8 ? (NT > 1 ? 6 : 4) : 3;  // granules of a warp's ring
  static constexpr int THREADS = WARPS * 32;
  static constexpr int ROW = FP8 ? HD : 2 * HD;      // bytes of a head's key
  static constexpr int SLOT = 2 * BLOCK * ROW;       // bytes of a granule: keys, then values
  static constexpr int SMEM = WARPS * SLOTS * SLOT;
  static constexpr int O = NT * DEC_O, ML = NT * DEC_ML;  // floats of a warp's outputs, of maxima and sums
  // A warp's outputs take the last slots of its ring; the others' granules of the
  // next segment are on their way by then.
  static constexpr int PRE = SLOTS - (O * 4 + SLOT - 1) / SLOT;
  static_assert(PRE >= 1 && PRE < SLOTS, "room for both");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(addr));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void store2(const PagedAttnArgs& a, int row, int head, int d, float o0,
                                       float o1, float f) {
  const size_t nq = (size_t)a.b.nkv * a.b.group;
  *reinterpret_cast<uint32_t*>(a.out + ((size_t)row * nq + head) * HD + d) = pack_bf2(o0 * f, o1 * f);
}

// Row r of a slot holds its 16-byte chunk c at chunk c ^ mix(r) (of each
// 128-byte half): the two rows an 8-lane load phase of the keys touches, and
// the four of the values, fall into distinct banks.
__device__ __forceinline__ int mix(int r) { return ((r & 1) << 2) | ((r >> 1) & 3); }

// The maximum of a row that has seen no key: finite, so that a masked score,
// -infinity, has the weight 0 against it too.
constexpr float LOWEST = -3.402823466e38f;

// Where the warp's granules lie: lane l holds granule 32 * batch + l.
struct Batch {
  int row;        // cache row of its first key; -1: its page is not there
  float ks, vs;   // E4M3: scales of its keys and values
};

// A share's part of a row.
struct Segment {
  int seq, kvh;
  int n, g0;   // granules, the first of them
  int c0, c1;  // the CTAs that share the row
  int next;    // where the share goes on
};

}  // namespace

template <bool FP8, int NT>
__global__ void __launch_bounds__(Cfg<FP8, NT>::THREADS, 1)
    paged_decode_kernel(const __grid_constant__ PagedAttnArgs a) {
  using C = Cfg<FP8, NT>;
  using Cuts = DecCut<FP8>;
  constexpr int WARPS = C::WARPS, THREADS = C::THREADS, SLOTS = C::SLOTS;
  constexpr int ROW = C::ROW, SLOT = C::SLOT, ROWS = 8 * NT;
  constexpr float LIFT = weight_lift<FP8>;
  extern __shared__ __align__(128) uint8_t s_ring[];
  __shared__ int s_pre[MAX_SEQS + 1];            // weight (of all heads) before each sequence
  __shared__ int4 s_seq[MAX_SEQS];               // {position, row, first granule, granules}
  __shared__ int s_scan[MAX_SEQS / 32];
  __shared__ int s_new[MAX_SEQS];                // rows of the sequence
  // Parts that are joined (the warps', the CTAs'): maxima, sums, factors; the rows' joint ones.
  constexpr int PARTS = WARPS > JOIN_MOST ? WARPS : JOIN_MOST;
  __shared__ float s_m[PARTS * ROWS], s_l[PARTS * ROWS], s_mm[ROWS], s_ll[ROWS];
  __shared__ __align__(16) float s_f[PARTS * ROWS];  // read four at a time
  __shared__ int s_cut[2], s_first, s_last, s_parts;
  pdl_wait();
  pdl_trigger();
  const PagedView& b = a.b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int nq = b.nkv * b.group, gshift = 31 - __clz(b.group);  // group is a power of two

  // ---- the cuts ---------------------------------------------------------------
  static_assert(MAX_SEQS * MAX_KV_HEADS * (MAX_LENGTH / BLOCK + Cuts::weight(1)) < 1ll << 31, "32 bits");
  int cnt = 0, pre = 0, rows = 0;
  int4 info = make_int4(-1, -1, 0, 0);
  if (tid < MAX_SEQS) {
    if (tid < b.n_seqs) {
      const Seq q = load_seq(b, tid);
      const int lo = a.window > 0 ? max(0, q.first - a.window + 1) : 0;
      if (q.n > 0) {
        info = make_int4(q.first, q.q0, lo >> 4, q.len > 0 ? ((q.len - 1) >> 4) + 1 - (lo >> 4) : 0);
        cnt = Cuts::weight(info.w) * b.nkv;
      }
      s_seq[tid] = info;
      s_new[tid] = rows = q.n;
    }
  }
  // Exclusive sums over the sequences, and the total; returns how many are nonzero.
  int total;
  auto scan = [&]() {
    pre = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += v;
    }
    if (lane == 31 && warp < MAX_SEQS / 32) s_scan[warp] = pre;
    pre -= cnt;
    const int some = __syncthreads_count(cnt > 0);
    total = 0;
#pragma unroll
    for (int w = 0; w < MAX_SEQS / 32; ++w) {
      if (w == warp) pre += total;
      total += s_scan[w];
    }
    return some;
  };
  if (tid < 2) s_cut[tid] = -1;
  const int n_rows = scan() * b.nkv;
  const Cuts cuts(total, gridDim.x);
  const int size = Cuts::deal(total, n_rows, gridDim.x);
  if (size > 0) {  // few short rows
    cnt = Cuts::parts(info.w, size) * b.nkv;
    __syncthreads();  // s_scan has been read
    scan();
  }
  if (tid < MAX_SEQS && tid < b.n_seqs) {
    s_pre[tid + 1] = pre + cnt;
    if (tid == 0) s_pre[0] = 0;
    if (size > 0) {
      if (pre <= (int)blockIdx.x && (int)blockIdx.x < pre + cnt) {
        s_cut[0] = pre;
        s_first = tid;
        s_parts = cnt / b.nkv;
      }
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const long long x = (long long)cuts.share * (blockIdx.x + k);
        if (pre <= x && x < pre + cnt) {  // this sequence holds the cut
          s_cut[k] = cuts.at((int)x, pre, info.w);
          if (k == 0) s_first = tid;
        }
      }
    }
    // Rows that see nothing: zeros.
    if (info.w == 0 && info.y >= 0 && tid % gridDim.x == blockIdx.x) {
      uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)info.y * nq * HD);
      for (int i = 0; i < rows * nq * HD / 8; ++i) o[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __syncthreads();
  const int cur = s_cut[0];
  const int end = s_cut[1] < 0 ? total : s_cut[1];
  if (cur < 0 || cur >= end) return;

  const size_t tok_bytes = (size_t)b.nkv * ROW;  // one token row of a cache
  const uint32_t ring = smem_addr(s_ring) + warp * SLOTS * SLOT;
  auto outputs = [&](int w) {  // of warp w
    return reinterpret_cast<float*>(s_ring + (w * SLOTS + C::PRE) * SLOT);
  };

  auto segment = [&](int cur, int s) {
    if (size > 0) {  // all that this CTA has
      const int4 sq = s_seq[s];
      const int at = (int)blockIdx.x - cur, parts = s_parts, kvh = at / parts, part = at - kvh * parts;
      const int off = sq.w * part / parts, to = sq.w * (part + 1) / parts, c0 = (int)blockIdx.x - part;
      return Segment{s, kvh, to - off, sq.z + off, c0, c0 + parts - 1, end};
    }
    while (cur >= s_pre[s + 1]) ++s;
    const int4 sq = s_seq[s];
    const int weight = Cuts::weight(sq.w), kvh = (cur - s_pre[s]) / weight;
    const int row0 = s_pre[s] + kvh * weight;
    int off, to;
    cuts.part(cur, end, row0, sq.w, off, to);
    int c0, c1;
    if (!cuts.shared(row0, sq.w, c0, c1)) c0 = c1 = blockIdx.x;
    return Segment{s, kvh, to - off, sq.z + off, c0, c1, min(end, row0 + weight)};
  };
  uint4 qw[NT][4];
  Batch now{-1, 0.0f, 0.0f}, old{-1, 0.0f, 0.0f};
  auto mine_of = [&](const Segment& sg) { return sg.n > warp ? (sg.n - warp + WARPS - 1) / WARPS : 0; };
  // (Looked up a batch ahead, 8 and 16 granules before its use, the long E4M3 cases
  // took 8 % longer: registers and branches in the loop.)
  auto look_up = [&](const Segment& sg, int batch) {
    const int i = warp + WARPS * (32 * batch + lane);
    old = now;
    now.row = -1;
    if (i < sg.n) {
      now.row = cache_row(b, sg.seq, (sg.g0 + i) << 4);
      if (FP8 && now.row >= 0) {
        const size_t at = (size_t)(now.row >> 4) * b.nkv + sg.kvh;
        now.ks = a.k_scale[at];
        now.vs = a.v_scale[at];
      }
    }
  };
  // Granule i of the warp on its way into slot i % SLOTS.
  const int cr = FP8 ? lane >> 3 : lane >> 4, cc = FP8 ? lane & 7 : lane & 15;
  const size_t src0 = (size_t)cr * tok_bytes + 16 * cc;
  auto issue = [&](const Segment& sg, int i) {
    if (i < mine_of(sg)) {
      if ((i & 31) == 0) look_up(sg, i >> 5);
      const int row = __shfl_sync(0xffffffffu, now.row, i & 31);
      if (row >= 0) {
        constexpr int STEP = FP8 ? 4 : 2;  // rows a warp copies at a time
        const size_t at = (size_t)row * tok_bytes + (size_t)sg.kvh * ROW + src0;
        const uint8_t* k = static_cast<const uint8_t*>(a.k_cache) + at;
        const uint8_t* v = static_cast<const uint8_t*>(a.v_cache) + at;
        const uint32_t dst = ring + (i % SLOTS) * SLOT + cr * ROW;
#pragma unroll
        for (int j = 0; j < BLOCK / STEP; ++j) {
          const int c = cc ^ mix(cr + STEP * j);
          cp_async16(dst + j * STEP * ROW + 16 * c, k + (size_t)(STEP * j) * tok_bytes);
          cp_async16(dst + BLOCK * ROW + j * STEP * ROW + 16 * c, v + (size_t)(STEP * j) * tok_bytes);
        }
      }
    }
    cp_commit();
  };
  // The queries' words, to arrive while the granules are looked up, and the first
  // granules.  Row r is token r / group, head r % group.
  auto begin = [&](const Segment& sg) {
    const int n_new = s_new[sg.seq], row = s_seq[sg.seq].y;
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const int r = 8 * u + g, tok = r >> gshift;
      const uint8_t* src = reinterpret_cast<const uint8_t*>(
          a.q + ((size_t)(row + tok) * nq + sg.kvh * b.group + (r & (b.group - 1))) * HD);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // E4M3: elements 16t .. 16t + 15 and 64 + 16t ..; bf16: 32i + 8t .. + 7
        const int at = FP8 ? (i >> 1) * 128 + 32 * t + (i & 1) * 16 : 64 * i + 16 * t;
        qw[u][i] = tok < n_new ? *reinterpret_cast<const uint4*>(src + at) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
#pragma unroll 1
    for (int i = 0; i < C::PRE; ++i) issue(sg, i);
  };

  Segment sg = segment(cur, s_first);
  begin(sg);
  for (;;) {
    const int4 sq = s_seq[sg.seq];
    const int mine_n = mine_of(sg);
    const int all_lo = a.window > 0 ? max(0, sq.x + s_new[sg.seq] - a.window) : 0;  // first key that all rows see
#pragma unroll 1
    for (int i = C::PRE; i < SLOTS - 1; ++i) issue(sg, i);

    // ---- the group's queries as A fragments -----------------------------------
    // E4M3: f16, each head scaled by a power of two so that its largest element
    // lies in [2^14, 2^15): a bf16 element is then exact down to 2^-31 of it.
    uint32_t qa[NT][8][2];
    float qs[NT];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      qs[u] = a.scale_log2;
      if constexpr (FP8) {
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x[4] = {qw[u][i].x, qw[u][i].y, qw[u][i].z, qw[u][i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) mx = fmaxf(mx, fmaxf(fabsf(bf_lo(x[j])), fabsf(bf_hi(x[j]))));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 127);
        const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
        qs[u] *= __uint_as_float((uint32_t)(127 - 14 + e) << 23);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x[4] = {qw[u][i].x, qw[u][i].y, qw[u][i].z, qw[u][i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            qa[u][2 * i + (j >> 1)][j & 1] = nvu::f16x2_of(bf_lo(x[j]) * up, bf_hi(x[j]) * up);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          qa[u][2 * i][0] = qw[u][i].x;
          qa[u][2 * i][1] = qw[u][i].y;
          qa[u][2 * i + 1][0] = qw[u][i].z;
          qa[u][2 * i + 1][1] = qw[u][i].w;
        }
      }
    }
    // Rows g and g + 8 of the fragments of row groups 2v and 2v + 1.
    auto q_frag = [&](int v, int k, int half, int word) {
      return 2 * v + half < NT ? qa[2 * v + half][k][word] : 0u;
    };

    float o[NT][8][4], m[NT], l[NT];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[u][j][i] = 0.0f;
      m[u] = LOWEST;
      l[u] = 0.0f;
    }

    for (int it = 0; it < mine_n; ++it) {
      issue(sg, it + SLOTS - 1);
      cp_wait<SLOTS - 1>();
      __syncwarp();  // the other lanes' copies of granule `it` too
      // The batch of granule `it`: the issue may already be in the next one.
      const bool behind = (it >> 5) != (min(it + SLOTS - 1, mine_n - 1) >> 5);
      const int row = __shfl_sync(0xffffffffu, behind ? old.row : now.row, it & 31);
      if (row < 0) continue;
      float scale = 1.0f, lv = 0.0f, iv = 1.0f;
      if constexpr (FP8) {
        scale = __shfl_sync(0xffffffffu, behind ? old.ks : now.ks, it & 31);
        const float vs = fmaxf(__shfl_sync(0xffffffffu, behind ? old.vs : now.vs, it & 31), LEAST_SCALE);
        lv = log2f(vs);
        iv = 1.0f / vs;
      }
      const uint32_t ks = ring + (it % SLOTS) * SLOT, vsm = ks + BLOCK * ROW;
      const int key0 = (sg.g0 + warp + WARPS * it) << 4;
      const bool cut = key0 < all_lo || key0 + 15 > sq.x;  // a granule cut by a row's mask

      float c[(NT + 1) / 2][2][4] = {};  // rows g and g + 8 of two row groups
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const uint32_t kr = ks + (8 * nt + g) * ROW;
#pragma unroll
        for (int i = 0; i < ROW / 64; ++i) {  // chunks t, t + 4, ...
          const uint4 w = lds128(kr + 16 * ((4 * i + t) ^ mix(g)));
          if constexpr (FP8) {
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t k0 = e4m3x2_to_f16x2(x[j] & 0xffffu), k1 = e4m3x2_to_f16x2(x[j] >> 16);
#pragma unroll
              for (int v = 0; v < (NT + 1) / 2; ++v)
                nvu::mma_f16(c[v][nt], q_frag(v, 4 * i + j, 0, 0), q_frag(v, 4 * i + j, 1, 0),
                             q_frag(v, 4 * i + j, 0, 1), q_frag(v, 4 * i + j, 1, 1), k0, k1);
            }
          } else {
#pragma unroll
            for (int v = 0; v < (NT + 1) / 2; ++v) {
              mma_bf16(c[v][nt], q_frag(v, 2 * i, 0, 0), q_frag(v, 2 * i, 1, 0), q_frag(v, 2 * i, 0, 1),
                       q_frag(v, 2 * i, 1, 1), w.x, w.y);
              mma_bf16(c[v][nt], q_frag(v, 2 * i + 1, 0, 0), q_frag(v, 2 * i + 1, 1, 0),
                       q_frag(v, 2 * i + 1, 0, 1), q_frag(v, 2 * i + 1, 1, 1), w.z, w.w);
            }
          }
        }
      }
      float p[NT][4], mx[NT];
      bool grows = false;
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        const float f = qs[u] * scale;
#pragma unroll
        for (int i = 0; i < 4; ++i) p[u][i] = fmaf(c[u >> 1][i >> 1][2 * (u & 1) + (i & 1)], f, lv);
      }
      uint32_t seen[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
      if (cut) {
        const int n_new = s_new[sg.seq], pos_last = sq.x + n_new - 1;
        const int some_lo = a.window > 0 ? max(0, sq.x - a.window + 1) : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = key0 + 8 * (i >> 1) + 2 * t + (i & 1);
          // Whatever bits the cache holds where no row sees must not meet a zero weight.
          if (key < some_lo || key > pos_last) seen[i] = 0u;
#pragma unroll
          for (int u = 0; u < NT; ++u) {
            const int pos = sq.x + min((8 * u + g) >> gshift, n_new - 1);
            if (key > pos || (a.window > 0 && key <= pos - a.window)) p[u][i] = -INFINITY;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        mx[u] = fmaxf(fmaxf(p[u][0], p[u][1]), fmaxf(p[u][2], p[u][3]));
        mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
        mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
        grows |= mx[u] > m[u] + LIFT + 8.0f;
      }
      // The maximum moves only when it grows by more than 2^8 (or from nothing), so
      // that the outputs are rarely scaled: weights stay below 2^(LIFT + 8).
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          const float mn = fmaxf(m[u], mx[u] - LIFT), r = ex2(m[u] - mn);
          l[u] *= r;
          m[u] = mn;
          const float r0 = __shfl_sync(0xffffffffu, r, 8 * t), r1 = __shfl_sync(0xffffffffu, r, 8 * t + 4);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            o[u][j][0] *= r0;
            o[u][j][1] *= r1;
            o[u][j][2] *= r0;
            o[u][j][3] *= r1;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < NT; ++u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[u][i] = ex2(p[u][i] - m[u]);
        l[u] = fmaf((p[u][0] + p[u][1]) + (p[u][2] + p[u][3]), iv, l[u]);
      }
      // Keys 2t, 2t + 1, 2t + 8, 2t + 9; chunk pi(g) of each.
      const int vc = (g >> 1) | ((g & 1) << 2);
      if constexpr (FP8) {
        uint32_t pb[NT][2];
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          pb[u][0] = nvu::f16x2_of(p[u][0], p[u][1]);
          pb[u][1] = nvu::f16x2_of(p[u][2], p[u][3]);
        }
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 2 * t + (i & 1) + 8 * (i >> 1);
          w[i] = lds128(vsm + r * ROW + 16 * (vc ^ mix(r)));
          if (cut) {
            w[i].x &= seen[i];
            w[i].y &= seen[i];
            w[i].z &= seen[i];
            w[i].w &= seen[i];
          }
        }
        const uint32_t x0[4] = {w[0].x, w[0].y, w[0].z, w[0].w}, x1[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
        const uint32_t y0[4] = {w[2].x, w[2].y, w[2].z, w[2].w}, y1[4] = {w[3].x, w[3].y, w[3].z, w[3].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // elements 16 pi(g) + 2j, + 1
          const uint32_t x = __byte_perm(x0[j >> 1], x1[j >> 1], j & 1 ? 0x7362 : 0x5140);
          const uint32_t y = __byte_perm(y0[j >> 1], y1[j >> 1], j & 1 ? 0x7362 : 0x5140);
          const uint32_t a0 = e4m3x2_to_f16x2(x & 0xffffu), a1 = e4m3x2_to_f16x2(x >> 16);
          const uint32_t a2 = e4m3x2_to_f16x2(y & 0xffffu), a3 = e4m3x2_to_f16x2(y >> 16);
#pragma unroll
          for (int u = 0; u < NT; ++u) nvu::mma_f16(o[u][j], a0, a1, a2, a3, pb[u][0], pb[u][1]);
        }
      } else {
        // A weight as a bf16 pair hi + lo: 16 significant bits.
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          split_bf2(p[u][0], p[u][1], ph[u][0], pl[u][0]);
          split_bf2(p[u][2], p[u][3], ph[u][1], pl[u][1]);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint4 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 2 * t + (i & 1) + 8 * (i >> 1);
            w[i] = lds128(vsm + r * ROW + 16 * ((8 * half + vc) ^ mix(r)));
            if (cut) {
              w[i].x &= seen[i];
              w[i].y &= seen[i];
              w[i].z &= seen[i];
              w[i].w &= seen[i];
            }
          }
          const uint32_t x0[4] = {w[0].x, w[0].y, w[0].z, w[0].w}, x1[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
          const uint32_t y0[4] = {w[2].x, w[2].y, w[2].z, w[2].w}, y1[4] = {w[3].x, w[3].y, w[3].z, w[3].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // elements 64 half + 8 pi(g) + 2j, + 1
            const uint32_t a0 = __byte_perm(x0[j], x1[j], 0x5410), a1 = __byte_perm(x0[j], x1[j], 0x7632);
            const uint32_t a2 = __byte_perm(y0[j], y1[j], 0x5410), a3 = __byte_perm(y0[j], y1[j], 0x7632);
#pragma unroll
            for (int u = 0; u < NT; ++u) {
              mma_bf16(o[u][4 * half + j], a0, a1, a2, a3, ph[u][0], ph[u][1]);
              mma_bf16(o[u][4 * half + j], a0, a1, a2, a3, pl[u][0], pl[u][1]);
            }
          }
        }
      }
      __syncwarp();  // the slot is free for granule it + SLOTS
    }
    cp_wait<0>();

    // ---- the warps' results ---------------------------------------------------
    // Output element e of tile j and lane row g, row 8u + h: at ((16u + 2j + e) * 8 + g) * 8 + h.
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
      l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
      if (t == 0) {
        s_m[warp * ROWS + 8 * u + g] = m[u] > LOWEST ? m[u] : -INFINITY;
        s_l[warp * ROWS + 8 * u + g] = l[u];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float2*>(outputs(warp) + ((16 * u + 2 * j + e) * 8 + g) * 8 + 2 * t) =
              make_float2(o[u][j][2 * e], o[u][j][2 * e + 1]);
    }
    // The next segment's first granules travel while this one's results are joined.
    const bool more = sg.next < end;
    Segment following = sg;
    if (more) {
      following = segment(sg.next, sg.seq);
      begin(following);
    }
    __syncthreads();
    // Factors of n parts and the rows' joint maxima and sums.
    auto weigh = [&](int n) {
      for (int i = tid; i < n * ROWS; i += THREADS) {
        const int r = i % ROWS;
        float mm = -INFINITY;
        for (int w = 0; w < n; ++w) mm = fmaxf(mm, s_m[w * ROWS + r]);
        s_f[i] = s_m[i] > -INFINITY ? ex2(s_m[i] - mm) : 0.0f;
      }
      __syncthreads();
      if (tid < ROWS) {
        float mm = -INFINITY, ll = 0.0f;
        for (int w = 0; w < n; ++w) {
          mm = fmaxf(mm, s_m[w * ROWS + tid]);
          ll = fmaf(s_l[w * ROWS + tid], s_f[w * ROWS + tid], ll);
        }
        s_mm[tid] = mm;
        s_ll[tid] = ll;
      }
      __syncthreads();
    };
    // Four rows' values of an element, item i of the layout above.
    auto rows_of = [&](int i) { return 8 * (i >> 8) + 4 * (i & 1); };
    auto add = [&](float4& x, const float4& v, int w, int i) {
      const float4 f = *reinterpret_cast<const float4*>(&s_f[w * ROWS + rows_of(i)]);
      x.x = fmaf(v.x, f.x, x.x);
      x.y = fmaf(v.y, f.y, x.y);
      x.z = fmaf(v.z, f.z, x.z);
      x.w = fmaf(v.w, f.w, x.w);
    };
    // Finished: lanes l and l ^ 16 hold the elements d and d + 1, and take two rows each.
    auto finish = [&](int i, const float4& x) {
      const bool e = (i >> 4) & 1;
      const float y0 = __shfl_xor_sync(0xffffffffu, e ? x.x : x.z, 16);
      const float y1 = __shfl_xor_sync(0xffffffffu, e ? x.y : x.w, 16);
      const int gg = (i >> 1) & 7, j = (i >> 5) & 7, pg = (gg >> 1) | ((gg & 1) << 2);
      const int d = FP8 ? 16 * pg + 2 * j : 64 * (j >> 2) + 8 * pg + 2 * (j & 3);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = rows_of(i) + 2 * e + k, tok = r >> gshift, head = sg.kvh * b.group + (r & (b.group - 1));
        const float mine = k ? (e ? x.w : x.y) : (e ? x.z : x.x), other = k ? y1 : y0;
        if (tok < s_new[sg.seq])
          store2(a, sq.y + tok, head, d, e ? other : mine, e ? mine : other, row_factor(a, head, s_mm[r], s_ll[r]));
      }
    };
    weigh(WARPS);
    const bool whole = sg.c0 == sg.c1;
    float* slot = dec_slot(a.ws, blockIdx.x, (int)blockIdx.x == sg.c0, NT);
    auto store_ml = [&](float* to) {
      if (tid < ROWS) {
        __stcg(to + tid, s_mm[tid]);
        __stcg(to + ROWS + tid, s_ll[tid]);
      }
    };
    for (int i = tid; i < 256 * NT; i += THREADS) {
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) add(x, *reinterpret_cast<const float4*>(outputs(w) + 4 * i), w, i);
      if (whole)
        finish(i, x);
      else
        __stcg(reinterpret_cast<float4*>(slot + C::ML) + i, x);
    }
    if (!whole) {
      store_ml(slot);
      for (Join jn(blockIdx.x, sg.c0, sg.c1);; jn.up()) {
        __threadfence();
        __syncthreads();
        if (tid == 0) s_last = jn.arrive(a.ws);
        __syncthreads();
        if (!s_last) break;
        for (int i = tid; i < jn.n * ROWS; i += THREADS) {
          const float* src = dec_slot(a.ws, jn.cta(i / ROWS), jn.begins(i / ROWS), NT);
          s_m[i] = __ldcg(src + i % ROWS);
          s_l[i] = __ldcg(src + ROWS + i % ROWS);
        }
        __syncthreads();
        weigh(jn.n);
        float* to = dec_slot(a.ws, jn.first, jn.begins(0), NT);
        for (int i = tid; i < 256 * NT; i += THREADS) {
          float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll JOIN
          for (int k = 0; k < jn.n; ++k) {
            const float* from = dec_slot(a.ws, jn.cta(k), jn.begins(k), NT) + C::ML;
            add(x, __ldcg(reinterpret_cast<const float4*>(from) + i), k, i);
          }
          if (jn.top)
            finish(i, x);
          else
            __stcg(reinterpret_cast<float4*>(to + C::ML) + i, x);
        }
        if (jn.top) break;
        store_ml(to);
      }
    }
    if (!more) break;
    __syncthreads();  // the shared buffers are free
    sg = following;
  }
}

namespace {
template <bool FP8, int NT>
cudaError_t launch(const PagedAttnArgs& a, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done;
  using C = Cfg<FP8, NT>;
  const cudaError_t e = set_smem_limit_once(paged_decode_kernel<FP8, NT>, C::SMEM, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms < MAX_CTAS ? sms : MAX_CTAS, 1, 1);
  cfg.blockDim = dim3(C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_decode_kernel<FP8, NT>, a);
}
}  // namespace

cudaError_t launch_paged_decode(const PagedAttnArgs& a, bool fp8, int sms, cudaStream_t stream) {
  if (a.b.max_q * a.b.group <= 8) return fp8 ? launch<true, 1>(a, sms, stream) : launch<false, 1>(a, sms, stream);
  return fp8 ? launch<true, 2>(a, sms, stream) : launch<false, 2>(a, sms, stream);
}

size_t paged_attn_workspace_bytes() { return attn_ws_bytes(); }
size_t paged_attn_workspace_clear_bytes() { return WS_HEAD; }
size_t paged_attn_workspace_error_at() { return WS_ERROR; }
size_t paged_attn_workspace_stall_at() { return WS_STALL; }

}  // namespace flint
