// paged_decode.cu — attention of next tokens (one query row a sequence) over a
// paged KV cache, bf16 or E4M3 with a scale per 16-token block and KV head.
//
// For a row and the `group` query heads that share KV head g: scores s_j =
// scale q.k_j, o = sum_j e^{s_j} v_j / (sum_j e^{s_j} + e^sink), in one pass
// over the keys with a running maximum m, sum l and output o (2^x throughout,
// the scale carrying log2 e).  E4M3: k_j = kc_j ks and v_j = vc_j vs with one
// ks and vs a 16-key block, so ks multiplies the block's scores and vs enters
// the exponent: p'_j = 2^(s_j + log2 vs - m) is the weight of the codes, and
// l gets p'_j / vs.  A weight is thus held as f16 relative to the largest
// contribution, whatever the scales of its block.
//
// Bound: the cache bytes.  16 (E4M3) or 8 (bf16) operations a byte at 8 query
// heads a KV head are far below the tensor cores' ridge but above the CUDA
// cores', so both products run on mma.sync m16n8k16:
//   S = Q K^T:     A = 8 query heads (rows 8..15 zero), B = 8 keys a tile
//   O^T = V^T P^T: A = V^T (16 elements x 16 keys), B = P^T: the score tile's
//                  accumulator registers are its operand registers.
// The order of the 128 elements inside a dot product and of the outputs is
// free, so a lane's 16-byte shared-memory loads are its operand words, and only
// V's keys have to be paired (one byte permute per two codes).  What a
// streaming kernel lives on is loads in flight: every warp copies its granules
// (16 keys: 4 KiB of codes, 8 KiB of bf16) into a ring of its own with cp.async,
// two or three of them on the way at any time, ~190 KiB an SM, with no barrier
// between warps.  (With the granule on its way in registers instead, 64 KiB an
// SM, 32 x 100K E4M3 took 440 us, 5.0 TB/s.)
// Work: the (sequence, KV head) rows of 16-key granules laid end to end and cut
// into equal shares, one per CTA (one per SM); a share's warps take its
// granules in turn.  A row cut between CTAs leaves partial results in the
// workspace, and the CTA that arrives last joins them in their order, so the
// bits do not depend on timing.  The lengths are on the device: every CTA
// computes the cuts itself, by a scan over the sequences.
#include "nv_util.cuh"
#include "paged.cuh"
#include "paged_work.cuh"

namespace flint {
namespace {

using namespace pg;

template <bool FP8>
struct Cfg {
  static constexpr int WARPS = FP8 ? 16 : 8;
  static constexpr int SLOTS = 3;                    // granules of a warp's ring
  static constexpr int THREADS = WARPS * 32;
  static constexpr int ROW = FP8 ? HD : 2 * HD;      // bytes of a head's key
  static constexpr int SLOT = 2 * BLOCK * ROW;       // bytes of a granule: keys, then values
  static constexpr int SMEM = WARPS * SLOTS * SLOT;  // the warps' results reuse it
  static_assert(SMEM >= WARPS * DEC_O * 4, "the joint buffer fits");
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

// Where the warp's granules lie: lane l holds granule 32 * batch + l.
struct Batch {
  int row;        // cache row of its first key; -1: its page is not there
  float ks, vs;   // E4M3: scales of its keys and values
};

}  // namespace

template <bool FP8>
__global__ void __launch_bounds__(Cfg<FP8>::THREADS, 1)
    paged_decode_kernel(const __grid_constant__ PagedAttnArgs a) {
  constexpr int WARPS = Cfg<FP8>::WARPS, THREADS = Cfg<FP8>::THREADS, SLOTS = Cfg<FP8>::SLOTS;
  constexpr int ROW = Cfg<FP8>::ROW, SLOT = Cfg<FP8>::SLOT;
  extern __shared__ __align__(128) float s_o[];  // the rings; then [WARPS][DEC_O]
  __shared__ int s_pre[MAX_SEQS + 1];            // weight (of all heads) before each sequence
  __shared__ int4 s_seq[MAX_SEQS];               // {position, row, first granule, granules}
  __shared__ int s_scan[MAX_SEQS / 32];
  __shared__ float s_m[WARPS * 8], s_l[WARPS * 8];
  __shared__ float s_jm[MAX_CTAS * 8], s_jl[MAX_CTAS * 8];
  __shared__ int s_cut[2], s_first, s_last;
  pdl_wait();
  pdl_trigger();
  const PagedView& b = a.b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int nq = b.nkv * b.group;

  // ---- the cuts ---------------------------------------------------------------
  // Lengths are below 2^23 tokens, so 256 sequences of 8 heads weigh below 2^31.
  int cnt = 0, pre = 0;
  int4 info = make_int4(-1, -1, 0, 0);
  if (tid < MAX_SEQS) {
    if (tid < b.n_seqs) {
      const Seq q = load_seq(b, tid);
      const int pos = q.first;  // one row a sequence
      const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
      if (q.n > 0) {
        info = make_int4(pos, q.q0, lo >> 4, pos >= 0 ? (pos >> 4) + 1 - (lo >> 4) : 0);
        cnt = DecCut::weight(info.w) * b.nkv;
      }
      s_seq[tid] = info;
    }
    pre = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += v;
    }
    if (lane == 31) s_scan[warp] = pre;
    pre -= cnt;
  }
  if (tid < 2) s_cut[tid] = -1;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < MAX_SEQS / 32; ++w) {
    if (w == warp) pre += total;
    total += s_scan[w];
  }
  const DecCut cuts(total, gridDim.x);
  if (tid < MAX_SEQS && tid < b.n_seqs) {
    s_pre[tid + 1] = pre + cnt;
    if (tid == 0) s_pre[0] = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const long long x = (long long)cuts.share * (blockIdx.x + k);
      if (pre <= x && x < pre + cnt) {  // this sequence holds the cut
        s_cut[k] = cuts.at((int)x, pre, info.w);
        if (k == 0) s_first = tid;
      }
    }
    // A row that sees nothing: zeros.
    if (info.w == 0 && info.y >= 0 && tid % gridDim.x == blockIdx.x) {
      uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)info.y * nq * HD);
      for (int i = 0; i < nq * HD / 8; ++i) o[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __syncthreads();
  int cur = s_cut[0];
  const int end = s_cut[1] < 0 ? total : s_cut[1];
  if (cur < 0 || cur >= end) return;
  int s = s_first;

  const size_t tok_bytes = (size_t)b.nkv * ROW;  // one token row of a cache
  const uint32_t ring = smem_addr(s_o) + warp * SLOTS * SLOT;

  while (cur < end) {
    while (cur >= s_pre[s + 1]) ++s;
    const int4 sq = s_seq[s];
    const int weight = DecCut::weight(sq.w), kvh = (cur - s_pre[s]) / weight;
    const int row0 = s_pre[s] + kvh * weight;
    int off, to;
    cuts.part(cur, end, row0, sq.w, off, to);
    const int n = to - off;                    // granules of this segment
    const int first_key = a.window > 0 ? max(0, sq.x - a.window + 1) : 0;
    const int g0 = sq.z + off;                 // the first of them

    // The queries' words, to arrive while the granules are looked up.
    uint4 qw[4];
    {
      const uint8_t* src = reinterpret_cast<const uint8_t*>(
          a.q + ((size_t)sq.y * nq + kvh * b.group + g) * HD);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // E4M3: elements 16t .. 16t + 15 and 64 + 16t ..; bf16: 32i + 8t .. + 7
        const int at = FP8 ? (i >> 1) * 128 + 32 * t + (i & 1) * 16 : 64 * i + 16 * t;
        qw[i] = g < b.group ? *reinterpret_cast<const uint4*>(src + at) : make_uint4(0u, 0u, 0u, 0u);
      }
    }

    const int mine_n = n > warp ? (n - warp + WARPS - 1) / WARPS : 0;
    Batch now{-1, 0.0f, 0.0f}, old{-1, 0.0f, 0.0f};
    auto look_up = [&](int batch) {
      const int i = warp + WARPS * (32 * batch + lane);
      old = now;
      now.row = -1;
      if (i < n) {
        now.row = cache_row(b, s, (g0 + i) << 4);
        if (FP8 && now.row >= 0) {
          const size_t at = (size_t)(now.row >> 4) * b.nkv + kvh;
          now.ks = __ldg(a.k_scale + at);
          now.vs = __ldg(a.v_scale + at);
        }
      }
    };
    // Granule i of the warp on its way into slot i % SLOTS.
    const int cr = FP8 ? lane >> 3 : lane >> 4, cc = FP8 ? lane & 7 : lane & 15;
    const size_t src0 = (size_t)cr * tok_bytes + (size_t)kvh * ROW + 16 * cc;
    auto issue = [&](int i) {
      if (i < mine_n) {
        if ((i & 31) == 0) look_up(i >> 5);
        const int row = __shfl_sync(0xffffffffu, now.row, i & 31);
        if (row >= 0) {
          constexpr int STEP = FP8 ? 4 : 2;  // rows a warp copies at a time
          const size_t at = (size_t)row * tok_bytes + src0;
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
#pragma unroll
    for (int i = 0; i < SLOTS - 1; ++i) issue(i);

    // ---- the group's queries as A fragments -----------------------------------
    // E4M3: f16, each head scaled by a power of two so that its largest element
    // lies in [2^14, 2^15): a bf16 element is then exact down to 2^-31 of it.
    uint32_t qa[8][2];
    float qs = a.scale_log2;
    if constexpr (FP8) {
      float mx = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x[4] = {qw[i].x, qw[i].y, qw[i].z, qw[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) mx = fmaxf(mx, fmaxf(fabsf(bf_lo(x[j])), fabsf(bf_hi(x[j]))));
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int e = min(max((int)(__float_as_uint(mx) >> 23) - 127, -100), 127);
      const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
      qs *= __uint_as_float((uint32_t)(127 - 14 + e) << 23);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x[4] = {qw[i].x, qw[i].y, qw[i].z, qw[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          qa[2 * i + (j >> 1)][j & 1] = nvu::f16x2_of(bf_lo(x[j]) * up, bf_hi(x[j]) * up);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        qa[2 * i][0] = qw[i].x;
        qa[2 * i][1] = qw[i].y;
        qa[2 * i + 1][0] = qw[i].z;
        qa[2 * i + 1][1] = qw[i].w;
      }
    }

    float o[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
    float m = -INFINITY, l = 0.0f;

    for (int it = 0; it < mine_n; ++it) {
      issue(it + SLOTS - 1);
      cp_wait<SLOTS - 1>();
      __syncwarp();  // the other lanes' copies of granule `it` too
      // The batch of granule `it`: the issue may already be in the next one.
      const bool behind = (it >> 5) != (min(it + SLOTS - 1, mine_n - 1) >> 5);
      const int row = __shfl_sync(0xffffffffu, behind ? old.row : now.row, it & 31);
      if (row < 0) continue;
      float f = qs, lv = 0.0f, iv = 1.0f;
      if constexpr (FP8) {
        f *= __shfl_sync(0xffffffffu, behind ? old.ks : now.ks, it & 31);
        // A scale of zero would take a block's weights out of the sum: 2^-100.
        const float vs = fmaxf(__shfl_sync(0xffffffffu, behind ? old.vs : now.vs, it & 31),
                               7.8886090522101181e-31f);
        lv = log2f(vs);
        iv = 1.0f / vs;
      }
      const uint32_t ks = ring + (it % SLOTS) * SLOT, vsm = ks + BLOCK * ROW;
      const int key0 = (g0 + warp + WARPS * it) << 4;
      const bool cut = key0 < first_key || key0 + 15 > sq.x;  // a granule cut by the mask

      float c[2][4] = {};
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const uint32_t kr = ks + (8 * nt + g) * ROW;
#pragma unroll
        for (int i = 0; i < ROW / 64; ++i) {  // chunks t, t + 4, ...
          const uint4 w = lds128(kr + 16 * ((4 * i + t) ^ mix(g)));
          if constexpr (FP8) {
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              nvu::mma_f16(c[nt], qa[4 * i + j][0], 0u, qa[4 * i + j][1], 0u,
                           e4m3x2_to_f16x2(x[j] & 0xffffu), e4m3x2_to_f16x2(x[j] >> 16));
          } else {
            mma_bf16(c[nt], qa[2 * i][0], 0u, qa[2 * i][1], 0u, w.x, w.y);
            mma_bf16(c[nt], qa[2 * i + 1][0], 0u, qa[2 * i + 1][1], 0u, w.z, w.w);
          }
        }
      }
      float p[4];
      p[0] = fmaf(c[0][0], f, lv);
      p[1] = fmaf(c[0][1], f, lv);
      p[2] = fmaf(c[1][0], f, lv);
      p[3] = fmaf(c[1][1], f, lv);
      uint32_t seen[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
      if (cut) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = key0 + 8 * (i >> 1) + 2 * t + (i & 1);
          if (key < first_key || key > sq.x) {
            p[i] = -INFINITY;
            seen[i] = 0u;  // whatever bits the cache holds there must not meet a zero weight
          }
        }
      }
      float mx = fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // The maximum moves only when it grows by more than 2^8 (or from
      // nothing): weights stay below 2^8, and the outputs are rarely scaled.
      if (__any_sync(0xffffffffu, mx > m + 8.0f)) {
        const float mn = fmaxf(m, mx);
        const float r = m > -INFINITY ? ex2(m - mn) : 0.0f;
        l *= r;
        m = mn;
        const float r0 = __shfl_sync(0xffffffffu, r, 8 * t), r1 = __shfl_sync(0xffffffffu, r, 8 * t + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j][0] *= r0;
          o[j][1] *= r1;
          o[j][2] *= r0;
          o[j][3] *= r1;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = ex2(p[i] - m);
      l = fmaf((p[0] + p[1]) + (p[2] + p[3]), iv, l);
      // Keys 2t, 2t + 1, 2t + 8, 2t + 9; chunk pi(g) of each.
      const int vc = (g >> 1) | ((g & 1) << 2);
      if constexpr (FP8) {
        const uint32_t b0 = nvu::f16x2_of(p[0], p[1]), b1 = nvu::f16x2_of(p[2], p[3]);
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
          nvu::mma_f16(o[j], e4m3x2_to_f16x2(x & 0xffffu), e4m3x2_to_f16x2(x >> 16),
                       e4m3x2_to_f16x2(y & 0xffffu), e4m3x2_to_f16x2(y >> 16), b0, b1);
        }
      } else {
        // A weight as a bf16 pair hi + lo: 16 significant bits.
        uint32_t h0, l0, h1, l1;
        split_bf2(p[0], p[1], h0, l0);
        split_bf2(p[2], p[3], h1, l1);
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
            mma_bf16(o[4 * half + j], a0, a1, a2, a3, h0, h1);
            mma_bf16(o[4 * half + j], a0, a1, a2, a3, l0, l1);
          }
        }
      }
      __syncwarp();  // the slot is free for granule it + SLOTS
    }
    cp_wait<0>();
    __syncthreads();  // the rings are done with: their memory takes the results

    // ---- the warps' results ---------------------------------------------------
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (t == 0) {
      s_m[warp * 8 + g] = m;
      s_l[warp * 8 + g] = l;
    }
    // Output element e of tile j and lane row g, head h at ((2j + e) * 8 + g) * 8 + h.
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        *reinterpret_cast<float2*>(s_o + warp * DEC_O + ((2 * j + e) * 8 + g) * 8 + 2 * t) =
            make_float2(o[j][2 * e], o[j][2 * e + 1]);
    __syncthreads();
    int c0, c1;
    const bool whole = !cuts.shared(row0, sq.w, c0, c1);
    float* slot = dec_slot(a.ws, blockIdx.x, (int)blockIdx.x == c0);
    for (int i = tid; i < 512; i += THREADS) {  // (tile j, lane row, head): elements d, d + 1
      const int h = i & 7, r = i >> 3, j = r >> 3, gg = r & 7;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) mm = fmaxf(mm, s_m[w * 8 + h]);
      float ll = 0.0f, o0 = 0.0f, o1 = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float mw = s_m[w * 8 + h], f = mw > -INFINITY ? ex2(mw - mm) : 0.0f;
        const float* src = s_o + w * DEC_O + (16 * j + gg) * 8 + h;
        ll = fmaf(s_l[w * 8 + h], f, ll);
        o0 = fmaf(src[0], f, o0);
        o1 = fmaf(src[64], f, o1);
      }
      if (whole) {
        const int pg = (gg >> 1) | ((gg & 1) << 2);
        const int d = FP8 ? 16 * pg + 2 * j : 64 * (j >> 2) + 8 * pg + 2 * (j & 3);
        if (h < b.group) store2(a, sq.y, kvh * b.group + h, d, o0, o1, row_factor(a, kvh * b.group + h, mm, ll));
      } else {
        __stcg(slot + DEC_ML + (16 * j + gg) * 8 + h, o0);
        __stcg(slot + DEC_ML + (16 * j + gg) * 8 + h + 64, o1);
        if (r == 0) {
          __stcg(slot + h, mm);
          __stcg(slot + 8 + h, ll);
        }
      }
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        uint32_t* ticket = ws_tickets(a.ws) + c0;
        const bool last = atomicAdd(ticket, 1u) == (uint32_t)(c1 - c0);
        if (last) *ticket = 0u;  // ready for the next call
        __threadfence();
        s_last = last;
      }
      __syncthreads();
      if (s_last) {
        const int segs = c1 - c0 + 1;
        for (int i = tid; i < segs * 8; i += THREADS) {
          const float* src = dec_slot(a.ws, c0 + (i >> 3), i < 8);
          s_jm[i] = __ldcg(src + (i & 7));
          s_jl[i] = __ldcg(src + 8 + (i & 7));
        }
        __syncthreads();
        const int h = tid & 7;
        float mm = -INFINITY, ll = 0.0f;
        for (int i = 0; i < segs; ++i) mm = fmaxf(mm, s_jm[i * 8 + h]);
        for (int i = 0; i < segs; ++i) {
          const float mw = s_jm[i * 8 + h], f = mw > -INFINITY ? ex2(mw - mm) : 0.0f;
          ll = fmaf(s_jl[i * 8 + h], f, ll);
        }
        for (int i = tid; i < 512; i += THREADS) {
          const int r = i >> 3, j = r >> 3, gg = r & 7;
          const int at = DEC_ML + (16 * j + gg) * 8 + h;
          float o0 = 0.0f, o1 = 0.0f;
#pragma unroll 8
          for (int k = 0; k < segs; ++k) {
            const float* src = dec_slot(a.ws, c0 + k, k == 0) + at;
            const float mw = s_jm[k * 8 + h], f = mw > -INFINITY ? ex2(mw - mm) : 0.0f;
            o0 = fmaf(__ldcg(src), f, o0);
            o1 = fmaf(__ldcg(src + 64), f, o1);
          }
          const int pg = (gg >> 1) | ((gg & 1) << 2);
        const int d = FP8 ? 16 * pg + 2 * j : 64 * (j >> 2) + 8 * pg + 2 * (j & 3);
          if (h < b.group) store2(a, sq.y, kvh * b.group + h, d, o0, o1, row_factor(a, kvh * b.group + h, mm, ll));
        }
      }
    }
    __syncthreads();  // the shared buffers are free
    cur = min(end, row0 + weight);
  }
}

cudaError_t launch_paged_decode(const PagedAttnArgs& a, bool fp8, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> done[2];
  const int smem = fp8 ? Cfg<true>::SMEM : Cfg<false>::SMEM;
  const cudaError_t e = fp8 ? set_smem_limit_once(paged_decode_kernel<true>, smem, done[1])
                            : set_smem_limit_once(paged_decode_kernel<false>, smem, done[0]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms < MAX_CTAS ? sms : MAX_CTAS, 1, 1);
  cfg.blockDim = dim3(fp8 ? Cfg<true>::THREADS : Cfg<false>::THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return fp8 ? cudaLaunchKernelEx(&cfg, paged_decode_kernel<true>, a)
             : cudaLaunchKernelEx(&cfg, paged_decode_kernel<false>, a);
}

size_t paged_attn_workspace_bytes() { return attn_ws_bytes(); }
size_t paged_attn_workspace_clear_bytes() { return WS_HEAD; }
size_t paged_attn_workspace_error_at() { return WS_ERROR; }

}  // namespace flint
