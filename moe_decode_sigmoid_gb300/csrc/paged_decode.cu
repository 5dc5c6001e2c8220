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
// cores', so both products run on mma.sync m16n8k16 with the operands loaded
// straight from global memory into fragments, without shared memory: the order
// of the 128 elements inside a dot product and of the outputs is free, so a
// lane's 16-byte loads are its operand words, and only V's keys have to be
// paired (one byte permute per two codes).
//   S = Q K^T:    A = 8 query heads (rows 8..15 zero), B = 8 keys a tile
//   O^T = V^T P^T: A = V^T (16 elements x 16 keys), B = P^T: the score tile's
//                  accumulator registers are its operand registers.
// Work: the (sequence, KV head) rows' 16-key granules laid end to end and cut
// into equal shares, one per CTA (one per SM); a share's warps take its
// granules in turn.  A row cut between CTAs leaves partial results in the
// workspace, and the CTA that arrives last joins them in their order, so the
// bits do not depend on timing.  The lengths are on the device: every CTA
// computes the cut itself, by a scan over the sequences.
#include "nv_util.cuh"
#include "paged.cuh"
#include "paged_work.cuh"

namespace flint {
namespace {

using namespace pg;

template <bool FP8>
struct Cfg {
  // Loads in flight are what a streaming kernel lives on: a warp keeps one
  // granule's K and V (4 KiB of codes, 8 KiB of bf16) in registers on the way.
  static constexpr int WARPS = FP8 ? 16 : 12;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int KW = FP8 ? 16 : 32;  // registers of a granule's keys (and values)
  static constexpr int SMEM = WARPS * DEC_O * 4;
};

__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// What a warp needs of one granule besides its bytes.
struct Granule {
  int row;      // cache row of its first key; -1: its page is not there
  float ks;     // E4M3: scale of its keys
  float lv;     // E4M3: log2 of the scale of its values
  float iv;     // E4M3: 1 / that scale
};

template <bool FP8>
struct Tile {
  uint32_t k[Cfg<FP8>::KW], v[Cfg<FP8>::KW];
};

}  // namespace

template <bool FP8>
__global__ void __launch_bounds__(Cfg<FP8>::THREADS, 1)
    paged_decode_kernel(const __grid_constant__ PagedAttnArgs a) {
  constexpr int WARPS = Cfg<FP8>::WARPS, THREADS = Cfg<FP8>::THREADS, KW = Cfg<FP8>::KW;
  constexpr int ES = FP8 ? 1 : 2;  // bytes of a cached element
  extern __shared__ __align__(16) float s_o[];  // [WARPS][DEC_O]
  __shared__ long long s_pre[MAX_SEQS + 1];     // granules (of all heads) before each sequence
  __shared__ int4 s_seq[MAX_SEQS];              // {position, row, first granule, granules}
  __shared__ long long s_scan[MAX_SEQS / 32];
  __shared__ float s_m[WARPS * 8], s_l[WARPS * 8];
  __shared__ float s_jm[MAX_CTAS * 8], s_jl[MAX_CTAS * 8];
  __shared__ int s_first, s_last;
  pdl_wait();
  pdl_trigger();
  const PagedView& b = a.b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int nq = b.nkv * b.group;

  // ---- the cut: granules before every sequence -------------------------------
  long long cnt = 0;
  if (tid < MAX_SEQS && tid < b.n_seqs) {
    const Seq q = load_seq(b, tid);
    const int pos = q.first;  // one row a sequence
    const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    const int g0 = lo >> 4, n = q.n > 0 && pos >= 0 ? (pos >> 4) + 1 - g0 : 0;
    s_seq[tid] = make_int4(q.n > 0 ? pos : -1, q.n > 0 ? q.q0 : -1, g0, n);
    cnt = (long long)n * b.nkv;
  }
  if (tid < MAX_SEQS) {
    long long incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_scan[warp] = incl;
    cnt = incl;
  }
  __syncthreads();
  if (tid < MAX_SEQS) {
    for (int w = 0; w < warp; ++w) cnt += s_scan[w];
    s_pre[tid + 1] = cnt;
    if (tid == 0) s_pre[0] = 0;
  }
  __syncthreads();
  const long long total = s_pre[b.n_seqs];
  const long long share = max((total + gridDim.x - 1) / gridDim.x, (long long)DEC_MIN_SHARE);
  long long cur = share * blockIdx.x;
  const long long end = min(cur + share, total);
  if (tid < b.n_seqs && tid < MAX_SEQS) {
    if (s_pre[tid] <= cur && cur < s_pre[tid + 1]) s_first = tid;
    // A row that sees nothing: zeros.
    if (s_seq[tid].w == 0 && s_seq[tid].y >= 0 && tid % gridDim.x == blockIdx.x) {
      uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)s_seq[tid].y * nq * HD);
      for (int i = 0; i < nq * HD / 8; ++i) o[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __syncthreads();
  if (cur >= end) return;
  int s = s_first;

  const size_t tok_bytes = (size_t)b.nkv * HD * ES;  // one token row of a cache

  while (cur < end) {
    while (cur >= s_pre[s + 1]) ++s;
    const int4 sq = s_seq[s];
    const int rel = (int)(cur - s_pre[s]);
    const int kvh = rel / sq.w, off = rel - kvh * sq.w;
    const int n = (int)min((long long)(sq.w - off), end - cur);  // granules of this segment
    const int first_key = a.window > 0 ? max(0, sq.x - a.window + 1) : 0;

    // ---- the group's queries as A fragments ---------------------------------
    // E4M3: f16, each head scaled by a power of two so that its largest element
    // lies in [2^14, 2^15): a bf16 element is then exact down to 2^-31 of it.
    uint32_t qa[8][2];
    float qs = a.scale_log2;
    {
      const uint8_t* src = reinterpret_cast<const uint8_t*>(
          a.q + ((size_t)sq.y * nq + kvh * b.group + g) * HD);
      const bool live = g < b.group;
      if constexpr (FP8) {
        uint4 w[4];  // elements 16t .. 16t + 15 and 64 + 16t ..
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = live ? *reinterpret_cast<const uint4*>(src + (i >> 1) * 128 + 32 * t + (i & 1) * 16)
                      : make_uint4(0u, 0u, 0u, 0u);
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
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
          const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            qa[2 * i + (j >> 1)][j & 1] = nvu::f16x2_of(bf_lo(x[j]) * up, bf_hi(x[j]) * up);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // elements 32i + 8t .. + 7
          const uint4 w = live ? *reinterpret_cast<const uint4*>(src + 64 * i + 16 * t)
                               : make_uint4(0u, 0u, 0u, 0u);
          qa[2 * i][0] = w.x;
          qa[2 * i][1] = w.y;
          qa[2 * i + 1][0] = w.z;
          qa[2 * i + 1][1] = w.w;
        }
      }
    }

    const uint8_t* kbase = static_cast<const uint8_t*>(a.k_cache) + (size_t)kvh * HD * ES + 16 * t;
    const uint8_t* vbase = static_cast<const uint8_t*>(a.v_cache) + (size_t)kvh * HD * ES + 16 * g;
    const int g0 = sq.z + off;  // first granule

    // Lane l looks up the warp's granule 32 * batch + l.
    Granule mine{-1, 0.0f, 0.0f, 1.0f};
    auto look_up = [&](int batch) {
      const int i = warp + WARPS * (32 * batch + lane);
      mine = Granule{-1, 0.0f, 0.0f, 1.0f};
      if (i < n) {
        mine.row = cache_row(b, s, (g0 + i) << 4);
        if (FP8 && mine.row >= 0) {
          const size_t at = (size_t)(mine.row >> 4) * b.nkv + kvh;
          // A scale of zero would take a block's weights out of the sum.
          const float vs = fmaxf(__ldg(a.v_scale + at), 7.8886090522101181e-31f);  // 2^-100
          mine.ks = __ldg(a.k_scale + at);
          mine.lv = log2f(vs);
          mine.iv = 1.0f / vs;
        }
      }
    };
    Tile<FP8> tile;
    auto load_k = [&](int row) {
      const uint8_t* p = kbase + (size_t)(row + g) * tok_bytes;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int i = 0; i < KW / 8; ++i) {
          const uint4 w = ldg_stream(p + (size_t)(8 * nt) * tok_bytes + 64 * i);
          uint32_t* d = tile.k + nt * (KW / 2) + 4 * i;
          d[0] = w.x; d[1] = w.y; d[2] = w.z; d[3] = w.w;
        }
    };
    auto load_v = [&](int row) {
      const uint8_t* p = vbase + (size_t)(row + 2 * t) * tok_bytes;
#pragma unroll
      for (int key = 0; key < 4; ++key)  // keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
        for (int i = 0; i < KW / 16; ++i) {
          const uint4 w = ldg_stream(p + (size_t)((key & 1) + 8 * (key >> 1)) * tok_bytes + 128 * i);
          uint32_t* d = tile.v + key * (KW / 4) + 4 * i;
          d[0] = w.x; d[1] = w.y; d[2] = w.z; d[3] = w.w;
        }
    };

    float o[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
    float m = -INFINITY, l = 0.0f;

    const int mine_n = n > warp ? (n - warp + WARPS - 1) / WARPS : 0;
    if (mine_n > 0) {
      look_up(0);
      Granule cg;
      auto pick = [&](int i) {
        Granule x;
        x.row = __shfl_sync(0xffffffffu, mine.row, i & 31);
        x.ks = FP8 ? __shfl_sync(0xffffffffu, mine.ks, i & 31) : 1.0f;
        x.lv = FP8 ? __shfl_sync(0xffffffffu, mine.lv, i & 31) : 0.0f;
        x.iv = FP8 ? __shfl_sync(0xffffffffu, mine.iv, i & 31) : 1.0f;
        return x;
      };
      cg = pick(0);
      if (cg.row >= 0) {
        load_k(cg.row);
        load_v(cg.row);
      }
      for (int it = 0; it < mine_n; ++it) {
        // The next granule.
        Granule ng{-1, 0.0f, 0.0f, 1.0f};
        if (it + 1 < mine_n) {
          if (((it + 1) & 31) == 0) look_up((it + 1) >> 5);
          ng = pick(it + 1);
        }
        float p[4];
        if (cg.row >= 0) {
          float c[2][4] = {};
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              if constexpr (FP8) {
                const uint32_t w = tile.k[nt * 8 + kk];
                nvu::mma_f16(c[nt], qa[kk][0], 0u, qa[kk][1], 0u, e4m3x2_to_f16x2(w & 0xffffu),
                             e4m3x2_to_f16x2(w >> 16));
              } else {
                mma_bf16(c[nt], qa[kk][0], 0u, qa[kk][1], 0u, tile.k[nt * 16 + 2 * kk],
                         tile.k[nt * 16 + 2 * kk + 1]);
              }
            }
          const float f = FP8 ? qs * cg.ks : qs;
          p[0] = fmaf(c[0][0], f, cg.lv);
          p[1] = fmaf(c[0][1], f, cg.lv);
          p[2] = fmaf(c[1][0], f, cg.lv);
          p[3] = fmaf(c[1][1], f, cg.lv);
          const int key0 = (g0 + warp + WARPS * it) << 4;
          if (key0 < first_key || key0 + 15 > sq.x) {  // a granule cut by the mask
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = key0 + 8 * (i >> 1) + 2 * t + (i & 1);
              if (key < first_key || key > sq.x) {
                p[i] = -INFINITY;
                // whatever bits the cache holds there, they must not meet a zero weight
#pragma unroll
                for (int w = 0; w < KW / 4; ++w) tile.v[i * (KW / 4) + w] = 0u;
              }
            }
          }
        }
        if (ng.row >= 0) load_k(ng.row);
        if (cg.row >= 0) {
          float mx = fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          // The maximum moves only when it grows by more than 2^8 (or from
          // nothing): weights stay below 2^8, and the outputs are rarely scaled.
          if (__any_sync(0xffffffffu, mx > m + 8.0f)) {
            const float mn = fmaxf(m, mx);
            const float f = m > -INFINITY ? ex2(m - mn) : 0.0f;
            l *= f;
            m = mn;
            const float f0 = __shfl_sync(0xffffffffu, f, 8 * t), f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              o[j][0] *= f0;
              o[j][1] *= f1;
              o[j][2] *= f0;
              o[j][3] *= f1;
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i] = ex2(p[i] - m);
          l = fmaf((p[0] + p[1]) + (p[2] + p[3]), cg.iv, l);
          if constexpr (FP8) {
            const uint32_t b0 = nvu::f16x2_of(p[0], p[1]), b1 = nvu::f16x2_of(p[2], p[3]);
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
              for (int h = 0; h < 2; ++h) {  // elements 16g + 4w + 2h, + 1
                const uint32_t x = __byte_perm(tile.v[w], tile.v[4 + w], h ? 0x7362 : 0x5140);
                const uint32_t y = __byte_perm(tile.v[8 + w], tile.v[12 + w], h ? 0x7362 : 0x5140);
                nvu::mma_f16(o[2 * w + h], e4m3x2_to_f16x2(x & 0xffffu), e4m3x2_to_f16x2(x >> 16),
                             e4m3x2_to_f16x2(y & 0xffffu), e4m3x2_to_f16x2(y >> 16), b0, b1);
              }
          } else {
            // A weight as a bf16 pair hi + lo: 16 significant bits.
            uint32_t h0, l0, h1, l1;
            split_bf2(p[0], p[1], h0, l0);
            split_bf2(p[2], p[3], h1, l1);
#pragma unroll
            for (int w = 0; w < 8; ++w) {  // elements 64 (w / 4) + 8g + 2 (w % 4), + 1
              const uint32_t x0 = __byte_perm(tile.v[w], tile.v[8 + w], 0x5410);
              const uint32_t x1 = __byte_perm(tile.v[w], tile.v[8 + w], 0x7632);
              const uint32_t y0 = __byte_perm(tile.v[16 + w], tile.v[24 + w], 0x5410);
              const uint32_t y1 = __byte_perm(tile.v[16 + w], tile.v[24 + w], 0x7632);
              mma_bf16(o[w], x0, x1, y0, y1, h0, h1);
              mma_bf16(o[w], x0, x1, y0, y1, l0, l1);
            }
          }
        }
        if (ng.row >= 0) load_v(ng.row);
        cg = ng;
      }
    }

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
    const bool whole = n == sq.w;
    // CTAs that share the row, and this one's slot.
    const long long row0 = cur - off;
    const int c0 = (int)(row0 / share), c1 = (int)((row0 + sq.w - 1) / share);
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
        const int d = FP8 ? 16 * gg + 2 * j : 64 * (j >> 2) + 8 * gg + 2 * (j & 3);
        if (h < b.group) dec_store(a, sq.y, kvh * b.group + h, d, mm, ll, o0, o1);
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
          const int d = FP8 ? 16 * gg + 2 * j : 64 * (j >> 2) + 8 * gg + 2 * (j & 3);
          if (h < b.group) dec_store(a, sq.y, kvh * b.group + h, d, mm, ll, o0, o1);
        }
      }
    }
    __syncthreads();  // the shared buffers are free
    cur += n;
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

}  // namespace flint
