// linear_rows.cu — matrix products of a few rows (plain up to FEW_ROWS, grouped up to
// FEW_GROUPED in all): every weight is read once, straight from global memory into the
// operands of the warp-level tensor-core product.
//
// D (16 weight rows x 8 NB rows of x) += W X^T in steps of 32 k.  The order of k
// inside a step is free as long as both operands take the same: lane 4 r + c reads
// the 16 bytes of k = 8c .. 8c + 7 of weight rows r and r + 8 and of x row r, which
// are the fragments of two m16n8k16 products as they come, with no staging.  The
// warps of a CTA share the 16 weight rows and take steps in turn; their sums meet in shared
// memory in a fixed order.  SwiGLU: the 16 weight rows are 8 gate and the 8 up rows of the
// same outputs.
//
// Groups: a CTA for every row and 16 weight rows, which works if the row is the first of a
// group, for all of the group's.
//
// Bound: launch and first-load latency at a few MB of weights, and their bytes, of which
// less is in flight than there could be: one row of 2048 -> 5120 (21 MB) takes 5.8 us from HBM
// and 4.5 from L2, 16 rows of 4096 -> 2048 8.8 and 5.4.  The loads of DEEP steps stand before
// their products, but the compiler gives the kernels 44 to 74 registers, where DEEP steps of
// weights alone take 64, and so moves some loads to their products; rows of x come with the
// products; and 320 equal CTAs lie on 152 SMs.  Tried: an L2 prefetch of the weights while the
// kernel before ends (8.1 us from HBM), more rows here (33: 14 us; the tiled kernel 9).
// Grouped, 2048 -> SwiGLU 512: 1 row 7 us (from L2 3.6; tiled 12.7), 6 rows 8-9 (13.7), 12 rows
// 15.8 (15.6), and 16 rows of 4096 -> 4096 116 (92).
#include "linear.cuh"

namespace flint {
namespace {

using namespace lin;

constexpr int DEEP = 8;   // steps whose weights are loaded before the first one's products

__device__ __forceinline__ uint4 ld16(const uint16_t* p, bool there) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (there) v = *reinterpret_cast<const uint4*>(p);
  return v;
}

// All rows of x, NB blocks of 8.
static_assert(FEW_ROWS == 16 && FEW_GROUPED == 8, "one or two blocks of rows, one");

template <int NB, bool SWIGLU, int WARPS, bool GROUPED>
__global__ void __launch_bounds__(32 * WARPS) linear_rows_kernel(const LinearArgs a) {
  constexpr int FE = SWIGLU ? 8 : 16, NT = 8 * NB;
  __shared__ float part[WARPS][NT][17];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  const int f0 = blockIdx.x * FE, m = a.n_out * (SWIGLU ? 2 : 1);
  pdl_wait();
  pdl_trigger();
  int g = 0;
  Rows rows = {0, a.n_rows};
  if constexpr (GROUPED) {
    __shared__ int found;
    if (tid == 0) found = GROUP_LIMIT;
    __syncthreads();
    for (int i = tid; i < a.n_groups; i += 32 * WARPS) {
      const Rows q = group_rows(a, i);
      if (q.n > 0 && q.r0 == (int)blockIdx.y) atomicMin(&found, i);
    }
    __syncthreads();
    g = found;
    if (g == GROUP_LIMIT) return;
    rows = group_rows(a, g);
  }
  const uint16_t* w = a.w + (size_t)g * m * a.n_in;
  // Weight rows of this lane, the second 8 further or the up row of the same output.
  const bool there0 = f0 + r < a.n_out, there1 = SWIGLU ? there0 : f0 + r + 8 < a.n_out;
  const uint16_t* w0 = w + (size_t)(f0 + r) * a.n_in;
  const uint16_t* w1 = w0 + (size_t)(SWIGLU ? a.n_out : 8) * a.n_in;
  const uint16_t* xr[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    int row = 8 * b + r < rows.n ? rows.r0 + 8 * b + r : -1;
    if (GROUPED && row >= 0 && a.index != nullptr) row = a.index[row];
    xr[b] = (unsigned)row < (unsigned)a.n_x ? a.x + (size_t)row * a.n_in : nullptr;
  }
  float acc[NB][4] = {};
  const int steps = (a.n_in + 31) / 32;
  for (int s0 = warp; s0 < steps; s0 += WARPS * DEEP) {
    uint4 u[DEEP], v[DEEP];
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
      const int k = 32 * (s0 + WARPS * d) + 8 * c;
      u[d] = ld16(w0 + k, k < a.n_in && there0);
      v[d] = ld16(w1 + k, k < a.n_in && there1);
    }
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
      const int k = 32 * (s0 + WARPS * d) + 8 * c;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint4 x = ld16(xr[b] + k, k < a.n_in && xr[b] != nullptr);
        mma_bf16(acc[b], u[d].x, v[d].x, u[d].y, v[d].y, x.x, x.y);
        mma_bf16(acc[b], u[d].z, v[d].z, u[d].w, v[d].w, x.z, x.w);
      }
    }
  }
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[warp][8 * b + 2 * c + (i & 1)][r + 8 * (i >> 1)] = acc[b][i];
  __syncthreads();
#pragma unroll
  for (int o = tid; o < FE * NT; o += 32 * WARPS) {
    const int t = o / FE, f = o % FE;
    const int row = rows.r0 + t;
    bool store = t < rows.n && f0 + f < a.n_out;
    if (GROUPED && store && a.index != nullptr) store = (unsigned)a.index[row] < (unsigned)a.n_x;
    if (store) {
      float v = 0.0f, up = 0.0f;
#pragma unroll
      for (int i = 0; i < WARPS; ++i) {
        v += part[i][t][f];
        if constexpr (SWIGLU) up += part[i][t][f + 8];
      }
      if (a.bias != nullptr) {
        v += a.bias[(size_t)g * m + f0 + f];
        if constexpr (SWIGLU) up += a.bias[(size_t)g * m + a.n_out + f0 + f];
      }
      if constexpr (SWIGLU)
        v = activate(v, ACT_SILU) * up;
      else
        v = activate(v, a.act);
      const size_t at = (size_t)row * a.n_out + f0 + f;
      if (a.out_f32) {
        if (a.residual != nullptr) v += static_cast<const float*>(a.residual)[at];
        static_cast<float*>(a.out)[at] = v;
      } else {
        if (a.residual != nullptr) v += bf_lo(static_cast<const uint16_t*>(a.residual)[at]);
        static_cast<uint16_t*>(a.out)[at] = f2bf(v);
      }
    }
  }
}

template <int NB, int WARPS, bool GROUPED>
cudaError_t launch(const LinearArgs& a, cudaStream_t stream) {
  const int fe = a.act == ACT_SWIGLU ? 8 : 16;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.n_out + fe - 1) / fe, GROUPED ? a.n_rows : 1, 1);
  cfg.blockDim = dim3(32 * WARPS, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.act == ACT_SWIGLU ? cudaLaunchKernelEx(&cfg, linear_rows_kernel<NB, true, WARPS, GROUPED>, a)
                             : cudaLaunchKernelEx(&cfg, linear_rows_kernel<NB, false, WARPS, GROUPED>, a);
}

template <int NB, bool GROUPED>
cudaError_t launch_as(const LinearArgs& a, cudaStream_t stream) {
  // Sixteen warps where eight would take more than one turn of DEEP steps.
  return a.n_in > 32 * 8 * DEEP ? launch<NB, 16, GROUPED>(a, stream) : launch<NB, 8, GROUPED>(a, stream);
}

}  // namespace

cudaError_t launch_linear_rows(const LinearArgs& a, cudaStream_t stream) {
  if (a.start != nullptr) return launch_as<1, true>(a, stream);
  return a.n_rows <= 8 ? launch_as<1, false>(a, stream) : launch_as<2, false>(a, stream);
}

}  // namespace flint
