// linear_rows.cu — matrix products of a few rows, plain or grouped: every weight
// is read once for up to 32 rows, straight from global memory into the operands
// of the warp-level tensor-core product.
//
// D (16 weight rows x 8 rows of x) += W X^T in steps of 32 k.  The order of k
// inside a step is free as long as both operands take the same: lane 4 r + c reads
// the 16 bytes of k = 8c .. 8c + 7 of weight rows r and r + 8 and of x row r, which
// are the fragments of two m16n8k16 products as they come, with no staging.  The
// eight warps of a CTA share the 16 weight rows and take every eighth step; their
// sums meet in shared memory in a fixed order.  SwiGLU: the 16 weight rows are 8 gate
// and the 8 up rows of the same outputs.
//
// Bound: the weights' bytes for one row, launch and first-load latency at a few MB.
#include "linear.cuh"

namespace flint {
namespace {

using namespace lin;

constexpr int THREADS = 256, WARPS = THREADS / 32;

__device__ __forceinline__ uint4 ld16(const uint16_t* p, bool there) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (there) v = __ldg(reinterpret_cast<const uint4*>(p));
  return v;
}

// NB blocks of 8 rows of x at a time.
template <int NB, bool SWIGLU>
__global__ void __launch_bounds__(THREADS) linear_rows_kernel(const LinearArgs a) {
  constexpr int FE = SWIGLU ? 8 : 16, NT = 8 * NB;
  __shared__ float part[WARPS][NT][17];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  pdl_wait();
  pdl_trigger();
  const int g = a.start == nullptr ? 0 : blockIdx.y;
  const Rows rows = group_rows(a, g);
  const int first = a.start == nullptr ? blockIdx.y * NT : 0;
  const int step_rows = a.start == nullptr ? gridDim.y * NT : NT;
  const int f0 = blockIdx.x * FE;
  const int m = a.n_out * (SWIGLU ? 2 : 1);
  const uint16_t* w = a.w_last != nullptr && g == a.n_groups - 1 ? a.w_last : a.w + (size_t)g * m * a.n_in;
  // Weight rows of this lane, the second 8 further or the up row of the same output.
  const bool there0 = f0 + r < a.n_out, there1 = SWIGLU ? there0 : f0 + r + 8 < a.n_out;
  const uint16_t* w0 = w + (size_t)(f0 + r) * a.n_in;
  const uint16_t* w1 = w0 + (size_t)(SWIGLU ? a.n_out : 8) * a.n_in;

  for (int t0 = first; t0 < rows.n; t0 += step_rows) {
    const uint16_t* xr[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int t = t0 + 8 * b + r;
      int row = t < rows.n ? rows.r0 + t : -1;
      if (row >= 0 && a.index != nullptr) row = __ldg(a.index + row);
      xr[b] = (unsigned)row < (unsigned)a.n_x ? a.x + (size_t)row * a.n_in : nullptr;
    }
    float acc[NB][4] = {};
#pragma unroll 4
    for (int k = 32 * warp + 8 * c; k < a.n_in + 8 * c; k += 32 * WARPS) {
      const bool in = k < a.n_in;
      const uint4 u = ld16(w0 + k, in && there0), v = ld16(w1 + k, in && there1);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint4 x = ld16(xr[b] + k, in && xr[b] != nullptr);
        mma_bf16(acc[b], u.x, v.x, u.y, v.y, x.x, x.y);
        mma_bf16(acc[b], u.z, v.z, u.w, v.w, x.z, x.w);
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[warp][8 * b + 2 * c + (i & 1)][r + 8 * (i >> 1)] = acc[b][i];
    __syncthreads();
    for (int o = tid; o < FE * NT; o += THREADS) {
      const int t = t0 + o / FE, f = o % FE;
      if (t < rows.n && f0 + f < a.n_out) {
        const int row = rows.r0 + t;
        bool ok = true;
        if (a.index != nullptr) ok = (unsigned)__ldg(a.index + row) < (unsigned)a.n_x;
        float v = 0.0f, up = 0.0f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) {
          v += part[i][o / FE][f];
          if constexpr (SWIGLU) up += part[i][o / FE][f + 8];
        }
        if (a.bias != nullptr) {
          v += __ldg(a.bias + (size_t)g * m + f0 + f);
          if constexpr (SWIGLU) up += __ldg(a.bias + (size_t)g * m + a.n_out + f0 + f);
        }
        if constexpr (SWIGLU)
          v = activate(v, ACT_SILU) * up;
        else
          v = activate(v, a.act);
        const size_t at = (size_t)row * a.n_out + f0 + f;
        if (ok && a.out_f32) {
          float* out = static_cast<float*>(a.out);
          if (a.residual != nullptr) v += static_cast<const float*>(a.residual)[at];
          out[at] = v;
        } else if (ok) {
          uint16_t* out = static_cast<uint16_t*>(a.out);
          if (a.residual != nullptr) v += bf_lo(static_cast<const uint16_t*>(a.residual)[at]);
          out[at] = f2bf(v);
        }
      }
    }
    __syncthreads();
  }
}

template <int NB, bool SWIGLU>
cudaError_t launch(const LinearArgs& a, cudaStream_t stream) {
  constexpr int FE = SWIGLU ? 8 : 16, NT = 8 * NB;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.n_out + FE - 1) / FE, a.start == nullptr ? (a.n_rows + NT - 1) / NT : a.n_groups, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, linear_rows_kernel<NB, SWIGLU>, a);
}

}  // namespace

cudaError_t launch_linear_rows(const LinearArgs& a, cudaStream_t stream) {
  const bool sw = a.act == ACT_SWIGLU;
  if (a.n_rows <= 8) return sw ? launch<1, true>(a, stream) : launch<1, false>(a, stream);
  if (a.n_rows <= 16) return sw ? launch<2, true>(a, stream) : launch<2, false>(a, stream);
  return sw ? launch<4, true>(a, stream) : launch<4, false>(a, stream);
}

}  // namespace flint
