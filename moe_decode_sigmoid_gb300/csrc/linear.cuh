// linear.cuh — what the kernels of the linear side of a prompt share: a group's
// rows with everything the host could not check kept in bounds, activations.
//
// Every input of these calls, weights and bias too, can be what the library's kernel before
// wrote, which may still run when this one begins.  So all are read by ordinary loads behind
// pdl_wait(), none through the read-only path, which is for what nobody writes while a kernel runs.
#pragma once

#include "common.cuh"
#include "linear.h"

namespace flint {
namespace lin {

// Rows [r0, r0 + n) of a group.
struct Rows {
  int r0, n;
};
__device__ __forceinline__ Rows group_rows(const LinearArgs& a, int g) {
  if (a.start == nullptr) return {0, a.n_rows};
  const int lo = min(max(a.start[g], 0), a.n_rows);
  return {lo, min(max(a.start[g + 1], lo), a.n_rows) - lo};
}

// v / (1 + exp(-v)), for v < 0 as v e / (1 + e) with e = exp(v), which does not overflow (from
// v = -88.8 on the first form is zero, the other down to -103, where e is); and
// v (1 + erf(v / sqrt 2)) / 2 by the complement, which keeps its relative accuracy where 1 + erf
// cancels.
__device__ __forceinline__ float activate(float v, int act) {
  if (act == ACT_SILU) {
    const float e = expf(-fabsf(v));
    return (v < 0.0f ? v * e : v) / (1.0f + e);
  }
  if (act == ACT_GELU) return 0.5f * v * erfcf(-0.70710678118654752f * v);
  return v;
}

}  // namespace lin
}  // namespace flint
