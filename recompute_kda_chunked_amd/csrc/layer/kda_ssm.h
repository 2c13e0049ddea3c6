// Internal interface between the entry points of a state-space layer's
// operators (kda_ssm_host.cpp) and their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// The scan's decoding form. Strides are elements between tokens.
struct SsmStepArgs {
  int n_seqs, H, G;
  int64_t T, n_slots;
  float dt_min, dt_max;
  const void *x, *dt, *B, *C;
  int64_t xs, dts, Bs, Cs;
  const float *A_log, *D, *dt_bias;
  const int32_t *cu, *idx;
  float* state;
  void* y;
  bool zero_rest;  // zero the rows of y that belong to no sequence (with cu)
};
hipError_t launch_ssm_recurrent(int dtype, int N, int P, const SsmStepArgs& a, hipStream_t s);

// Group norm. Partial sums: group_norm_partials(...) rows of dweight [C] then
// (with a bias) dbias [C].
struct GroupNormArgs {
  int64_t rows, xs, gs;  // strides of x and gate in elements
  int C, groups, W, act, center;
  float eps;
  const void *x, *gate, *dy;
  const float *weight, *bias;
  void *y, *dx, *dgate;
  float* partials;
};
int64_t group_norm_partials(int dtype, int C, int groups, int64_t rows);
hipError_t launch_group_norm_fwd(int dtype, int gate, const GroupNormArgs& a, hipStream_t s);
hipError_t launch_group_norm_bwd(int dtype, int gate, const GroupNormArgs& a, hipStream_t s);


// A step size: clamp(softplus(raw + bias)), NaN kept.
__device__ __forceinline__ float ssm_step(float z, float lo, float hi) {
  const float s = fmaxf(z, 0.f) + log1pf(expf(-fabsf(z)));
  const float d = z != z ? z : s;
  return d < lo ? lo : (d > hi ? hi : d);
}

}  // namespace kda
