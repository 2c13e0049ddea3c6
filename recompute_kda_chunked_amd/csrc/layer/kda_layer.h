// Internal interface between the entry points of the operators around the
// chunked one (kda_layer_host.cpp) and their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// The recurrent form. Strides are elements between tokens.
struct RecurrentArgs {
  int N, H;
  int64_t T, n_slots;
  float scale, lb, eps;
  int gate_mode, gate_head;
  const void *q, *k, *v, *g, *beta, *bk, *wv;  // beta, or (GDN-2) raw_b and raw_w
  int64_t qs, ks, vs, gs, bes, bks, wvs;
  const float *A_log, *dt_bias;
  const int32_t *cu, *idx;
  float* state;
  void* o;
};
hipError_t launch_recurrent(int dtype, int D, bool gdn2, const RecurrentArgs& a, hipStream_t s);

}  // namespace kda
