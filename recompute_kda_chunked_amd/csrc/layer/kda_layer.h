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

// Sums of `nb` partial rows of M = n0 + n1 floats, in a fixed order: the
// first n0 columns to out0, the rest to out1 unless it is null (nb = 0:
// zeros).
struct ParamReduceArgs {
  const float* partials;
  int64_t nb;
  int n0, n1;
  float *out0, *out1;
};
hipError_t launch_param_reduce(const ParamReduceArgs& a, hipStream_t s);

// The norm behind the operator; rows of V elements. Partial sums of dweight:
// gated_norm_blocks(...) rows of V floats.
struct GatedNormArgs {
  int64_t rows;
  int act;  // KDA_ACT_*
  float eps;
  const void *o, *gate, *dy;
  const float* weight;
  void *y, *d_o, *dgate;
  float* partials;
};
int gated_norm_blocks(int dtype, int V, int64_t rows);
hipError_t launch_gated_norm_fwd(int dtype, int V, const GatedNormArgs& a, hipStream_t s);
hipError_t launch_gated_norm_bwd(int dtype, int V, const GatedNormArgs& a, hipStream_t s);

// Between two blocks; rows of D elements. Partial sums: block_norm_blocks(...)
// rows of dw_post (when w_post) then dw_pre.
struct BlockNormArgs {
  int64_t T;
  int D;
  float scale, eps;
  const void *x, *y, *gate, *dx_out, *dh;
  const float *w_post, *w_pre;
  void *x_out, *h, *dx, *dy, *dgate;
  float* partials;
};
int block_norm_blocks(int dtype, int D, int64_t T);
hipError_t launch_block_norm_fwd(int dtype, int gate, const BlockNormArgs& a, hipStream_t s);
hipError_t launch_block_norm_bwd(int dtype, int gate, const BlockNormArgs& a, hipStream_t s);

// The short convolution. Partial sums: short_conv_blocks(...) rows of dweight
// [C][W] then dbias [C].
struct ShortConvArgs {
  int N, C;
  int64_t T, xs, n_slots;
  int act;  // KDA_ACT_*
  const void *x, *init, *dy, *dfinal;
  const float *weight, *bias;
  const int32_t *cu, *idx;
  void *y, *final_state, *dx, *dinit, *state;
  float* partials;
};
int64_t short_conv_blocks(int C, int64_t T);
hipError_t launch_short_conv_fwd(int dtype, int W, const ShortConvArgs& a, hipStream_t s);
hipError_t launch_short_conv_bwd(int dtype, int W, const ShortConvArgs& a, hipStream_t s);
hipError_t launch_short_conv_update(int dtype, int W, const ShortConvArgs& a, hipStream_t s);

}  // namespace kda
