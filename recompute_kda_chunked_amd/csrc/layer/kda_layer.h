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
  bool zero_rest;  // zero the rows of o that belong to no sequence (with cu)
};
hipError_t launch_recurrent(int dtype, int D, bool gdn2, const RecurrentArgs& a, hipStream_t s);

// Whether a launch of the row kernels that moves `bytes` loads and stores its
// rows past the caches (non-temporal). From about the 256 MiB that the
// memory-side cache holds they cannot be in it and only push each other out;
// below, rows that the kernel before wrote often are, and the kernel behind
// finds the ones stored. bf16, microseconds with plain loads / with loads past
// the caches, rows in the caches where they fit (in brackets: never in them):
//   gated norm forward    275 MB 41.7 / 43.1 (42.9 / 43.5)   334 MB 55.7 / 52.5   403 MB 69.3 / 60.5
//   gated norm backward   168 MB 33.0 / 35.9 (36.0 / 35.8)   335 MB 66.7 / 62.2   671 MB 133 / 113
//   block norm forward    268 MB 41.2 / 48.2 (48.2 / 48.3)   335 MB 65.6 / 58.8
//   block norm backward   268 MB 55.2 / 57.0 (56.0 / 56.3)   393 MB 82.0 / 73.4   537 MB 108 / 95
//   convolution backward  201 MB 48.3 / 52.6 (50.6 / 53.0)   295 MB 83.2 / 82.9   403 MB 90.3 / 85.9
// Stores on top of that, with the outputs kept and an elementwise kernel that
// reads them behind (in brackets: without it), plain / past the caches:
//   gated norm forward    101 MB 29.1 / 30.7 (19.6 / 18.6)   403 MB 106.7 / 103.7 (66.8 / 63.1)
// and for a forward with its backward behind, outputs kept: gated norm 8192 x
// 64 x 128 199 / 186, block norm 8191 x 4096 164 / 158, convolution 8192 x 8192
// 147 / 143.
inline bool streams_past_caches(int64_t bytes) { return bytes >= (int64_t{288} << 20); }

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
  bool zero_rest;  // update: zero the rows of y that belong to no sequence (with cu)
};
int64_t short_conv_blocks(int C, int64_t T);
hipError_t launch_short_conv_fwd(int dtype, int W, const ShortConvArgs& a, hipStream_t s);
hipError_t launch_short_conv_bwd(int dtype, int W, const ShortConvArgs& a, hipStream_t s);
hipError_t launch_short_conv_update(int dtype, int W, const ShortConvArgs& a, hipStream_t s);

}  // namespace kda
