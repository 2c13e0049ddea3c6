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

// The scan over packed sequences, in chunks of ssm_chunk(dtype) tokens of one
// sequence. A chunk has a slot: sequence n's first is cu[n] / Q + n, which
// leaves room for every sequence's chunks in T / Q + n_seqs slots and needs no
// table; a slot without a chunk is passed over.
constexpr int ssm_chunk(int dtype) { return dtype == 0 ? 64 : 128; }
struct SsmArgs {
  int n_seqs, H, G, P;
  int64_t T, slots;
  float dt_min, dt_max;
  const void *x, *dt, *B, *C, *dy;
  int64_t xs, dts, Bs, Cs;
  const float *A_log, *D, *dt_bias, *init, *dfinal;
  const int32_t* cu;
  void *y, *dx, *ddt, *dB, *dC;
  float *final_state, *dinit;
  // Workspace. steps [slots][H][Q]: {dt, high and low part of the chunk's
  // running sum of log2 decays, d dt / d raw_dt}. S and dS: the states entering
  // each chunk and the gradients of those leaving it, [slots][H][P / 64] and then in
  // the order of accumulators, in the problem's dtype [N / 16][64 / 32][lane][2][4],
  // or with S_full in fp32 [N / 16][64 / 16][lane][4].
  float* steps;
  void *S, *dS;
  bool S_full;
  // Segments of `seg` chunks (0: none) of sequences of more than long_from tokens,
  // in seg_slots slots of their own: what each adds to its state, and its log2
  // decay, [directions][seg_slots][H].., the former in the order of accumulators.
  int seg;
  int64_t seg_slots, long_from;
  float *local, *seg_log;
  // Of the gradients (see k_ssm_scalars): per token {what dl adds up from it on in
  // the chunk, before it, the step size's own part, from it on in its tile of 16
  // tokens} [slots][H][Q] of four, and before it in its tile; per chunk {states'
  // part of dl, dD} and the sums over pairs of tiles [slots][H][Q / 16][Q / 16].
  float *sums, *before, *ends, *cross;
  float *pB, *pC;        // partial dB and dC [blocks behind the whole ones][Q][N] where sets > 1
  float *param;          // per slot {dA, ddt_bias, dD} [3 H]
  // Blocks that take all heads of a group in a chunk, and into how many the heads
  // of each chunk and group behind those are divided.
  unsigned whole;
  int sets;
};
hipError_t launch_ssm_steps(int dtype, const SsmArgs& a, hipStream_t s);
// `dirs` directions from dir0: 0 in sequence order, 1 (gradients) back.
hipError_t launch_ssm_state(int dtype, int N, int dirs, int dir0, const SsmArgs& a, hipStream_t s);
hipError_t launch_ssm_out(int dtype, int N, const SsmArgs& a, hipStream_t s);
hipError_t launch_ssm_grad(int dtype, int N, const SsmArgs& a, hipStream_t s);
hipError_t launch_ssm_scalars(int dtype, const SsmArgs& a, hipStream_t s);
hipError_t launch_ssm_reduce(int dtype, int N, const SsmArgs& a, hipStream_t s);

// Group norm. Partial sums: group_norm_partials(...) rows of dweight [C] then
// (with `dbias`, wanted with or without a bias) dbias [C].
struct GroupNormArgs {
  int64_t rows, xs, gs;  // strides of x and gate in elements
  int C, groups, W, act, center;
  bool dbias;
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
