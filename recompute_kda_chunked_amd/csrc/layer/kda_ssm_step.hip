// The selective scan's decoding form: one token after another from a state in
// HBM.
//
// Per (sequence, head), with the state S [N][P] in fp32:
//   S = a S + (dt B) x^T,  y = S^T C + D x,  a = exp(-exp(A_log) dt)
//
// What bounds it: the state's bytes, 8 N P read and written once per sequence
// and head whatever the number of tokens. Every column of S is independent, so
// a wave takes all N rows of 32 columns (a lane: 4 columns and every 8th group
// of 4 rows), the tile in registers over all tokens, and no wave waits for
// another. A lane reads the B and C of its own rows, which the heads of a group
// and the waves of a head find in the caches; the next token's rows are loaded
// during a token's step. States go past the caches as in the recurrent form of
// the delta rule: 193 sequences of one token, 64 heads, N 128, P 64, take 151 us
// (5.4 TB/s), 33 of up to 6 tokens with 48 heads 19.5. Sums and the state are fp32 for either dtype; only y is
// rounded, once.
#include "../kda_device.h"
#include "kda_rows.h"
#include "kda_ssm.h"

namespace kda {

namespace {

template <typename TI, int N, int P, bool MANY>
__global__ void __launch_bounds__(2 * P) k_ssm_recurrent(SsmStepArgs a) {
  constexpr int CW = 32, RS = 4 * 64 / (CW / 4), NJ = N / RS;
  const int n = blockIdx.x / a.H, h = blockIdx.x % a.H;
  if (n >= a.n_seqs) {
    const unsigned own = static_cast<unsigned>(a.n_seqs) * a.H;
    zero_rest(a.y, static_cast<size_t>(a.H) * P * sizeof(TI), a.cu, a.n_seqs, a.T, blockIdx.x - own, gridDim.x - own);
    return;
  }
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int64_t t0 = n, t1 = n + 1;
  if (a.cu) {
    t0 = a.cu[n];
    t1 = a.cu[n + 1];
    t0 = t0 < 0 ? 0 : (t0 > a.T ? a.T : t0);
    t1 = t1 > a.T ? a.T : t1;
  }
  if (t0 >= t1) return;
  const int64_t slot = find_slot<MANY>(a.idx, a.cu, a.T, n, a.n_slots);
  TI* y = static_cast<TI*>(a.y) + static_cast<size_t>(h) * P;
  const size_t os = static_cast<size_t>(a.H) * P;
  const int cg = lane % (CW / 4), rg = lane / (CW / 4);
  const int col = CW * w + 4 * cg;
  if (slot < 0) {  // padded: zeros; a slot it cannot have: NaN
    const float f = slot == kPadded ? 0.f : nan_value();
    if (rg == 0)
      for (int64_t t = t0; t < t1; ++t) store4<TI>(y + t * os + col, f32x4{f, f, f, f});
    return;
  }
  float A = -expf(a.A_log[h]);  // finite: a step of zero decays nothing
  A = A < -FLT_MAX ? -FLT_MAX : A;
  const float D = a.D ? a.D[h] : 0.f, bias = a.dt_bias ? a.dt_bias[h] : 0.f;
  const int g = h / (a.H / a.G);

  struct Token {
    uint32_t dt, x[4], B[NJ][4], C[NJ][4];
  };
  auto load = [&](int64_t t, Token& k) {
    k.dt = load_bits<TI>(static_cast<const TI*>(a.dt) + t * a.dts + h);
    load4_raw<TI>(static_cast<const TI*>(a.x) + t * a.xs + static_cast<size_t>(h) * P + col, k.x);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const size_t c = static_cast<size_t>(g) * N + RS * j + 4 * rg;
      load4_raw<TI>(static_cast<const TI*>(a.B) + t * a.Bs + c, k.B[j]);
      load4_raw<TI>(static_cast<const TI*>(a.C) + t * a.Cs + c, k.C[j]);
    }
  };
  Token next;
  load(t0, next);

  // rows RS j + 4 rg + r of the lane's four columns
  float* Sp = a.state + (static_cast<size_t>(slot) * a.H + h) * (N * P) + 4 * rg * P + col;
  f32x4 s[NJ][4];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) s[j][r] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(Sp + (RS * j + r) * P));

  for (int64_t t = t0; t < t1; ++t) {
    const Token k = next;
    if (t + 1 < t1) load(t + 1, next);
    const float dt = ssm_step(bits_to_f<TI>(k.dt) + bias, a.dt_min, a.dt_max), decay = expf(A * dt);
    const f32x4 x = unpack4<TI>(k.x), xd = dt * x;
    f32x4 o = zero4();
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const f32x4 b = unpack4<TI>(k.B[j]), c = unpack4<TI>(k.C[j]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s[j][r] = decay * s[j][r] + b[r] * xd;
        o += c[r] * s[j][r];
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = sum_row_groups(o[r]) + D * x[r];
    if (rg == 0) store4<TI>(y + t * os + col, o);
  }

#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) vstore<true>(reinterpret_cast<f32x4*>(Sp + (RS * j + r) * P), s[j][r]);
}

template <typename TI, int N, int P>
hipError_t launch_np(const SsmStepArgs& a, hipStream_t s) {
  const unsigned nh = static_cast<unsigned>(a.n_seqs) * static_cast<unsigned>(a.H);
  // blocks of 256 threads, below 2^32 in all
  const unsigned rest = rest_blocks(a.zero_rest, a.T * a.H * P * static_cast<int64_t>(sizeof(TI)), (1 << 24) - 1 - nh);
  if (a.idx && a.n_seqs > kScanAlone) k_ssm_recurrent<TI, N, P, true><<<nh + rest, 2 * P, 0, s>>>(a);
  else k_ssm_recurrent<TI, N, P, false><<<nh + rest, 2 * P, 0, s>>>(a);
  return hipGetLastError();
}
template <typename TI>
hipError_t launch_t(int N, int P, const SsmStepArgs& a, hipStream_t s) {
  if (N == 64) return P == 64 ? launch_np<TI, 64, 64>(a, s) : launch_np<TI, 64, 128>(a, s);
  return P == 64 ? launch_np<TI, 128, 64>(a, s) : launch_np<TI, 128, 128>(a, s);
}

}  // namespace

hipError_t launch_ssm_recurrent(int dtype, int N, int P, const SsmStepArgs& a, hipStream_t s) {
  return dtype == KDA_F32 ? launch_t<float>(N, P, a, s) : launch_t<bf16>(N, P, a, s);
}

}  // namespace kda
