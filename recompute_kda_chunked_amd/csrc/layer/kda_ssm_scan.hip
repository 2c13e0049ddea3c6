// The selective scan over packed sequences, forward and backward, in chunks of
// Q tokens of one sequence (128 for bf16, 64 for fp32).
//
// With cum_i the sum of the log decays of a chunk up to its token i, S the state
// entering the chunk, dS' the gradient of the one leaving it, L_ij =
// exp(cum_i - cum_j) for j <= i, G_ij = C_i . B_j, E_ij = dy_i . x_j:
//   y_i  = sum_j L_ij G_ij dt_j x_j + exp(cum_i) S^T C_i + D x_i
//   S'   = exp(cum_Q) S + sum_j exp(cum_Q - cum_j) dt_j B_j x_j^T
//   u_j  = sum_i L_ij G_ij dy_i + exp(cum_Q - cum_j) dS'^T B_j
//   dx_j = dt_j u_j + D dy_j,  d dt_j (as a factor) = x_j . u_j
//   dC_i = sum over heads of  sum_j L_ij E_ij dt_j B_j + exp(cum_i) S dy_i
//   dB_j = sum over heads of  dt_j (sum_i L_ij E_ij C_i + exp(cum_Q - cum_j) dS' x_j)
//   dS   = exp(cum_Q) dS' + sum_i exp(cum_i) C_i dy_i^T
// and of the log decay of token t, with F_ij = L_ij G_ij E_ij, Z = S dy, V = dS' x:
//   dl_t = sum_{i>=t} (sum_j F_ij dt_j - dt_i sum_k F_ki + exp(cum_i) C_i . Z_i)
//        + sum_{j<t} dt_j exp(cum_Q - cum_j) B_j . V_j + exp(cum_Q) <S, dS'>
// which differs only within a chunk, so that no sum over the sequence has to
// cancel.
//
// The states entering chunks come from one pass along each sequence and the
// gradients of those leaving them from one back (k_ssm_state, the state in
// accumulators, fp32), which leaves the rest to blocks that know nothing of each
// other: k_ssm_out and k_ssm_grad, a chunk each, the heads of a group in turn,
// so that C B^T is formed once for them and dB and dC add up in registers.
//
// Roundings of a bf16 problem: scores and states as operands of the products
// whose results are rounded to bf16 anyway; where fp32 outputs depend on them
// (the states themselves, dA_log, ddt_bias) a value is a pair of bf16, 16 bits.
// Running sums of log decays are fp64, kept as pairs of fp32.
#include "../kda_internal.h"
#include "kda.h"
#include "kda_rows.h"
#include "kda_ssm.h"
#include "kda_ssm_tile.h"

namespace kda {

namespace {

template <typename TI>
struct Chunk {
  static constexpr int Q = sizeof(TI) == 4 ? 64 : 128;
};

// A value that the compiler takes for a new one each time: what is computed
// from a lane's number is cheap, but kept in registers over a loop (some hundred
// addresses) it would spill the accumulators.
__device__ __forceinline__ int once(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// The wave's number in its block, known to be the same for its lanes.
__device__ __forceinline__ int wave_number() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

__device__ __forceinline__ int64_t clamp_cu(const SsmArgs& a, int n) {
  if (!a.cu) return n == 0 ? 0 : a.T;
  const int64_t c = a.cu[n];
  return c < 0 ? 0 : (c > a.T ? a.T : c);
}

// The chunk of a slot: its first token and its tokens (<= 0: none).
struct Place {
  int64_t t0;
  int rows;
};
template <int Q>
__device__ __forceinline__ Place find_chunk(const SsmArgs& a, int64_t slot) {
  if (a.n_seqs == 0) return {0, 0};
  int lo = 0, hi = a.n_seqs;  // the last sequence whose first slot is not behind
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (clamp_cu(a, mid) / Q + mid <= slot) lo = mid;
    else hi = mid;
  }
  const int64_t s = clamp_cu(a, lo), e = clamp_cu(a, lo + 1), pos = slot - (s / Q + lo);
  if (pos < 0) return {0, 0};
  const int64_t left = e - s - pos * Q;
  return {s + pos * Q, static_cast<int>(left < Q ? (left < 0 ? 0 : left) : Q)};
}

// ------------------------------------------------------------ step sizes

// One wave per (chunk, head), Q / 64 tokens a lane.
template <typename TI>
__global__ void __launch_bounds__(256) k_ssm_steps(SsmArgs a) {
  constexpr int Q = Chunk<TI>::Q, R = Q / 64;
  const int nhb = (a.H + 3) / 4;
  const int64_t slot = blockIdx.x / nhb;
  const int h = (blockIdx.x % nhb) * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  const Place c = find_chunk<Q>(a, slot);
  if (c.rows <= 0 || h >= a.H) return;
  const double l2 = -exp(static_cast<double>(a.A_log[h])) * 1.4426950408889634;
  const float bias = a.dt_bias ? a.dt_bias[h] : 0.f;
  float dt[R], slope[R];
  double cum[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int t = R * lane + r;
    dt[r] = slope[r] = 0.f;
    if (t < c.rows) {
      const float z = to_f(static_cast<const TI*>(a.dt)[(c.t0 + t) * a.dts + h]) + bias;
      dt[r] = ssm_step(z, a.dt_min, a.dt_max);
      if (!(dt[r] <= a.dt_min || dt[r] >= a.dt_max) || z != z) slope[r] = 1.f / (1.f + expf(-z));
    }
    cum[r] = l2 * dt[r] + (r ? cum[r - 1] : 0.0);
  }
  double tot = cum[R - 1];
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const double up = __shfl_up(tot, o, 64);
    if (lane >= o) tot += up;
  }
  double before = __shfl_up(tot, 1, 64);
  if (lane == 0) before = 0.0;
  f32x4* out = reinterpret_cast<f32x4*>(a.steps) + (slot * a.H + h) * Q + R * lane;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const double x = before + cum[r];
    const float hi = static_cast<float>(x);
    out[r] = f32x4{dt[r], hi, static_cast<float>(x - hi), slope[r]};
  }
}

// ------------------------------------------------------------ states

template <typename T>
__device__ __forceinline__ float low_part(float x) {
  return x - static_cast<float>(static_cast<T>(x));
}

// One block walks a sequence's chunks with 64 columns and 32 rows of one
// head's state: S' = e^tot S + (w B)^T x, w_j = dt_j exp(cum_Q - cum_j); reverse,
// dS = e^tot dS' + (w C)^T dy, w_i = exp(cum_i). The weighted rows are a pair of
// bf16, x and dy are exact. Wave w holds columns 16 w .. of the transposed
// state, a lane four of them in a row of it.
template <typename TI, int N, bool REV, bool LO>
__global__ void __launch_bounds__(256) k_ssm_state(SsmArgs a) {
  constexpr int Q = Chunk<TI>::Q, U = 16 / sizeof(TI), NB = 32;
  constexpr int XU = Q * 64 / U / 256, BU = Q * NB / U / 256;  // 16-byte units a thread
  constexpr bool kPair = sizeof(TI) == 2;
  __shared__ __align__(16) TI xs[Q * 64], bh[Q * NB], bl[kPair ? Q * NB : 1];
  const int halves = a.P / 64, nsplit = N / NB;
  const int per_seq = a.H * halves * nsplit;
  const int n = blockIdx.x / per_seq, rest = blockIdx.x % per_seq;
  const int n0 = (rest % nsplit) * NB, hp = rest / nsplit, h = hp / halves, half = hp % halves;
  const int grp = h / (a.H / a.G);
  const int tid = threadIdx.x, lane = tid & 63, w = wave_number(), i = lane & 15, g = lane >> 4;
  const int64_t s0 = clamp_cu(a, n), s1 = clamp_cu(a, n + 1), len = s1 > s0 ? s1 - s0 : 0;
  const int64_t nch = (len + Q - 1) / Q, first = s0 / Q + n;
  const TI* src = static_cast<const TI*>(REV ? a.dy : a.x) + static_cast<size_t>(h) * a.P + half * 64;
  const int64_t sst = REV ? static_cast<int64_t>(a.H) * a.P : a.xs;
  const TI* rsrc = static_cast<const TI*>(REV ? a.C : a.B) + static_cast<size_t>(grp) * N + n0;
  const int64_t rst = REV ? a.Cs : a.Bs;
  const float* from = REV ? a.dfinal : a.init;
  float* to = REV ? a.dinit : a.final_state;
  const size_t state = ((static_cast<size_t>(n) * a.H + h) * N + n0 + i) * a.P + half * 64 + 16 * w + 4 * g;

  const LaneAt<TI, 64> lx(lane);
  const LaneAt<TI, NB> lb(lane);
  f32x4 acc[2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
    acc[t] = from ? *reinterpret_cast<const f32x4*>(from + state + static_cast<size_t>(16 * t) * a.P) : zero4();

  uint4 rx[XU], rb[BU];
  float wt[BU], tot = 0.f;
  auto load = [&](int64_t c) {
    const int64_t t0 = s0 + c * Q;
    const int rows = static_cast<int>(s1 - t0 < Q ? s1 - t0 : Q);
#pragma unroll
    for (int m = 0; m < XU; ++m) {
      const int u = tid + 256 * m, r = u / (64 / U);
      rx[m] = make_uint4(0, 0, 0, 0);
      if (r < rows) rx[m] = *reinterpret_cast<const uint4*>(src + (t0 + r) * sst + (u % (64 / U)) * U);
    }
    const f32x4* st = reinterpret_cast<const f32x4*>(a.steps) + ((first + c) * a.H + h) * Q;
    const f32x4 end = st[Q - 1];
    tot = exp2_(end[1] + end[2]);
#pragma unroll
    for (int m = 0; m < BU; ++m) {
      const int u = tid + 256 * m, r = u / (NB / U);
      rb[m] = make_uint4(0, 0, 0, 0);
      if (r < rows) rb[m] = *reinterpret_cast<const uint4*>(rsrc + (t0 + r) * rst + (u % (NB / U)) * U);
      const f32x4 k = st[r];
      wt[m] = REV ? exp2_(k[1] + k[2]) : k[0] * exp2_((end[1] - k[1]) + (end[2] - k[2]));
    }
  };
  if (nch > 0) load(REV ? nch - 1 : 0);
  for (int64_t k = 0; k < nch; ++k) {
    const int64_t c = REV ? nch - 1 - k : k;
    __syncthreads();
#pragma unroll
    for (int m = 0; m < XU; ++m) {
      const int u = tid + 256 * m;
      *reinterpret_cast<uint4*>(xs + tile_at<TI, 64>(u / (64 / U), (u % (64 / U)) * U)) = rx[m];
    }
#pragma unroll
    for (int m = 0; m < BU; ++m) {
      const int u = tid + 256 * m, at = tile_at<TI, NB>(u / (NB / U), (u % (NB / U)) * U);
      RowVec<TI> v, lo;
      float f[U], l[U];
      v.u = rb[m];
      v.get(f);
#pragma unroll
      for (int e = 0; e < U; ++e) {
        f[e] *= wt[m];
        l[e] = low_part<TI>(f[e]);
      }
      v.set(f);
      *reinterpret_cast<uint4*>(bh + at) = v.u;
      if constexpr (kPair) {
        lo.set(l);
        *reinterpret_cast<uint4*>(bl + at) = lo.u;
      }
    }
    const float decay = tot;
    __syncthreads();
    if (k + 1 < nch) load(REV ? c - 1 : c + 1);
    TI* out = static_cast<TI*>(REV ? a.dS : a.S) + (((first + c) * a.H * halves + hp) * N + n0 + i) * 64 + 16 * w + 4 * g;
    TI* out_lo = LO ? static_cast<TI*>(REV ? a.dS_lo : a.S_lo) + (((first + c) * a.H * halves + hp) * N + n0 + i) * 64 + 16 * w + 4 * g : nullptr;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      store4<TI>(out + 16 * t * 64, acc[t]);
      if constexpr (LO) {
        f32x4 l;
#pragma unroll
        for (int r = 0; r < 4; ++r) l[r] = low_part<TI>(acc[t][r]);
        store4<TI>(out_lo + 16 * t * 64, l);
      }
      acc[t] *= decay;
    }
#pragma unroll
    for (int k0 = 0; k0 < Q; k0 += 32) {
      const Frag<TI> ax = frag_col<false>(xs, lx, k0, 16 * w);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        acc[t] = mma32(ax, frag_col<false>(bh, lb, k0, 16 * t), acc[t]);
        if constexpr (kPair) acc[t] = mma32(ax, frag_col<false>(bl, lb, k0, 16 * t), acc[t]);
      }
    }
  }
  if (to) {
#pragma unroll
    for (int t = 0; t < 2; ++t) *reinterpret_cast<f32x4*>(to + state + static_cast<size_t>(16 * t) * a.P) = acc[t];
  }
}

// ------------------------------------------------------------ shared by out and grad

// A wave's tile of 16 tokens: those of wave w and w + NW / 2, which share a
// SIMD, are as far from the diagonal's ends as each other, so that every SIMD
// has the same number of score tiles.
template <int NW>
__device__ __forceinline__ int own_tile(int w) {
  return w < NW / 2 ? w : NW - 1 - (w - NW / 2);
}

// COLS columns of `rows` rows `st` apart to a tile of Q rows (zeros behind).
template <typename TI, int R, int COLS, int THREADS>
__device__ __forceinline__ void load_tile(TI* tile, const TI* src, int64_t st, int rows) {
  constexpr int U = 16 / sizeof(TI), PER = R * COLS / U / THREADS;
  const int tid = once(threadIdx.x);
  uint4 v[PER];
#pragma unroll
  for (int m = 0; m < PER; ++m) {
    const int u = tid + THREADS * m, r = u / (COLS / U);
    v[m] = make_uint4(0, 0, 0, 0);
    if (r < rows) v[m] = *reinterpret_cast<const uint4*>(src + r * st + (u % (COLS / U)) * U);
  }
#pragma unroll
  for (int m = 0; m < PER; ++m) {
    const int u = tid + THREADS * m;
    *reinterpret_cast<uint4*>(tile + tile_at<TI, COLS>(u / (COLS / U), (u % (COLS / U)) * U)) = v[m];
  }
}

// Zeroes `width` elements of each row that belongs to no sequence.
template <typename T>
__device__ __forceinline__ void zero_rows(T* o, int64_t width, const SsmArgs& a, unsigned b, unsigned nb) {
  const int64_t before = clamp_cu(a, 0), end = clamp_cu(a, a.n_seqs), behind = end < before ? before : end;
  const int64_t step = static_cast<int64_t>(nb) * blockDim.x, at = static_cast<int64_t>(b) * blockDim.x + threadIdx.x;
  for (int64_t i = at; i < before * width; i += step) o[i] = static_cast<T>(0.f);
  for (int64_t i = behind * width + at; i < a.T * width; i += step) o[i] = static_cast<T>(0.f);
}

// ------------------------------------------------------------ output

// Wave: 16 tokens i of the chunk. Scores are formed as [j][i] accumulators, an
// operand as they stand of y^T[p][i] = sum_j x_j[p] (L G dt)_ij.
template <typename TI, int N>
__global__ void __launch_bounds__(4 * Chunk<TI>::Q) k_ssm_out(SsmArgs a) {
  constexpr int Q = Chunk<TI>::Q, NW = Q / 16, TH = 64 * NW;
  __shared__ __align__(16) TI buf[2 * Q * N];
  __shared__ float chi[Q], clo[Q], cdt[Q];
  const unsigned own = static_cast<unsigned>(a.slots) * a.G * a.sets;
  if (blockIdx.x >= own) {
    zero_rows(static_cast<TI*>(a.y), static_cast<int64_t>(a.H) * a.P, a, blockIdx.x - own, gridDim.x - own);
    return;
  }
  const int set = blockIdx.x % a.sets, grp = (blockIdx.x / a.sets) % a.G;
  const int64_t slot = blockIdx.x / (a.sets * a.G);
  const Place c = find_chunk<Q>(a, slot);
  if (c.rows <= 0) return;
  const int tid = threadIdx.x, lane = tid & 63, w = wave_number(), i = lane & 15, g = lane >> 4;
  const int it = own_tile<NW>(w), per = a.H / a.G, halves = a.P / 64;
  const int h0 = grp * per + set * a.hb, h1 = set * a.hb + a.hb < per ? h0 + a.hb : (grp + 1) * per;

  const LaneAt<TI, N> ln(lane);
  const LaneAt<TI, 64> lx(lane);
  TI *Bt = buf, *Ct = buf + Q * N;
  load_tile<TI, Q, N, TH>(Bt, static_cast<const TI*>(a.B) + c.t0 * a.Bs + static_cast<size_t>(grp) * N, a.Bs, c.rows);
  load_tile<TI, Q, N, TH>(Ct, static_cast<const TI*>(a.C) + c.t0 * a.Cs + static_cast<size_t>(grp) * N, a.Cs, c.rows);
  __syncthreads();
  Frag<TI> cf[N / 32];
#pragma unroll
  for (int k = 0; k < N / 32; ++k) cf[k] = frag_row(Ct, ln, 16 * it, 32 * k);
  f32x4 G[NW];
#pragma unroll
  for (int jt = 0; jt < NW; ++jt) {
    G[jt] = zero4();
    if (jt <= it) {
#pragma unroll
      for (int k = 0; k < N / 32; ++k) G[jt] = mma32(frag_row(Bt, ln, 16 * jt, 32 * k), cf[k], G[jt]);
    }
  }
  TI *xs = buf, *Ss = buf + Q * 64;
  for (int h = h0; h < h1; ++h) {
    const float D = a.D ? a.D[h] : 0.f;
    for (int half = 0; half < halves; ++half) {
      __syncthreads();
      load_tile<TI, Q, 64, TH>(xs, static_cast<const TI*>(a.x) + c.t0 * a.xs + static_cast<size_t>(h) * a.P + half * 64, a.xs, c.rows);
      load_tile<TI, N, 64, TH>(Ss, static_cast<const TI*>(a.S) + ((slot * a.H + h) * halves + half) * N * 64, 64, N);
      if (tid < Q) {
        const f32x4 k = reinterpret_cast<const f32x4*>(a.steps)[(slot * a.H + h) * Q + tid];
        cdt[tid] = k[0];
        chi[tid] = k[1];
        clo[tid] = k[2];
      }
      __syncthreads();
      const float hi = chi[16 * it + i], lo = clo[16 * it + i], ei = exp2_(hi + lo);
      f32x4 y[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        y[p] = zero4();
#pragma unroll
        for (int k = 0; k < N / 32; ++k) y[p] = mma32(frag_col<false>(Ss, lx, 32 * k, 16 * p), cf[k], y[p]);
        y[p] *= ei;
      }
#pragma unroll
      for (int m = 0; m < NW / 2; ++m) {
        if (2 * m > it) continue;
        f32x4 W[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int j0 = 16 * (2 * m + q) + 4 * g;
          const f32x4 h4 = *reinterpret_cast<const f32x4*>(chi + j0), l4 = *reinterpret_cast<const f32x4*>(clo + j0);
          const f32x4 d4 = *reinterpret_cast<const f32x4*>(cdt + j0);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            W[q][r] = j0 + r <= 16 * it + i ? G[2 * m + q][r] * exp2_((hi - h4[r]) + (lo - l4[r])) * d4[r] : 0.f;
        }
        const Frag<TI> wf = pair_frag<TI>(W[0], W[1]);
#pragma unroll
        for (int p = 0; p < 4; ++p) y[p] = mma32(frag_col<true>(xs, lx, 32 * m, 16 * p), wf, y[p]);
      }
      const int row = 16 * it + i;
      if (row < c.rows) {
        TI* out = static_cast<TI*>(a.y) + ((c.t0 + row) * a.H + h) * a.P + half * 64 + 4 * g;
#pragma unroll
        for (int p = 0; p < 4; ++p) store4<TI>(out + 16 * p, y[p] + D * tile_get4(xs, lx, 16 * it, 16 * p));
      }
    }
  }
}

// ------------------------------------------------------------ gradients

// Sum over the four lane groups (lanes i, i + 16, i + 32, i + 48), every lane
// receiving it.
__device__ __forceinline__ float sum_lane_groups(float x) {
  const uint32_t b = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  const uint32_t c = __float_as_uint(x);
  const auto h = __builtin_amdgcn_permlane32_swap(c, c, false, false);
  return __uint_as_float(h[0]) + __uint_as_float(h[1]);
}

// Two roles of a wave. First, 16 tokens j of the chunk: the scores of all i >= j
// as [i][j] accumulators, dx_j, and L E dt to LDS. Then 16 rows of the state (or
// several, or half the tokens; NT tiles of rows and TT of tokens), in which dB
// and dC add up over the heads, transposed: [n][token].
template <typename TI, int N>
struct GradShape {
  static constexpr int Q = Chunk<TI>::Q, NW = Q / 16, RT = N / 16;
  static constexpr int NT = RT > NW ? RT / NW : 1;         // row tiles a wave
  static constexpr int NG = RT / NT;                       // groups of row tiles
  static constexpr int TT = NW / (NW / NG);                // token tiles a wave
};

template <typename TI, int N>
__global__ void __launch_bounds__(4 * Chunk<TI>::Q) k_ssm_grad(SsmArgs a) {
  using SH = GradShape<TI, N>;
  constexpr int Q = SH::Q, NW = SH::NW, TH = 64 * NW, NT = SH::NT, NG = SH::NG, TT = SH::TT;
  constexpr bool kPair = sizeof(TI) == 2;
  __shared__ __align__(16) TI Bt[Q * N], Ct[Q * N], xs[Q * 64], dys[Q * 64], MT[Q * Q], Gs[N * 64];
  __shared__ __align__(16) float chi[2][Q], clo[2][Q], cdt[2][Q], rowF[NW][Q], iC[NG][Q], iB[NG][Q], colF[Q];
  __shared__ float sd[NW], xd[NW];
  const unsigned own = static_cast<unsigned>(a.slots) * a.G * a.sets;
  if (blockIdx.x >= own) {
    const unsigned b = blockIdx.x - own, nb = gridDim.x - own;
    zero_rows(static_cast<TI*>(a.dx), static_cast<int64_t>(a.H) * a.P, a, b, nb);
    zero_rows(static_cast<TI*>(a.ddt), a.H, a, b, nb);
    if (a.sets == 1) {
      zero_rows(static_cast<TI*>(a.dB), static_cast<int64_t>(a.G) * N, a, b, nb);
      zero_rows(static_cast<TI*>(a.dC), static_cast<int64_t>(a.G) * N, a, b, nb);
    }
    return;
  }
  const int set = blockIdx.x % a.sets, grp = (blockIdx.x / a.sets) % a.G;
  const int64_t slot = blockIdx.x / (a.sets * a.G);
  const Place c = find_chunk<Q>(a, slot);
  const int tid = threadIdx.x, lane = tid & 63, w = wave_number(), i = lane & 15, g = lane >> 4;
  const int jt = own_tile<NW>(w), per = a.H / a.G, halves = a.P / 64;
  const int h0 = grp * per + set * a.hb, h1 = set * a.hb + a.hb < per ? h0 + a.hb : (grp + 1) * per;
  if (c.rows <= 0) {  // its partial sums are added up all the same
    for (int h = h0 + tid; h < h1; h += TH) {
      a.part2[slot * 2 * a.H + h] = a.part2[slot * 2 * a.H + a.H + h] = 0.f;
      a.part1[slot * a.H + h] = 0.f;
    }
    return;
  }
  load_tile<TI, Q, N, TH>(Bt, static_cast<const TI*>(a.B) + c.t0 * a.Bs + static_cast<size_t>(grp) * N, a.Bs, c.rows);
  load_tile<TI, Q, N, TH>(Ct, static_cast<const TI*>(a.C) + c.t0 * a.Cs + static_cast<size_t>(grp) * N, a.Cs, c.rows);
  __syncthreads();
  // of the first role: rows of B, and C B^T
  Frag<TI> bf[N / 32];
  f32x4 G[NW];
  const LaneAt<TI, N> ln(lane);
#pragma unroll
  for (int k = 0; k < N / 32; ++k) bf[k] = frag_row(Bt, ln, 16 * jt, 32 * k);
#pragma unroll
  for (int t = 0; t < NW; ++t) {
    G[t] = zero4();
    if (t >= jt) {
#pragma unroll
      for (int k = 0; k < N / 32; ++k) G[t] = mma32(frag_row(Ct, ln, 16 * t, 32 * k), bf[k], G[t]);
    }
  }
  // of the second: tokens t0 16 .., rows n0 .. of B^T and C^T
  const int ng = w % NG, tt0 = (w / NG) * TT, n0 = ng * NT * 16;
  f32x4 dC[NT][TT], dB[NT][TT];
#pragma unroll
  for (int u = 0; u < NT; ++u)
#pragma unroll
    for (int t = 0; t < TT; ++t) dC[u][t] = dB[u][t] = zero4();

  int par = 0;
  for (int h = h0; h < h1; ++h) {
    const float D = a.D ? a.D[h] : 0.f;
    for (int half = 0; half < halves; ++half, par ^= 1) {
      load_tile<TI, Q, 64, TH>(xs, static_cast<const TI*>(a.x) + c.t0 * a.xs + static_cast<size_t>(h) * a.P + half * 64, a.xs, c.rows);
      load_tile<TI, Q, 64, TH>(dys, static_cast<const TI*>(a.dy) + (c.t0 * a.H + h) * a.P + half * 64, static_cast<int64_t>(a.H) * a.P, c.rows);
      const size_t sat = ((slot * a.H + h) * halves + half) * static_cast<size_t>(N) * 64;
      load_tile<TI, N, 64, TH>(Gs, static_cast<const TI*>(a.dS) + sat, 64, N);
      if (tid < Q) {
        const f32x4 k = reinterpret_cast<const f32x4*>(a.steps)[(slot * a.H + h) * Q + tid];
        cdt[par][tid] = k[0];
        chi[par][tid] = k[1];
        clo[par][tid] = k[2];
      }
      __syncthreads();
      const int fresh = once(lane);
      const LaneAt<TI, N> ln(fresh);
      const LaneAt<TI, 64> lx(fresh);
      const LaneAt<TI, Q> lq(fresh);
      const float *hiv = chi[par], *lov = clo[par], *dtv = cdt[par];
      const float hQ = hiv[Q - 1], lQ = lov[Q - 1];

      {  // first role
        const int row = 16 * jt + i;
        const float hj = hiv[row], lj = lov[row], dtj = dtv[row], rj = exp2_((hQ - hj) + (lQ - lj));
        Frag<TI> xf[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) xf[k] = frag_row(xs, lx, 16 * jt, 32 * k);
        f32x4 dx[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          dx[p] = zero4();
#pragma unroll
          for (int k = 0; k < N / 32; ++k) dx[p] = mma32(frag_col<false>(Gs, lx, 32 * k, 16 * p), bf[k], dx[p]);
          dx[p] *= rj;
        }
        float cf = 0.f, diag = 0.f;
#pragma unroll
        for (int m = 0; m < NW / 2; ++m) {
          if (2 * m + 1 < jt) continue;
          f32x4 W[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int t = 2 * m + q, i0 = 16 * t + 4 * g;
            W[q] = zero4();
            f32x4 M = zero4();
            if (t >= jt) {
              f32x4 e = zero4(), f;
#pragma unroll
              for (int k = 0; k < 2; ++k) e = mma32(frag_row(dys, lx, 16 * t, 32 * k), xf[k], e);
              const f32x4 h4 = *reinterpret_cast<const f32x4*>(hiv + i0), l4 = *reinterpret_cast<const f32x4*>(lov + i0);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float L = i0 + r >= row ? exp2_((h4[r] - hj) + (l4[r] - lj)) : 0.f;
                if (i0 + r == row) diag += e[r];
                W[q][r] = L * G[t][r];
                M[r] = L * e[r] * dtj;
                const float F = W[q][r] * e[r];
                cf += F;
                f[r] = F * dtj;
              }
              const float v[4] = {f[0], f[1], f[2], f[3]};
              const float s = transpose_sum16<4>(v);  // lane i: of f[i % 4]
              if (i < 4) rowF[w][i0 + i] = s;
            }
            store4<TI>(MT + shifted<LaneAt<TI, Q>>(lq.four, 16 * t) + 16 * jt * Q, M);
          }
          const Frag<TI> wf = pair_frag<TI>(W[0], W[1]);
#pragma unroll
          for (int p = 0; p < 4; ++p) dx[p] = mma32(frag_col<true>(dys, lx, 32 * m, 16 * p), wf, dx[p]);
          __builtin_amdgcn_sched_barrier(0);
        }
        cf = sum_lane_groups(cf);
        if (g == 0) colF[row] = cf;
        diag = sum_wave(diag);
        if (lane == 0) xd[w] = diag;
        if (row < c.rows) {
          TI* out = static_cast<TI*>(a.dx) + ((c.t0 + row) * a.H + h) * a.P + half * 64 + 4 * g;
#pragma unroll
          for (int p = 0; p < 4; ++p) store4<TI>(out + 16 * p, dtj * dx[p] + D * tile_get4(dys, lx, 16 * jt, 16 * p));
        }
      }
      __syncthreads();

      {  // second role
        float dot = 0.f;
        Frag<TI> sf[NT][2], sl[NT][2], gf[NT][2], gl[NT][2];
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int nr = n0 + 16 * u;
            sf[u][k] = frag_mem(static_cast<const TI*>(a.S) + sat, nr, 32 * k, 64, fresh);
            gf[u][k] = frag_mem(static_cast<const TI*>(a.dS) + sat, nr, 32 * k, 64, fresh);
            if constexpr (kPair) {
              sl[u][k] = frag_mem(static_cast<const TI*>(a.S_lo) + sat, nr, 32 * k, 64, fresh);
              gl[u][k] = frag_mem(static_cast<const TI*>(a.dS_lo) + sat, nr, 32 * k, 64, fresh);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              if constexpr (kPair) dot += (to_f(sf[u][k][e]) + to_f(sl[u][k][e])) * (to_f(gf[u][k][e]) + to_f(gl[u][k][e]));
              else dot += sf[u][k][e] * gf[u][k][e];
            }
          }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const int tt = tt0 + t, row = 16 * tt + i;
          const float ei = exp2_(hiv[row] + lov[row]), rj = exp2_((hQ - hiv[row]) + (lQ - lov[row])), dtj = dtv[row];
          float ic = 0.f, ib = 0.f;
#pragma unroll
          for (int u = 0; u < NT; ++u) {
            const int nr = n0 + 16 * u;
            f32x4 z = zero4(), v = zero4();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const Frag<TI> yf = frag_row(dys, lx, 16 * tt, 32 * k), xf = frag_row(xs, lx, 16 * tt, 32 * k);
              z = mma32(sf[u][k], yf, z);
              v = mma32(gf[u][k], xf, v);
              if constexpr (kPair) {
                z = mma32(sl[u][k], yf, z);
                v = mma32(gl[u][k], xf, v);
              }
            }
            z *= ei;
            v *= rj;
            const f32x4 c4 = tile_get4(Ct, ln, 16 * tt, nr), b4 = tile_get4(Bt, ln, 16 * tt, nr);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              ic += c4[r] * z[r];
              ib += b4[r] * v[r];
            }
            dC[u][t] += z;
            dB[u][t] += dtj * v;
#pragma unroll
            for (int m = 0; m < NW / 2; ++m) {
              if (2 * m <= tt) dC[u][t] = mma32(frag_col<false>(Bt, ln, 32 * m, nr), frag_col<false>(MT, lq, 32 * m, 16 * tt), dC[u][t]);
              if (2 * m + 1 >= tt) dB[u][t] = mma32(frag_col<false>(Ct, ln, 32 * m, nr), frag_row(MT, lq, 16 * tt, 32 * m), dB[u][t]);
            }
          }
          ic = sum_lane_groups(ic);
          ib = sum_lane_groups(ib);
          if (g == 0) {
            iC[ng][row] = ic;
            iB[ng][row] = ib;
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        dot = sum_wave(dot);
        if (lane == 0) sd[w] = tt0 == 0 ? dot : 0.f;  // waves of the same rows have the same
      }
      __syncthreads();

      if (w == 0) {  // the scalars of the head, R tokens a lane
        constexpr int R = Q / 64;
        const int t0 = R * once(lane);
        float dots = 0.f, diag = 0.f, own[R], col[R], before[R], direct[R];
#pragma unroll
        for (int r = 0; r < R; ++r) own[r] = before[r] = 0.f;
#pragma unroll 1
        for (int k = 0; k < NW; ++k) {
          dots += sd[k];
          diag += xd[k];
          if (t0 / 16 >= own_tile<NW>(k))
#pragma unroll
            for (int r = 0; r < R; ++r) own[r] += rowF[k][t0 + r];
        }
#pragma unroll 1
        for (int k = 0; k < NG; ++k)
#pragma unroll
          for (int r = 0; r < R; ++r) {
            own[r] += iC[k][t0 + r];
            before[r] += iB[k][t0 + r];
          }
        // dl_t: own over the tokens from t on, before over those before it
        float sa = 0.f, sb = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          col[r] = colF[t0 + r];
          direct[r] = col[r] + before[r];
          own[r] -= dtv[t0 + r] * col[r];
          before[r] *= dtv[t0 + r];
          sa += own[r];
          sb += before[r];
        }
        const float lb = sb;
#pragma unroll
        for (int o = 1; o < 64; o *= 2) {
          const float da = __shfl_down(sa, o, 64), ub = __shfl_up(sb, o, 64);
          if (lane + o < 64) sa += da;
          if (lane >= o) sb += ub;
        }
        sb += exp2_(hQ + lQ) * dots - lb;
        const float Ah = expf(a.A_log[h]);
        const size_t at = (slot * a.H + h) * Q + t0;
        float dA = 0.f, db = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float dl = sa + sb;
          sa -= own[r];
          sb += before[r];
          float d = (direct[r] - Ah * dl) * a.steps[4 * (at + r) + 3];
          dA -= Ah * dtv[t0 + r] * dl;
          db += d;
          if (halves > 1) {  // of two halves of a head the second adds to the first's
            if (half) d += a.ddt_half[at + r];
            else a.ddt_half[at + r] = d;
          }
          if (t0 + r < c.rows && half == halves - 1) static_cast<TI*>(a.ddt)[(c.t0 + t0 + r) * a.H + h] = from_f<TI>(d);
        }
        dA = sum_wave(dA);
        db = sum_wave(db);
        if (lane == 0) {
          float *p2 = a.part2 + slot * 2 * a.H + h, *p1 = a.part1 + slot * a.H + h;
          *p2 = half ? *p2 + dA : dA;
          p2[a.H] = half ? p2[a.H] + db : db;
          *p1 = half ? *p1 + diag : diag;
        }
      }
    }
  }
  // dB and dC of the heads: to the outputs, or to this set's partial sums
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int row = 16 * (tt0 + t) + i;
    if (row >= c.rows) continue;
    const size_t at = ((c.t0 + row) * a.G + grp) * N + n0 + 4 * g;
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      if (a.sets == 1) {
        store4<TI>(static_cast<TI*>(a.dB) + at + 16 * u, dB[u][t]);
        store4<TI>(static_cast<TI*>(a.dC) + at + 16 * u, dC[u][t]);
      } else {
        const size_t far = static_cast<size_t>(set) * a.T * a.G * N;
        store4<float>(a.pB + far + at + 16 * u, dB[u][t]);
        store4<float>(a.pC + far + at + 16 * u, dC[u][t]);
      }
    }
  }
}

// Sums of dB and dC over the sets of heads.
template <typename TI>
__global__ void __launch_bounds__(256) k_ssm_reduce(SsmArgs a, int64_t width) {
  const int64_t before = clamp_cu(a, 0) * width, end = clamp_cu(a, a.n_seqs) * width, all = a.T * width;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256 * 4;
  for (int64_t e = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; e < all; e += step) {
    f32x4 b = zero4(), c = zero4();
    if (e >= before && e < end) {
      for (int s = 0; s < a.sets; ++s) {
        b += *reinterpret_cast<const f32x4*>(a.pB + s * all + e);
        c += *reinterpret_cast<const f32x4*>(a.pC + s * all + e);
      }
    }
    store4<TI>(static_cast<TI*>(a.dB) + e, b);
    store4<TI>(static_cast<TI*>(a.dC) + e, c);
  }
}

unsigned out_rest(const SsmArgs& a, int64_t bytes) {
  return a.cu ? rest_blocks(true, bytes, 1024) : 0;
}

template <typename TI, int N>
hipError_t launch_state_n(bool reverse, const SsmArgs& a, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.n_seqs) * a.H * (a.P / 64) * (N / 32);
  const bool lo = sizeof(TI) == 2 && (reverse || a.S_lo);
  if (reverse) {
    if (lo) k_ssm_state<TI, N, true, true><<<grid, 256, 0, s>>>(a);
    else k_ssm_state<TI, N, true, false><<<grid, 256, 0, s>>>(a);
  } else {
    if (lo) k_ssm_state<TI, N, false, true><<<grid, 256, 0, s>>>(a);
    else k_ssm_state<TI, N, false, false><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}
template <typename TI, int N>
hipError_t launch_out_n(const SsmArgs& a, hipStream_t s) {
  const unsigned own = static_cast<unsigned>(a.slots) * a.G * a.sets;
  k_ssm_out<TI, N><<<own + out_rest(a, a.T * a.H * a.P * static_cast<int64_t>(sizeof(TI))), 4 * Chunk<TI>::Q, 0, s>>>(a);
  return hipGetLastError();
}
template <typename TI, int N>
hipError_t launch_grad_n(const SsmArgs& a, hipStream_t s) {
  const unsigned own = static_cast<unsigned>(a.slots) * a.G * a.sets;
  k_ssm_grad<TI, N><<<own + out_rest(a, a.T * a.H * a.P * static_cast<int64_t>(sizeof(TI))), 4 * Chunk<TI>::Q, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ssm_steps(int dtype, const SsmArgs& a, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.slots) * ((a.H + 3) / 4);
  if (dtype == KDA_F32) k_ssm_steps<float><<<grid, 256, 0, s>>>(a);
  else k_ssm_steps<bf16><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}
hipError_t launch_ssm_state(int dtype, int N, bool reverse, const SsmArgs& a, hipStream_t s) {
  if (dtype == KDA_F32) return N == 64 ? launch_state_n<float, 64>(reverse, a, s) : launch_state_n<float, 128>(reverse, a, s);
  return N == 64 ? launch_state_n<bf16, 64>(reverse, a, s) : launch_state_n<bf16, 128>(reverse, a, s);
}
hipError_t launch_ssm_out(int dtype, int N, const SsmArgs& a, hipStream_t s) {
  if (dtype == KDA_F32) return N == 64 ? launch_out_n<float, 64>(a, s) : launch_out_n<float, 128>(a, s);
  return N == 64 ? launch_out_n<bf16, 64>(a, s) : launch_out_n<bf16, 128>(a, s);
}
hipError_t launch_ssm_grad(int dtype, int N, const SsmArgs& a, hipStream_t s) {
  if (dtype == KDA_F32) return N == 64 ? launch_grad_n<float, 64>(a, s) : launch_grad_n<float, 128>(a, s);
  return N == 64 ? launch_grad_n<bf16, 64>(a, s) : launch_grad_n<bf16, 128>(a, s);
}
hipError_t launch_ssm_reduce(int dtype, int N, const SsmArgs& a, hipStream_t s) {
  const int64_t width = static_cast<int64_t>(a.G) * N, want = (a.T * width + 1023) / 1024;
  const unsigned grid = static_cast<unsigned>(want < 8192 ? want : 8192);
  if (dtype == KDA_F32) k_ssm_reduce<float><<<grid, 256, 0, s>>>(a, width);
  else k_ssm_reduce<bf16><<<grid, 256, 0, s>>>(a, width);
  return hipGetLastError();
}

}  // namespace kda
