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
// (the states themselves, dA_log, ddt_bias) a value is three bf16, its 24 bits.
// Running sums of log decays are fp64, kept as pairs of fp32.
//
// What bounds it, at 8192 tokens in three sequences, 64 heads of 8 groups, N 128,
// P 64, bf16, forward and backward: nothing at its full rate (350 MB at the least
// are 68 us, the products' 52 GFLOP 46 us at the rate of a large product). Of 584
// us the state passes take 64 + 45 forward (as segments, see k_ssm_state) and 180
// backward, a chunk's step a chain of loads, LDS writes, LDS reads and products
// that 1.4 waves a SIMD cannot hide (3.3 us alone), and 270 MB of states go to HBM
// and come back. The gradient kernel takes 222: one block of 8 waves a CU by its LDS, vector
// instructions issued about half of the time (counters), the LDS in use a third and
// the matrix cores a fifth, one after another between barriers. The output
// takes 64, two blocks a CU. Chunks of 128 and not 64 tokens halve the states'
// bytes and the steps of the chain; fp32 tiles of 128 would not fit the LDS.
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

// The piece of L tokens of one sequence that a slot holds (see SsmArgs): the
// sequence (-1: none), its first token and end, the piece's number in it, and its
// tokens (<= 0: none).
struct Place {
  int n, pos, rows;
  int64_t s0, s1, t0;
};
__device__ __forceinline__ Place find_piece(const SsmArgs& a, int64_t slot, uint32_t L) {
  if (a.n_seqs == 0) return {-1, 0, 0, 0, 0, 0};
  auto first = [&](int n) { return static_cast<int64_t>(static_cast<uint32_t>(clamp_cu(a, n)) / L) + n; };
  int lo = 0, hi = a.n_seqs;  // the last sequence whose first slot is not behind
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first(mid) <= slot) lo = mid;
    else hi = mid;
  }
  const int64_t s = clamp_cu(a, lo), e = clamp_cu(a, lo + 1), pos = slot - first(lo);
  if (pos < 0) return {-1, 0, 0, 0, 0, 0};
  const int64_t left = e - s - pos * L;
  return {lo, static_cast<int>(pos), static_cast<int>(left < L ? (left < 0 ? 0 : left) : L), s, e, s + pos * L};
}

// ------------------------------------------------------------ step sizes

// One wave per (chunk, head), Q / 64 tokens a lane.
template <typename TI>
__global__ void __launch_bounds__(256) k_ssm_steps(SsmArgs a) {
  constexpr int Q = Chunk<TI>::Q, R = Q / 64;
  const int nhb = (a.H + 3) / 4;
  const int64_t slot = blockIdx.x / nhb;
  const int h = (blockIdx.x % nhb) * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  const Place c = find_piece(a, slot, Q);
  if (c.rows <= 0 || h >= a.H) return;
  // finite, so that no step (also a token behind the chunk's last) decays nothing
  double l2 = -exp(static_cast<double>(a.A_log[h])) * 1.4426950408889634;
  l2 = l2 < -1e300 ? -1e300 : l2;
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
    // a decay below 2^-1024 is zero in fp32 already; sums stay finite (NaN stays)
    const double log = l2 * dt[r];
    cum[r] = (log < -1024.0 ? -1024.0 : log) + (r ? cum[r - 1] : 0.0);
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

// Of units of a row, the largest bits without signs: whether a value is NaN or
// infinite.
template <typename TI>
struct Largest {
  typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;
  uint32_t top = 0;
  __device__ __forceinline__ void add(const uint4& u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(TI) == 2)
        top = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, top), __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu)));
      else
        top = max(top, w[i] & 0x7fffffffu);
    }
  }
  __device__ __forceinline__ bool finite() const {
    if constexpr (sizeof(TI) == 2) return !((top + 0x00800080u) & 0x80008000u);
    else return top < 0x7f800000u;
  }
};

// A chunk's R rows of COLS columns on their way to a tile: 16-byte units, thread
// t's m-th unit number t + TH m. Addresses are a base that the block shares plus
// 32 bits (token strides are below 2^22 elements). Rows behind the chunk's last
// are read as its last and made zero when they are stored, and what is loaded
// ahead at the end is loaded twice: a load under a condition would be waited for
// where the condition ends. For the same reason nothing is computed from a load
// before its use, and no part of one is left unused: its registers would be given
// to other values, which wait for it.
template <typename TI, int R, int COLS, int TH>
struct Rows {
  static constexpr int U = 16 / sizeof(TI), PER = R * COLS / U / TH, RPM = TH / (COLS / U);
  static_assert(RPM % 8 == 0, "a thread's units lie whole periods of the tile's order apart, or half ones");
  uint4 v[PER];
  __device__ __forceinline__ void load(const TI* base, uint32_t stride, int rows, int tid) {
    const uint32_t r0 = static_cast<uint32_t>(tid) / (COLS / U), col = 16 * (static_cast<uint32_t>(tid) % (COLS / U));
    const uint32_t last = static_cast<uint32_t>(rows - 1);
#pragma unroll
    for (int m = 0; m < PER; ++m) {
      const uint32_t r = r0 + RPM * m, at = r < last ? r : last;
      v[m] = *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(base) + (__umul24(at, stride * static_cast<uint32_t>(sizeof(TI))) + col));
    }
  }
  static __device__ __forceinline__ int place(int tid, int m) {
    const int at = tile_at<TI, COLS>(tid / (COLS / U), (tid % (COLS / U)) * U);
    return (at ^ (RPM * m & 8 ? TileFlip<TI, COLS>::units(8) * U : 0)) + m * RPM * COLS;
  }
  __device__ __forceinline__ uint4 kept(int rows, int tid, int m) const {
    return tid / (COLS / U) + RPM * m < rows ? v[m] : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void store(TI* tile, int rows, int tid) const {
#pragma unroll
    for (int m = 0; m < PER; ++m) *reinterpret_cast<uint4*>(tile + place(tid, m)) = kept(rows, tid, m);
  }
  __device__ __forceinline__ bool finite() const {
    Largest<TI> l;
#pragma unroll
    for (int m = 0; m < PER; ++m) l.add(v[m]);
    return l.finite();
  }
  // Stores zeros for what is no finite number, and in `first` (of each column) the
  // first row that has one.
  __device__ __forceinline__ void store_finite(TI* tile, int rows, int tid, int* first) const {
#pragma unroll 1
    for (int m = 0; m < PER; ++m) {
      uint4 u = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < PER; ++k)
        if (k == m) u = kept(rows, tid, k);
      RowVec<TI> r;
      float f[U];
      r.u = u;
      r.get(f);
#pragma unroll
      for (int e = 0; e < U; ++e)
        if (!(fabsf(f[e]) <= FLT_MAX)) {
          f[e] = 0.f;
          atomicMin(first + (tid % (COLS / U)) * U + e, tid / (COLS / U) + RPM * m);
        }
      r.set(f);
      *reinterpret_cast<uint4*>(tile + place(tid, m)) = r.u;
    }
  }
};
// A state of 64 columns on its way from accumulators to k_ssm_out's tile, in TI:
// [N / 16][64 / 32][lane][2][4], lane i + 16 g with columns 4 g .. 4 g + 3 and 16
// on of row i.
template <typename TI, int N>
struct StateRows {
  static constexpr int TH = 4 * Chunk<TI>::Q, U = 16 / sizeof(TI), PER = N * 64 / U / TH;
  f32x4 v[PER];
  static __device__ __forceinline__ void put(TI* at, int u, const f32x4& a, const f32x4& b) {
    if constexpr (U == 8) {
      bf16x8 f = pair_frag<TI>(a, b);
      *reinterpret_cast<bf16x8*>(at + u * 1024) = f;
    } else {
      *reinterpret_cast<f32x4*>(at + u * 1024) = a;
      *reinterpret_cast<f32x4*>(at + u * 1024 + 4) = b;
    }
  }
  __device__ __forceinline__ void load(const TI* s, int tid) {
#pragma unroll
    for (int m = 0; m < PER; ++m) v[m] = *reinterpret_cast<const f32x4*>(s + (tid + TH * m) * U);
  }
  __device__ __forceinline__ void store(TI* tile, int tid) const {
    constexpr int PARTS = 8 / U, RPM = TH / (128 * PARTS) * 16;  // units a lane, rows a step of TH units
    const int l = tid / PARTS % 64, i = l & 15, g = l >> 4, c = tid / (64 * PARTS) % 2, r = tid / (128 * PARTS) * 16 + i;
#pragma unroll
    for (int m = 0; m < PER; ++m) {
      if constexpr (U == 8) {
        const f32x4 x = v[m];
        typedef __attribute__((ext_vector_type(2))) float f32x2;
        *reinterpret_cast<f32x2*>(tile + tile_at<TI, 64>(r, 32 * c + 4 * g) + m * RPM * 64) = f32x2{x[0], x[1]};
        *reinterpret_cast<f32x2*>(tile + tile_at<TI, 64>(r, 32 * c + 16 + 4 * g) + m * RPM * 64) = f32x2{x[2], x[3]};
      } else {
        *reinterpret_cast<f32x4*>(tile + tile_at<TI, 64>(r, 32 * c + 16 * (tid % 2) + 4 * g) + m * RPM * 64) = v[m];
      }
    }
  }
};

// A token's step size and running sum.
struct Step {
  float dt, hi, lo;
};
__device__ __forceinline__ Step load_step(const float* steps, int64_t at) {
  return *reinterpret_cast<const Step*>(steps + 4 * at);
}

// Blocks of consecutive numbers on one XCD (the hardware deals them out in turn
// over eight), for those that read the same rows. `total` is a multiple of 8.
__device__ __forceinline__ unsigned on_one_xcd(unsigned b, unsigned total) {
  return (b & 7) * (total / 8) + b / 8;
}

// A row of U values as K vectors of TI that add up to them: fp32 itself, or
// three bf16, which hold 24 bits. What is left of an infinity, NaN, is made a
// finite number, at most 2^119 as what is left of those is (1 of 158 us of a
// forward at 8192 x 64 heads; a comparison and a choice 3.5).
template <typename TI>
struct Terms {
  static constexpr int K = sizeof(TI) == 4 ? 1 : 3, U = 16 / sizeof(TI);
  static __device__ __forceinline__ void split(float (&f)[U], RowVec<TI> (&v)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k].set(f);
      if (k + 1 < K) {
        float h[U];
        v[k].get(h);
#pragma unroll
        for (int e = 0; e < U; ++e) f[e] = k > 0 ? f[e] - h[e] : __builtin_amdgcn_fmed3f(f[e] - h[e], -0x1p119f, 0x1p119f);
      }
    }
  }
};

// One block walks the chunks of a segment with 64 columns of one head's state:
// S' = e^tot S + B^T (w x), w_j = dt_j exp(cum_Q - cum_j); in reverse
// dS = e^tot dS' + C^T (w dy), w_i = exp(cum_i). The weighted rows are three bf16
// each, B and C are exact, so that states are fp32 states. A wave holds 32 columns
// by half the rows of the transposed state, a lane four columns of a row of each
// of its tiles.
//
// A sequence is one segment unless it is long (see SsmArgs::long_from); of those,
// kLocal leaves what each segment adds to a state that enters it as zero, and the
// second launch starts each segment from the states that the ones before it have
// left.
enum { kLocal = 0, kStates = 1, kFullStates = 2 };  // leave what a segment adds; states in TI; in fp32
template <typename TI, int N, int MODE>
__global__ void __launch_bounds__(256, 2) k_ssm_state(SsmArgs a, int dirs, int dir0, unsigned blocks) {
  constexpr int Q = Chunk<TI>::Q, U = 16 / sizeof(TI), NT = N / 32;
  constexpr int K = Terms<TI>::K;
  constexpr bool LOCAL = MODE == kLocal;
  __shared__ __align__(16) TI bs[Q * N], xs[K][Q * 64];
  const int halves = a.P / 64, seg = a.seg;
  unsigned b = on_one_xcd(blockIdx.x, gridDim.x);
  if (b >= blocks) return;
  // heads vary slowest: each XCD has some of them, with all their segments,
  // whose lengths differ
  const unsigned per_head = blocks / (a.H * halves);
  const int hp = b / per_head, h = hp / halves, half = hp % halves;
  b %= per_head;
  const int rev = dirs > 1 ? b % 2 : dir0;
  const int64_t sslot = dirs > 1 ? b / 2 : b;
  // without segments a slot is a sequence, also one without tokens
  Place c;
  if (seg) {
    c = find_piece(a, sslot, seg * Q);
  } else {
    c = {static_cast<int>(sslot), 0, 0, clamp_cu(a, sslot), clamp_cu(a, sslot + 1), 0};
    c.t0 = c.s0;
    c.rows = static_cast<int>(c.s1 > c.s0 ? c.s1 - c.s0 : 0);
  }
  const int64_t len = c.s1 > c.s0 ? c.s1 - c.s0 : 0;
  int segs = 1;  // of the sequence
  if (seg) {
    if (c.n < 0) return;
    if (len > a.long_from) segs = static_cast<int>((len + seg * Q - 1) / (seg * Q));
    else c.rows = static_cast<int>(len);
    if (c.pos >= segs) return;
  }
  const bool ends = rev ? c.pos == 0 : c.pos == segs - 1;  // its state leaves the sequence
  if (LOCAL && ends) return;
  const int grp = h / (a.H / a.G);
  const int tid = threadIdx.x, lane = tid & 63, w = wave_number(), i = lane & 15, g = lane >> 4;
  const int p0 = 32 * (w & 1), nt = (N / 2) * (w >> 1);
  const int64_t t0 = c.t0;
  const int tokens = c.rows, nch = (tokens + Q - 1) / Q;
  const int64_t first = static_cast<uint32_t>(c.s0) / Q + c.n + (t0 - c.s0) / Q;  // slot of the first chunk
  const TI* src = static_cast<const TI*>(rev ? a.dy : a.x) + static_cast<size_t>(h) * a.P + half * 64;
  const int64_t sst = rev ? static_cast<int64_t>(a.H) * a.P : a.xs;
  const TI* rsrc = static_cast<const TI*>(rev ? a.C : a.B) + static_cast<size_t>(grp) * N;
  const int64_t rst = rev ? a.Cs : a.Bs;
  const float* from = rev ? a.dfinal : a.init;
  float* to = rev ? a.dinit : a.final_state;
  const size_t state = ((static_cast<size_t>(c.n) * a.H + h) * N + nt + i) * a.P + half * 64 + p0 + 4 * g;
  // of a slot, as in SsmArgs::S without and with S_full
  const size_t tile = static_cast<size_t>(hp) * N * 64 + (nt / 16 * 2 + p0 / 32) * 512 + 8 * lane, step = static_cast<size_t>(a.H) * halves * N * 64;
  const size_t order = static_cast<size_t>(hp) * N * 64 + (nt / 16 * 4 + p0 / 16) * 256 + 4 * lane;
  float* local = a.local + rev * a.seg_slots * step + order;

  const LaneAt<TI, 64> lx(lane);
  const LaneAt<TI, N> lb(lane);
  f32x4 acc[NT][2];
#pragma unroll
  for (int u = 0; u < NT; ++u)
#pragma unroll
    for (int t = 0; t < 2; ++t)
      acc[u][t] = from && !LOCAL ? *reinterpret_cast<const f32x4*>(from + state + static_cast<size_t>(16 * u) * a.P + 16 * t) : zero4();
  if (!LOCAL && seg) {
    for (int k = 0; k < (rev ? segs - 1 - c.pos : c.pos); ++k) {
      const int64_t at = sslot - c.pos + (rev ? segs - 1 - k : k);
      const float d = exp2_(a.seg_log[(rev * a.seg_slots + at) * a.H + h]);
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          acc[u][t] = d * acc[u][t] + *reinterpret_cast<const f32x4*>(local + at * step + (4 * u + t) * 256);
    }
  }

  using RX = Rows<TI, Q, 64, 256>;
  RX rx;
  Rows<TI, Q, N, 256> rb;
  Step rk[RX::PER];
  float end_hi, end_lo;
  auto load = [&](int k) __attribute__((always_inline)) {
    const int ch = rev ? nch - 1 - k : k, rows = tokens - ch * Q;
    const int64_t at = t0 + static_cast<int64_t>(ch) * Q;
    const float* steps = a.steps + ((first + ch) * a.H + h) * (4 * Q);
    end_hi = steps[4 * Q - 3];
    end_lo = steps[4 * Q - 2];
    rx.load(src + at * sst, static_cast<uint32_t>(sst), rows, tid);
#pragma unroll
    for (int m = 0; m < RX::PER; ++m) rk[m] = load_step(steps, tid / (64 / U) + RX::RPM * m);
    rb.load(rsrc + at * rst, static_cast<uint32_t>(rst), rows, tid);
  };
  double total = 0.0;
  if (nch > 0) load(0);
  for (int k = 0; k < nch; ++k) {
    const int ch = rev ? nch - 1 - k : k;
    const int rows = tokens - ch * Q;
    __syncthreads();
    rb.store(bs, rows, tid);
#pragma unroll
    for (int m = 0; m < RX::PER; ++m) {
      RowVec<TI> v, t[K];
      float f[U];
      v.u = rx.kept(rows, tid, m);
      v.get(f);
      const float wt = rev ? exp2_(rk[m].hi + rk[m].lo) : rk[m].dt * exp2_((end_hi - rk[m].hi) + (end_lo - rk[m].lo));
#pragma unroll
      for (int e = 0; e < U; ++e) f[e] *= wt;
      Terms<TI>::split(f, t);
#pragma unroll
      for (int q = 0; q < K; ++q) *reinterpret_cast<uint4*>(xs[q] + RX::place(tid, m)) = t[q].u;
    }
    const float log = end_hi + end_lo, decay = exp2_(log);
    total += log;
    __syncthreads();
    load(k + 1 < nch ? k + 1 : k);
    if constexpr (!LOCAL) {
      const size_t at = (first + ch) * step;
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        // whole lines at once, fp32 past the caches
        if constexpr (MODE == kFullStates) {
#pragma unroll
          for (int t = 0; t < 2; ++t) store4<float, true>(static_cast<float*>(rev ? a.dS : a.S) + at + order + (4 * u + t) * 256, acc[u][t]);
        } else {
          StateRows<TI, N>::put(static_cast<TI*>(a.S) + at + tile, u, acc[u][0], acc[u][1]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int t = 0; t < 2; ++t) acc[u][t] *= decay;
    // operands a step ahead of their products: the wave waits for no read
    struct Operands {
      Frag<TI> x[2][K], b[NT];
    } f[2];
    auto read = [&](int k0, Operands& o) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int q = 0; q < K; ++q) o.x[t][q] = frag_col<false>(xs[q], lx, k0, p0 + 16 * t);
#pragma unroll
      for (int u = 0; u < NT; ++u) o.b[u] = frag_col<false>(bs, lb, k0, nt + 16 * u);
    };
    read(0, f[0]);
#pragma unroll
    for (int k0 = 0; k0 < Q; k0 += 32) {
      Operands& o = f[(k0 / 32) % 2];
      if (k0 + 32 < Q) read(k0 + 32, f[(k0 / 32 + 1) % 2]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int q = K - 1; q >= 0; --q)
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int t = 0; t < 2; ++t) acc[u][t] = mma32(o.x[t][q], o.b[u], acc[u][t]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if constexpr (LOCAL) {
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int t = 0; t < 2; ++t) *reinterpret_cast<f32x4*>(local + sslot * step + (4 * u + t) * 256) = acc[u][t];
    if (tid == 0 && half == 0) a.seg_log[(rev * a.seg_slots + sslot) * a.H + h] = static_cast<float>(total);
  } else if (to && ends) {
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        *reinterpret_cast<f32x4*>(to + state + static_cast<size_t>(16 * u) * a.P + 16 * t) = acc[u][t];
  }
}

// ------------------------------------------------------------ shared by out and grad

__host__ __device__ inline unsigned own_blocks(const SsmArgs& a) {
  return a.whole + (static_cast<unsigned>(a.slots) * a.G - a.whole) * a.sets;
}
// What block b of k_ssm_out and k_ssm_grad does: the heads [h0, h1) of a group in
// a chunk, all of them in the first a.whole blocks, a.sets blocks a chunk and
// group behind those.
struct Unit {
  int64_t slot;
  int grp, set, h0, h1;
};
__device__ __forceinline__ Unit unit_of(const SsmArgs& a, unsigned b) {
  const int per = a.H / a.G;
  const unsigned k = b < a.whole ? 0 : b - a.whole, unit = b < a.whole ? b : a.whole + k / a.sets;
  Unit u;
  u.set = k % a.sets;
  u.grp = unit % a.G;
  u.slot = unit / a.G;
  const int hb = b < a.whole ? per : (per + a.sets - 1) / a.sets, last = (u.set + 1) * hb;
  u.h0 = u.grp * per + (u.set * hb < per ? u.set * hb : per);
  u.h1 = u.grp * per + (last < per ? last : per);
  return u;
}

// A wave's tile of 16 tokens: those of wave w and w + NW / 2, which share a
// SIMD, are as far from the diagonal's ends as each other, so that every SIMD
// has the same number of score tiles.
template <int NW>
__device__ __forceinline__ int own_tile(int w) {
  return w < NW / 2 ? w : NW - 1 - (w - NW / 2);
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

// One group's chunk a block, the heads in turn: 64 us at 8192 x 64 heads. C B^T
// stays in registers over the heads (at 128 registers, two blocks a CU, with 9 of
// them spilled at N = 128; operands read further ahead spill more), the next head's rows and state are loaded during a
// head's products. Wave: 16 tokens i of the chunk. Scores are formed as [j][i] accumulators, an
// operand as they stand of y^T[p][i] = sum_j x_j[p] (L G dt)_ij.
template <typename TI, int N>
__global__ void __launch_bounds__(4 * Chunk<TI>::Q, sizeof(TI) == 2 ? 4 : 2) k_ssm_out(SsmArgs a) {
  constexpr int Q = Chunk<TI>::Q, NW = Q / 16, TH = 64 * NW;
  __shared__ __align__(16) TI buf[2 * Q * N];
  __shared__ float chi[Q], clo[Q], cdt[Q];
  __shared__ __align__(16) int first[2][64];  // by turns: of each column of x, the first row that is not finite
  __shared__ int odd[2];                      // whether there is one
  const unsigned own = own_blocks(a);
  if (blockIdx.x >= own) {
    zero_rows(static_cast<TI*>(a.y), static_cast<int64_t>(a.H) * a.P, a, blockIdx.x - own, gridDim.x - own);
    return;
  }
  const Unit unit = unit_of(a, blockIdx.x);
  const int64_t slot = unit.slot;
  const int grp = unit.grp, h0 = unit.h0, h1 = unit.h1;
  const Place c = find_piece(a, slot, Q);
  const int rows = c.rows;
  const int64_t t0 = c.t0;
  if (rows <= 0 || h0 >= h1) return;
  const int tid = threadIdx.x, lane = tid & 63, w = wave_number(), i = lane & 15, g = lane >> 4;
  const int it = own_tile<NW>(w), halves = a.P / 64;

  const LaneAt<TI, N> ln(lane);
  TI *Bt = buf, *Ct = buf + Q * N;
  {
    Rows<TI, Q, N, TH> rb, rc;
    rb.load(static_cast<const TI*>(a.B) + t0 * a.Bs + static_cast<size_t>(grp) * N, static_cast<uint32_t>(a.Bs), rows, tid);
    rc.load(static_cast<const TI*>(a.C) + t0 * a.Cs + static_cast<size_t>(grp) * N, static_cast<uint32_t>(a.Cs), rows, tid);
    rb.store(Bt, rows, tid);
    rc.store(Ct, rows, tid);
  }
  if (tid < 64) first[0][tid] = Q;
  if (tid == 0) odd[0] = 0;
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
  Rows<TI, Q, 64, TH> nx;  // the next head's x and state
  StateRows<TI, N> ns;
  Step nstep;
  auto load = [&](int h, int half) __attribute__((always_inline)) {
    nx.load(static_cast<const TI*>(a.x) + t0 * a.xs + static_cast<size_t>(h) * a.P + half * 64, static_cast<uint32_t>(a.xs), rows, tid);
    ns.load(static_cast<const TI*>(a.S) + ((slot * a.H + h) * halves + half) * static_cast<size_t>(N) * 64, tid);
    nstep = load_step(a.steps, (slot * a.H + h) * Q + tid % Q);
  };
  load(h0, 0);
  int turn = 0;
  for (int h = h0; h < h1; ++h) {
    const float D = a.D ? a.D[h] : 0.f;
    for (int half = 0; half < halves; ++half, turn ^= 1) {
      __syncthreads();
      if (tid < 64) first[turn ^ 1][tid] = Q;
      if (tid == 0) odd[turn ^ 1] = 0;
      // The products take whole pairs of tiles, and the zero scores of the tokens
      // behind i times NaN or an infinity would be NaN: x is stored without them, and
      // what they belong to is made NaN below (which token by token it is too, an
      // infinity by C S of rows of both signs). Looking for them costs 2.5 of 120 to
      // 250 us of a forward at 8192 x 64 heads.
      if (__builtin_expect(__any(!nx.finite()), 0)) {
        nx.store_finite(xs, rows, once(tid), first[turn]);
        odd[turn] = 1;
      } else {
        nx.store(xs, rows, tid);
      }
      ns.store(Ss, once(tid));
      if (tid < Q) {
        cdt[tid] = nstep.dt;
        chi[tid] = nstep.hi;
        clo[tid] = nstep.lo;
      }
      __syncthreads();
      const bool next = half + 1 == halves && h + 1 < h1;
      load(next ? h + 1 : h, half + 1 < halves ? half + 1 : next ? 0 : half);
      const LaneAt<TI, 64> lx(once(lane));
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
      if (__builtin_expect(odd[turn], 0)) {
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (row >= first[turn][16 * p + 4 * g + r]) y[p][r] = nan_value();
      }
      if (row < rows) {
        TI* out = static_cast<TI*>(a.y) + ((t0 + row) * a.H + h) * a.P + half * 64 + 4 * g;
#pragma unroll
        for (int p = 0; p < 4; ++p) store4<TI>(out + 16 * p, y[p] + D * tile_get4(xs, lx, 16 * it, 16 * p));
      }
    }
  }
}

// ------------------------------------------------------------ gradients

// Sums over the four lane groups (lanes i, i + 16, i + 32, i + 48), gfx950's swaps
// of half and quarter waves: of one value, every lane receiving it, and of four at
// once, group g receiving that of v[(g >> 1) | 2 (g & 1)].
__device__ __forceinline__ float sum_lane_groups(float x) {
  const uint32_t b = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  const uint32_t c = __float_as_uint(x);
  const auto h = __builtin_amdgcn_permlane32_swap(c, c, false, false);
  return __uint_as_float(h[0]) + __uint_as_float(h[1]);
}
__device__ __forceinline__ float sum_lane_groups4(const float (&v)[4]) {
  float s[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[2 * k]), __float_as_uint(v[2 * k + 1]), false, false);
    s[k] = __uint_as_float(h[0]) + __uint_as_float(h[1]);
  }
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(s[0]), __float_as_uint(s[1]), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Values of an fp32 state as operands that add up to them (three bf16 are 24 bits).
template <typename TI>
struct Split {
  static constexpr int K = sizeof(TI) == 4 ? 1 : 3;
  Frag<TI> f[K];
  __device__ __forceinline__ void set(f32x8 x) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[k][e] = static_cast<TI>(x[e]);
        if (k + 1 < K) x[e] -= static_cast<float>(f[k][e]);
      }
  }
  __device__ __forceinline__ f32x4 mma(Frag<TI> b, f32x4 c) const {
#pragma unroll
    for (int k = K - 1; k >= 0; --k) c = mma32(f[k], b, c);
    return c;
  }
};

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

// The next head's rows are loaded while a head's are worked on. The sums over a
// row or column of scores that the step sizes' gradient needs are left to
// k_ssm_scalars: what is added up over the chunk there costs a wave some
// microseconds that the others would wait for here.
template <typename TI, int N>
__global__ void __launch_bounds__(4 * Chunk<TI>::Q) k_ssm_grad(SsmArgs a) {
  using SH = GradShape<TI, N>;
  constexpr int Q = SH::Q, NW = SH::NW, TH = 64 * NW, NT = SH::NT, NG = SH::NG, TT = SH::TT;
  constexpr int U = 16 / sizeof(TI);
  __shared__ __align__(16) TI Bt[Q * N], Ct[Q * N], xs[Q * 64], dys[Q * 64], MT[Q * Q], Gs[N * 64];
  // per token: step size, decays from the chunk's start to it and from it to the
  // end, and the running sum of log2 decays, whose differences lose their digits
  // unless both parts are taken
  __shared__ __align__(16) float cdt[Q], cin[Q], cout[Q], chi[Q], clo[Q], rowF[NW][Q], iC[NG][Q], iB[NG][Q], colF[Q], ownF[Q];
  __shared__ float sd[NW], xd[NW];
  const unsigned own = own_blocks(a);
  if (blockIdx.x >= own) {
    const unsigned b = blockIdx.x - own, nb = gridDim.x - own;
    zero_rows(static_cast<TI*>(a.dx), static_cast<int64_t>(a.H) * a.P, a, b, nb);
    zero_rows(static_cast<TI*>(a.ddt), a.H, a, b, nb);
    zero_rows(static_cast<TI*>(a.dB), static_cast<int64_t>(a.G) * N, a, b, nb);
    zero_rows(static_cast<TI*>(a.dC), static_cast<int64_t>(a.G) * N, a, b, nb);
    return;
  }
  const Unit unit = unit_of(a, blockIdx.x);
  const int64_t slot = unit.slot;
  const int grp = unit.grp, h0 = unit.h0, h1 = unit.h1;
  const Place c = find_piece(a, slot, Q);
  const int rows = c.rows;
  const int64_t t0 = c.t0;
  if (rows <= 0 || h0 >= h1) return;
  const int tid = threadIdx.x, lane = tid & 63, w = wave_number();
  const int jt = own_tile<NW>(w), halves = a.P / 64;
  // the sums over a diagonal tile's columns lie where the waves of the last tiles
  // have no rows
  auto tile_cols = [&](int t) __attribute__((always_inline)) { return t + 1 < NW ? rowF[NW / 2] + 16 * t : rowF[NW / 2 + 1]; };
  const int ng = NG == NW ? w : w % NG, tt0 = NG == NW ? 0 : (w / NG) * TT, n0 = ng * NT * 16;  // of the second role

  Rows<TI, Q, 64, TH> nx, ny;
  Step nstep;
  float end_hi, end_lo;
  f32x8 G0[NT][2], S0[NT][2];  // dS and S, rows n0 .. as operands
  auto load_rows = [&](int h, int half) __attribute__((always_inline)) {
    const int64_t ds = static_cast<int64_t>(a.H) * a.P;
    const int ft = once(tid);
    nx.load(static_cast<const TI*>(a.x) + t0 * a.xs + static_cast<size_t>(h) * a.P + half * 64, static_cast<uint32_t>(a.xs), rows, ft);
    ny.load(static_cast<const TI*>(a.dy) + t0 * ds + static_cast<size_t>(h) * a.P + half * 64, static_cast<uint32_t>(ds), rows, ft);
    const int64_t at = (slot * a.H + h) * Q;
    nstep = load_step(a.steps, at + ft % Q);
    end_hi = a.steps[4 * (at + Q) - 3];
    end_lo = a.steps[4 * (at + Q) - 2];
  };
  auto load_state = [&](f32x8 (&f)[NT][2], const void* from, int h, int half) __attribute__((always_inline)) {
    const float* m = static_cast<const float*>(from) + ((slot * a.H + h) * halves + half) * static_cast<size_t>(N) * 64;
    const int fresh = once(lane);
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int k = 0; k < 2; ++k) f[u][k] = frag_state(m, n0 + 16 * u, 32 * k, fresh);
  };
  load_rows(h0, 0);
  load_state(G0, a.dS, h0, 0);
  {
    Rows<TI, Q, N, TH> rb, rc;
    rb.load(static_cast<const TI*>(a.B) + t0 * a.Bs + static_cast<size_t>(grp) * N, static_cast<uint32_t>(a.Bs), rows, tid);
    rc.load(static_cast<const TI*>(a.C) + t0 * a.Cs + static_cast<size_t>(grp) * N, static_cast<uint32_t>(a.Cs), rows, tid);
    rb.store(Bt, rows, tid);
    rc.store(Ct, rows, tid);
  }
  __syncthreads();
  f32x4 dC[NT][TT], dB[NT][TT];
#pragma unroll
  for (int u = 0; u < NT; ++u)
#pragma unroll
    for (int t = 0; t < TT; ++t) dC[u][t] = dB[u][t] = zero4();

  for (int h = h0; h < h1; ++h) {
    const float D = a.D ? a.D[h] : 0.f;
    for (int half = 0; half < halves; ++half) {
      const int fresh = once(lane), i = fresh & 15, g = fresh >> 4;
      const LaneAt<TI, N> ln(fresh);
      const LaneAt<TI, 64> lx(fresh);
      const LaneAt<TI, Q> lq(fresh);
      {
        const int ft = once(tid);
        nx.store(xs, rows, ft);
        ny.store(dys, rows, ft);
        if (tid < Q) {
          cdt[ft] = nstep.dt;
          cin[ft] = exp2_(nstep.hi + nstep.lo);
          cout[ft] = exp2_((end_hi - nstep.hi) + (end_lo - nstep.lo));
          chi[ft] = nstep.hi;
          clo[ft] = nstep.lo;
        }
        if (tt0 == 0) {  // dS as the first role's operand
#pragma unroll
          for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
              for (int e = 0; e < 8; e += U) {
                RowVec<TI> v;
                float f[U];
#pragma unroll
                for (int q = 0; q < U; ++q) f[q] = G0[u][k][e + q];
                v.set(f);
                *reinterpret_cast<uint4*>(Gs + shifted<LaneAt<TI, 64>>(lx.row, 32 * k + e) + (n0 + 16 * u) * 64) = v.u;
              }
            }
        }
      }
      __syncthreads();
      const bool more = half + 1 < halves || h + 1 < h1;
      const bool next = half + 1 == halves && more;
      const int nh = next ? h + 1 : h, nhalf = half + 1 < halves ? half + 1 : next ? 0 : half;
      const float all = cin[Q - 1];

      {  // first role
        const int row = 16 * jt + i;
        const float dtj = cdt[row], rj = cout[row], hj = chi[row], lj = clo[row];
        Frag<TI> xf[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) xf[k] = frag_row(xs, lx, 16 * jt, 32 * k);
        f32x4 dx[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) dx[p] = zero4();
        Frag<TI> bf[N / 32];
        {
          Frag<TI> gf[2][4];
          auto read = [&](int k) __attribute__((always_inline)) {
            bf[k] = frag_row(Bt, ln, 16 * jt, 32 * k);
#pragma unroll
            for (int p = 0; p < 4; ++p) gf[k % 2][p] = frag_col<false>(Gs, lx, 32 * k, 16 * p);
          };
          read(0);
#pragma unroll
          for (int k = 0; k < N / 32; ++k) {
            if (k + 1 < N / 32) read(k + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int p = 0; p < 4; ++p) dx[p] = mma32(gf[k % 2][p], bf[k], dx[p]);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) dx[p] *= rj;
        // what follows j: behind its own tile of 16 tokens, and in it
        float cf = 0.f, cd = 0.f, diag = 0.f;
#pragma unroll
        for (int m = 0; m < NW / 2; ++m) {
          if (2 * m + 1 < jt) continue;
          // a tile's operands are read at once; those of one above the diagonal for
          // nothing
          Frag<TI> yc[4];
          f32x4 W[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int t = 2 * m + q, i0 = 16 * t + 4 * g;
            Frag<TI> yf[2], qf[N / 32];
#pragma unroll
            for (int k = 0; k < 2; ++k) yf[k] = frag_row(dys, lx, 16 * t, 32 * k);
            // C B^T is formed anew for each head: kept, it would spill
#pragma unroll
            for (int k = 0; k < N / 32; ++k) qf[k] = frag_row(Ct, ln, 16 * t, 32 * k);
            const f32x4 h4 = *reinterpret_cast<const f32x4*>(chi + i0), l4 = *reinterpret_cast<const f32x4*>(clo + i0);
            if (q == 1) {
#pragma unroll
              for (int p = 0; p < 4; ++p) yc[p] = frag_col<true>(dys, lx, 32 * m, 16 * p);
            }
            __builtin_amdgcn_sched_barrier(0);
            W[q] = zero4();
            f32x4 M = zero4();
            if (t >= jt) {
              f32x4 e = zero4(), cb = zero4(), f;
#pragma unroll
              for (int k = 0; k < N / 32; ++k) {
                if (k < 2) e = mma32(yf[k], xf[k], e);
                cb = mma32(qf[k], bf[k], cb);
              }
              const bool below = t > jt;
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float L = below || 4 * g + r >= i ? exp2_((h4[r] - hj) + (l4[r] - lj)) : 0.f;
                W[q][r] = L * cb[r];
                M[r] = L * e[r] * dtj;
                f[r] = W[q][r] * e[r];
              }
              if (!below) {  // a token's own score, which decays nowhere, apart
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  if (4 * g + r == i) {
                    diag += e[r];
                    ownF[row] = f[r];
                    f[r] = 0.f;
                  }
              }
              const float sum = (f[0] + f[1]) + (f[2] + f[3]);
              if (below) cf += sum;
              else cd = sum;
#pragma unroll
              for (int r = 0; r < 4; ++r) f[r] *= dtj;
              const float v[4] = {f[0], f[1], f[2], f[3]};
              const float s = transpose_sum16<4>(v);  // lane i: of f[i % 4]
              if (i < 4) rowF[w][i0 + i] = s;
            }
            store4<TI>(MT + shifted<LaneAt<TI, Q>>(lq.four, 16 * t) + 16 * jt * Q, M);
            __builtin_amdgcn_sched_barrier(0);
          }
          const Frag<TI> wf = pair_frag<TI>(W[0], W[1]);
#pragma unroll
          for (int p = 0; p < 4; ++p) dx[p] = mma32(yc[p], wf, dx[p]);
          __builtin_amdgcn_sched_barrier(0);
        }
        cf = sum_lane_groups(cf);
        cd = sum_lane_groups(cd);
        if (g == 0) {
          colF[row] = cf;
          tile_cols(jt)[i] = cd;
        }
        diag = sum_wave(diag);
        if (lane == 0) xd[w] = diag;
        if (row < rows) {
          TI* out = static_cast<TI*>(a.dx) + ((t0 + row) * a.H + h) * a.P + half * 64 + 4 * g;
#pragma unroll
          for (int p = 0; p < 4; ++p) store4<TI>(out + 16 * p, dtj * dx[p] + D * tile_get4(dys, lx, 16 * jt, 16 * p));
        }
      }
      load_state(S0, a.S, h, half);
      __syncthreads();

      {  // second role: dC, then dB
        static_assert(TT % 4 == 0, "sums of four token tiles at once");
        const int order = (g >> 1) | 2 * (g & 1);
        float dot = 0.f, four[4];
        Split<TI> sf[NT][2];
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) dot += S0[u][k][e] * G0[u][k][e];
            sf[u][k].set(S0[u][k]);
          }
        // a token tile's operands are read while the one before it is worked on
        struct Tile {
          Frag<TI> v[2], m[NW / 2];
          uint32_t c4[NT][4];
          float in, wt;
        } tile[2];
        Frag<TI> rows_t[NT][NW / 2];  // this wave's columns of B, then of C, by tokens
        auto read_rows = [&](const TI* from) __attribute__((always_inline)) {
#pragma unroll
          for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int m = 0; m < NW / 2; ++m) rows_t[u][m] = frag_col<false>(from, ln, 32 * m, n0 + 16 * u);
        };
        auto read_c = [&](int t) __attribute__((always_inline)) {
          Tile& o = tile[t % 2];
          const int tt = tt0 + t;
#pragma unroll
          for (int k = 0; k < 2; ++k) o.v[k] = frag_row(dys, lx, 16 * tt, 32 * k);
#pragma unroll
          for (int u = 0; u < NT; ++u) load4_raw<TI>(Ct + shifted<LaneAt<TI, N>>(ln.four, n0 + 16 * u) + 16 * tt * N, o.c4[u]);
          o.in = cin[16 * tt + i];
#pragma unroll
          for (int m = 0; m < NW / 2; ++m)
            if (2 * m <= tt) o.m[m] = frag_col<false>(MT, lq, 32 * m, 16 * tt);
        };
        read_rows(Bt);
        read_c(0);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const int tt = tt0 + t;
          Tile& o = tile[t % 2];
          if (t) read_c(t);
          __builtin_amdgcn_sched_barrier(0);
          float ic = 0.f;
#pragma unroll
          for (int u = 0; u < NT; ++u) {
            f32x4 z = zero4();
#pragma unroll
            for (int k = 0; k < 2; ++k) z = sf[u][k].mma(o.v[k], z);
#pragma unroll
            for (int m = 0; m < NW / 2; ++m)
              if (2 * m <= tt) dC[u][t] = mma32(rows_t[u][m], o.m[m], dC[u][t]);
            const f32x4 c4 = unpack4<TI>(o.c4[u]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              ic += c4[r] * z[r];
              dC[u][t][r] += o.in * z[r];
            }
          }
          four[t % 4] = ic * o.in;
          if (t % 4 == 3) iC[ng][16 * (tt - 3 + order) + i] = sum_lane_groups4(four);
          __builtin_amdgcn_sched_barrier(0);
        }
        dot = sum_wave(dot);
        if (lane == 0) sd[w] = tt0 == 0 ? dot : 0.f;  // waves of the same rows have the same
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int k = 0; k < 2; ++k) sf[u][k].set(G0[u][k]);
        load_rows(nh, nhalf);
        auto read_b = [&](int t) __attribute__((always_inline)) {
          Tile& o = tile[t % 2];
          const int tt = tt0 + t;
#pragma unroll
          for (int k = 0; k < 2; ++k) o.v[k] = frag_row(xs, lx, 16 * tt, 32 * k);
#pragma unroll
          for (int u = 0; u < NT; ++u) load4_raw<TI>(Bt + shifted<LaneAt<TI, N>>(ln.four, n0 + 16 * u) + 16 * tt * N, o.c4[u]);
          o.in = cout[16 * tt + i];
          o.wt = cdt[16 * tt + i];
#pragma unroll
          for (int m = 0; m < NW / 2; ++m)
            if (2 * m + 1 >= tt) o.m[m] = frag_row(MT, lq, 16 * tt, 32 * m);
        };
        read_rows(Ct);
        read_b(0);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const int tt = tt0 + t;
          Tile& o = tile[t % 2];
          if (t) read_b(t);
          __builtin_amdgcn_sched_barrier(0);
          float ib = 0.f;
          if (t == TT / 2) load_state(G0, a.dS, nh, nhalf);
#pragma unroll
          for (int u = 0; u < NT; ++u) {
            f32x4 v = zero4();
#pragma unroll
            for (int k = 0; k < 2; ++k) v = sf[u][k].mma(o.v[k], v);
#pragma unroll
            for (int m = 0; m < NW / 2; ++m)
              if (2 * m + 1 >= tt) dB[u][t] = mma32(rows_t[u][m], o.m[m], dB[u][t]);
            const f32x4 b4 = unpack4<TI>(o.c4[u]);
            const float wj = o.in * o.wt;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              ib += b4[r] * v[r];
              dB[u][t][r] += wj * v[r];
            }
          }
          four[t % 4] = ib * o.in;
          if (t % 4 == 3) iB[ng][16 * (tt - 3 + order) + i] = sum_lane_groups4(four);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      __syncthreads();

      {  // what k_ssm_scalars adds up: four lanes a token
        const int ft = once(tid), t = ft >> 2, part = ft & 3;
        float rf = 0.f, cc = 0.f, cb = 0.f;
#pragma unroll
        for (int k = 0; k < NW / 4; ++k)
          if (t / 16 >= own_tile<NW>(part * (NW / 4) + k)) rf += rowF[part * (NW / 4) + k][t];
#pragma unroll
        for (int k = 0; k < NG / 4; ++k) {
          cc += iC[part * (NG / 4) + k][t];
          cb += iB[part * (NG / 4) + k][t];
        }
        rf = group_sum<4>(rf);
        cc = group_sum<4>(cc);
        cb = group_sum<4>(cb);
        if (part == 0) {
          const float col = colF[t], in = tile_cols(t / 16)[t % 16], d = cdt[t];
          const int64_t at = (slot * a.H + h) * Q + t;
          f32x4* out = reinterpret_cast<f32x4*>(a.sums) + at;
          f32x4 v = f32x4{cc, d * cb, ((col + in) + ownF[t]) + cb, rf - d * in};
          float b = d * col;
          if (half) {  // the head's first half, of this thread
            v += *out;
            b += a.before[at];
          }
          *out = v;
          a.before[at] = b;
        }
        // this wave's columns by the tiles of the rows behind theirs
#pragma unroll
        for (int k = 0; k < Q / 64; ++k) {
          const int l = ft & 63, tile = 4 * k + (l >> 4);
          float x = group_sum<16>(tile > jt ? rowF[w][64 * k + l] : 0.f);
          float* out = a.cross + (slot * a.H + h) * (NW * NW) + jt * NW + tile;
          if (l % 16 == 0) *out = half ? *out + x : x;
        }
        if (tid == 0) {
          float dots = 0.f, diag = 0.f;
#pragma unroll
          for (int k = 0; k < NW; ++k) {
            dots += sd[k];
            diag += xd[k];
          }
          float* out = a.ends + 2 * (slot * a.H + h);
          dots *= all;
          out[0] = half ? out[0] + dots : dots;
          out[1] = half ? out[1] + diag : diag;
        }
      }
      if (more) __syncthreads();
    }
  }
  // dB and dC of the heads: to the outputs, or to this set's partial sums
  const int i = lane & 15, g = lane >> 4;
  const bool whole = blockIdx.x < a.whole || a.sets == 1;
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int row = 16 * (tt0 + t) + i;
    if (row >= rows) continue;
    const size_t at = ((t0 + row) * a.G + grp) * N + n0 + 4 * g;
    const size_t part = (static_cast<size_t>(blockIdx.x - a.whole) * Q + row) * N + n0 + 4 * g;
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      if (whole) {
        store4<TI>(static_cast<TI*>(a.dB) + at + 16 * u, dB[u][t]);
        store4<TI>(static_cast<TI*>(a.dC) + at + 16 * u, dC[u][t]);
      } else {
        store4<float>(a.pB + part + 16 * u, dB[u][t]);
        store4<float>(a.pC + part + 16 * u, dC[u][t]);
      }
    }
  }
}

// One wave per (chunk, head), Q / 64 tokens a lane: the gradient of each token's
// log decay, of the step sizes, and the chunk's parts of the parameters'.
//
// Of dl_t's first sum, over i >= t > j, pairs of different tiles of 16 tokens are
// added up as they are, by where t lies: in i's tile (a sum over rows from t on),
// in j's (over columns before t) or between them (`cross`, sums over a pair of
// tiles). Those of one tile are differences of what rows and columns from t on add
// up to. Taken over the whole chunk, those differences are short but their roundings
// reach every t before them: dA_log was off by 1e-5 where steps are long, 1e-6 so.
template <typename TI>
__global__ void __launch_bounds__(256) k_ssm_scalars(SsmArgs a) {
  constexpr int Q = Chunk<TI>::Q, R = Q / 64, NW = Q / 16, LT = 16 / R;  // LT: lanes of a tile
  const int nhb = (a.H + 3) / 4;
  const int64_t slot = blockIdx.x / nhb;
  const int h = (blockIdx.x % nhb) * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (h >= a.H) return;
  const Place c = find_piece(a, slot, Q);
  float* out = a.param + slot * 3 * a.H + h;
  if (c.rows <= 0) {  // its parts are added up all the same
    if (lane == 0) out[0] = out[a.H] = out[2 * a.H] = 0.f;
    return;
  }
  const int64_t head = slot * a.H + h, at = head * Q + R * lane;
  f32x4 v[R], st[R];
  float bf[R];
  float sa = 0.f, sb = 0.f, ta = 0.f, tb = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    v[r] = reinterpret_cast<const f32x4*>(a.sums)[at + r];
    st[r] = reinterpret_cast<const f32x4*>(a.steps)[at + r];
    bf[r] = a.before[at + r];
    sa += v[r][0];
    sb += v[r][1];
    ta += v[r][3];
    tb += bf[r];
  }
  const float pair = lane < NW * NW ? a.cross[head * (NW * NW) + lane] : 0.f;
  const float q0 = a.ends[2 * head], diag = a.ends[2 * head + 1];
  // from the lane on, and up to it
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const float da = __shfl_down(sa, o, 64), ub = __shfl_up(sb, o, 64);
    if (lane + o < 64) sa += da;
    if (lane >= o) sb += ub;
    if (o < LT) {
      const float dt = __shfl_down(ta, o, 64), ut = __shfl_up(tb, o, 64);
      if (lane % LT + o < LT) ta += dt;
      if (lane % LT >= o) tb += ut;
    }
  }
  const float ub = __shfl_up(sb, 1, 64), ut = __shfl_up(tb, 1, 64);
  sb = lane ? ub : 0.f;
  tb = lane % LT ? ut : 0.f;
  float over = 0.f;
#pragma unroll
  for (int k = 1; k + 1 < NW; ++k) {
    const float s = sum_wave(lane % NW > k && lane / NW < k ? pair : 0.f);
    if (lane / LT == k) over = s;
  }
  over += q0;
  float Ah = expf(a.A_log[h]);  // finite: what decays at once has a dl of zero
  Ah = Ah > FLT_MAX ? FLT_MAX : Ah;
  float dA = 0.f, db = 0.f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int t = R * lane + r;
    const float dl = t < c.rows ? ((sa + sb) + (ta + tb)) + over : 0.f, d = st[r][3] != 0.f ? (v[r][2] - Ah * dl) * st[r][3] : 0.f;
    sa -= v[r][0];
    sb += v[r][1];
    ta -= v[r][3];
    tb += bf[r];
    dA -= Ah * (st[r][0] * dl);
    db += d;
    if (t < c.rows) static_cast<TI*>(a.ddt)[(c.t0 + t) * a.H + h] = from_f<TI>(d);
  }
  dA = sum_wave(dA);
  db = sum_wave(db);
  if (lane == 0) {
    out[0] = dA;
    out[a.H] = db;
    out[2 * a.H] = diag;
  }
}

// Sums of dB and dC over the sets of heads of the chunks and groups behind the
// whole ones.
template <typename TI, int N>
__global__ void __launch_bounds__(256) k_ssm_reduce(SsmArgs a) {
  constexpr int Q = Chunk<TI>::Q;
  const unsigned unit = a.whole + blockIdx.x;
  const int grp = unit % a.G;
  const Place c = find_piece(a, unit / a.G, Q);
  // sets that have heads: the last ones may have none
  const int per = a.H / a.G, hb = (per + a.sets - 1) / a.sets, sets = (per + hb - 1) / hb;
  for (int e = 4 * (blockIdx.y * 256 + threadIdx.x); e < c.rows * N; e += 4 * 256 * gridDim.y) {
    f32x4 b = zero4(), q = zero4();
    for (int s = 0; s < sets; ++s) {
      const size_t at = (static_cast<size_t>(blockIdx.x) * a.sets + s) * Q * N + e;
      b += *reinterpret_cast<const f32x4*>(a.pB + at);
      q += *reinterpret_cast<const f32x4*>(a.pC + at);
    }
    const size_t to = ((c.t0 + e / N) * a.G + grp) * N + e % N;
    store4<TI>(static_cast<TI*>(a.dB) + to, b);
    store4<TI>(static_cast<TI*>(a.dC) + to, q);
  }
}

unsigned out_rest(const SsmArgs& a, int64_t bytes) {
  return a.cu ? rest_blocks(true, bytes, 1024) : 0;
}

// One or both directions; in segments two launches.
template <typename TI, int N>
hipError_t launch_state_n(int dirs, int dir0, const SsmArgs& a, hipStream_t s) {
  const unsigned blocks = static_cast<unsigned>(a.seg ? a.seg_slots : a.n_seqs) * dirs * a.H * (a.P / 64);
  const unsigned grid = (blocks + 7) / 8 * 8;
  if (a.seg) k_ssm_state<TI, N, kLocal><<<grid, 256, 0, s>>>(a, dirs, dir0, blocks);
  if (a.S_full) k_ssm_state<TI, N, kFullStates><<<grid, 256, 0, s>>>(a, dirs, dir0, blocks);
  else k_ssm_state<TI, N, kStates><<<grid, 256, 0, s>>>(a, dirs, dir0, blocks);
  return hipGetLastError();
}
template <typename TI, int N>
hipError_t launch_out_n(const SsmArgs& a, hipStream_t s) {
  const unsigned own = own_blocks(a);
  k_ssm_out<TI, N><<<own + out_rest(a, a.T * a.H * a.P * static_cast<int64_t>(sizeof(TI))), 4 * Chunk<TI>::Q, 0, s>>>(a);
  return hipGetLastError();
}
template <typename TI, int N>
hipError_t launch_grad_n(const SsmArgs& a, hipStream_t s) {
  const unsigned own = own_blocks(a);
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
hipError_t launch_ssm_state(int dtype, int N, int dirs, int dir0, const SsmArgs& a, hipStream_t s) {
  if (dtype == KDA_F32) return N == 64 ? launch_state_n<float, 64>(dirs, dir0, a, s) : launch_state_n<float, 128>(dirs, dir0, a, s);
  return N == 64 ? launch_state_n<bf16, 64>(dirs, dir0, a, s) : launch_state_n<bf16, 128>(dirs, dir0, a, s);
}
hipError_t launch_ssm_scalars(int dtype, const SsmArgs& a, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.slots) * ((a.H + 3) / 4);
  if (dtype == KDA_F32) k_ssm_scalars<float><<<grid, 256, 0, s>>>(a);
  else k_ssm_scalars<bf16><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
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
  const dim3 grid(static_cast<unsigned>(a.slots) * a.G - a.whole, 8);
  if (dtype == KDA_F32) {
    if (N == 64) k_ssm_reduce<float, 64><<<grid, 256, 0, s>>>(a);
    else k_ssm_reduce<float, 128><<<grid, 256, 0, s>>>(a);
  } else {
    if (N == 64) k_ssm_reduce<bf16, 64><<<grid, 256, 0, s>>>(a);
    else k_ssm_reduce<bf16, 128><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace kda
