// The short causal convolution in front of the operator: depthwise over the
// channels, W = 2 .. 4 taps, packed sequences, initial and final states; its
// backward; and its decoding form on a pool of states.
//
// With e the W-1 rows of a sequence's state followed by its tokens:
//   p_t = bias + sum_j w_j e_{t+j},  y_t = act(p_t)
//   dp_t = dy_t act'(p_t),  de_r = sum_j w_j dp_{r-j} (+ the final state's
//   gradient on the last W-1 rows),  dw_j = sum_t dp_t e_{t+j}
// All are bound by HBM (about 10 operations per element and direction). In
// the packed forms a wave takes 256 channels, four per lane, over a run of
// consecutive tokens, the rows it still needs in registers, so that each row
// is read once and W-1 rows before (and, backward, behind) the run again. One
// run per wave keeps every decision about sequences in scalar registers. Four
// channels per lane rather than eight halve the registers (the backward keeps
// 4 W + 2 values per channel), so more waves cover the loads' latency.
#include "../kda_internal.h"
#include "kda.h"
#include "kda_layer.h"
#include "kda_rows.h"

namespace kda {

namespace {

constexpr int kThreads = 256;
constexpr int kRuns = kThreads / 64;  // waves, and runs, per block
constexpr int kLaneCh = 4;            // channels per lane
constexpr int kWaveCh = 64 * kLaneCh;
constexpr int kAhead = 4;             // tokens loaded together, one such group ahead

// How a launch covers [T][C]: runs of `R` tokens, ncb blocks across the
// channels times nrb along the tokens.
struct Cover {
  int R, ncb;
  int64_t nrb;
};

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Bounds [s, e) of sequence n, inside [0, T] whatever cu_seqlens holds.
struct Bounds {
  int s, e;
};
__device__ __forceinline__ Bounds bounds(const ShortConvArgs& a, int n) {
  const int T = static_cast<int>(a.T);
  if (!a.cu) return Bounds{0, T};
  int s = a.cu[n], e = a.cu[n + 1];
  s = s < 0 ? 0 : (s > T ? T : s);
  e = e > T ? T : e;
  return Bounds{s, e < s ? s : e};
}
__device__ __forceinline__ Bounds uniform_bounds(const ShortConvArgs& a, int n) {
  const Bounds q = bounds(a, n);
  return Bounds{uniform(q.s), uniform(q.e)};
}
// The sequence of token t (the one before it, if t lies in none).
__device__ __forceinline__ int seq_of(const ShortConvArgs& a, int t) {
  return a.cu && a.N > 0 ? uniform(find_seq(a.cu, a.N, t)) : 0;
}

// The lane's channels, `lane_bytes` into a row the whole wave is at: a scalar
// base and a 32-bit lane offset.
template <typename TI>
__device__ __forceinline__ const TI* in_row(const TI* row, uint32_t lane_bytes) {
  return reinterpret_cast<const TI*>(reinterpret_cast<const char*>(row) + lane_bytes);
}
template <typename TI>
__device__ __forceinline__ TI* in_row(TI* row, uint32_t lane_bytes) {
  return reinterpret_cast<TI*>(reinterpret_cast<char*>(row) + lane_bytes);
}

// Four values of a row.
template <typename TI>
struct Row4 {
  uint32_t u[4];
  template <bool NT = false>
  __device__ __forceinline__ void load(const TI* p) {
    typedef __attribute__((ext_vector_type(sizeof(TI)))) uint32_t words;
    const words x = vload<NT>(reinterpret_cast<const words*>(p));
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(TI)); ++i) u[i] = x[i];
  }
  __device__ __forceinline__ f32x4 get() const { return unpack4<TI>(u); }
};

// Row `tt` of the sequence n that starts at s (tt >= s - (W-1)): a token, or
// a row of the initial state.
template <typename TI, int W>
__device__ __forceinline__ f32x4 row_at(const ShortConvArgs& a, int n, int s, int tt, int c) {
  Row4<TI> v;
  if (tt >= s) {
    v.load(static_cast<const TI*>(a.x) + tt * a.xs + c);
  } else if (a.init) {
    v.load(static_cast<const TI*>(a.init) +
           (static_cast<size_t>(n) * (W - 1) + static_cast<size_t>(W - 1 - (s - tt))) * a.C + c);
  } else {
    return zero4();
  }
  return v.get();
}

// Taps [j] of the lane's channels (weight rows [C][W] in order).
template <int W>
__device__ __forceinline__ void load_taps4(const ShortConvArgs& a, int c, f32x4 (&w)[W], f32x4& b) {
  float f[4 * W];
  load_params<4 * W>(a.weight + static_cast<size_t>(c) * W, f);
#pragma unroll
  for (int j = 0; j < W; ++j) w[j] = f32x4{f[j], f[W + j], f[2 * W + j], f[3 * W + j]};
  b = a.bias ? *reinterpret_cast<const f32x4*>(a.bias + c) : zero4();
}

// p = bias + the taps over the W-1 rows of the window and the newest row.
template <int W>
__device__ __forceinline__ f32x4 taps4(const f32x4 (&win)[W - 1], const f32x4& x, const f32x4 (&w)[W],
                                       const f32x4& b) {
  f32x4 p = b;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) p += w[j] * win[j];
  return p + w[W - 1] * x;
}
template <int W>
__device__ __forceinline__ void shift4(f32x4 (&win)[W - 1], const f32x4& x) {
#pragma unroll
  for (int j = 0; j + 1 < W - 1; ++j) win[j] = win[j + 1];
  win[W - 2] = x;
}

// Row len + i of e for i in [0, W-1): the final state (threads past the runs'
// blocks, one per four channels).
template <typename TI, int W>
__device__ __forceinline__ void copy_final(const ShortConvArgs& a, int64_t id) {
  const int nvec = a.C / kLaneCh;
  const int64_t row = id / nvec;
  const int c = static_cast<int>(id - row * nvec) * kLaneCh;
  const int64_t n = row / (W - 1);
  if (n >= a.N) return;
  const Bounds q = bounds(a, static_cast<int>(n));
  const int tt = q.e - (W - 1) + static_cast<int>(row - n * (W - 1));
  store4<TI>(static_cast<TI*>(a.final_state) + static_cast<size_t>(row) * a.C + c,
             row_at<TI, W>(a, static_cast<int>(n), q.s, tt, c));
}

// The part of a run [t0, t1) that lies in one sequence: tokens [a0, a1) of
// sequence n with bounds q. `next` walks the parts in order from token `pos`;
// rows before a0 (and, when it returns false, all left) lie in no sequence.
struct Part {
  int n, a0, a1;
  Bounds q;
};
__device__ __forceinline__ bool next_part(const ShortConvArgs& a, int t1, int pos, int& n, Part& p) {
  for (; n < a.N; ++n) {
    const Bounds q = uniform_bounds(a, n);
    if (q.e <= pos) continue;
    if (q.s >= t1) return false;
    p = Part{n, q.s > pos ? q.s : pos, q.e < t1 ? q.e : t1, q};
    ++n;
    return true;
  }
  return false;
}
template <typename TI>
__device__ __forceinline__ void zero_rows(TI* y, size_t stride, uint32_t lb, int from, int to) {
  for (int t = from; t < to; ++t) store4<TI>(in_row(y + t * stride, lb), zero4());
}

template <typename TI, int W, bool NT>
__global__ void __launch_bounds__(kThreads) k_short_conv(ShortConvArgs a, Cover g) {
  constexpr int U = kAhead;
  const int64_t rb = blockIdx.x / g.ncb;
  if (rb >= g.nrb) {
    copy_final<TI, W>(a, (static_cast<int64_t>(blockIdx.x) - g.nrb * g.ncb) * kThreads + threadIdx.x);
    return;
  }
  const int c = static_cast<int>(blockIdx.x % g.ncb) * kWaveCh + (threadIdx.x & 63) * kLaneCh;
  const int64_t first = (rb * kRuns + uniform(threadIdx.x >> 6)) * g.R;
  if (first >= a.T || c >= a.C) return;
  const int T = static_cast<int>(a.T), t0 = static_cast<int>(first);
  const int t1 = T - t0 > g.R ? t0 + g.R : T;
  const uint32_t lb = c * sizeof(TI);
  const TI* x = static_cast<const TI*>(a.x);
  TI* y = static_cast<TI*>(a.y);
  const size_t xs = a.xs, ys = a.C;
  f32x4 w[W], b;
  load_taps4<W>(a, c, w, b);
  int n = seq_of(a, t0), pos = t0;
  Part p;
  while (pos < t1 && next_part(a, t1, pos, n, p)) {
    zero_rows<TI>(y, ys, lb, pos, p.a0);
    f32x4 win[W - 1];
    auto step = [&](int t, const Row4<TI>& row) {
      const f32x4 xv = row.get();
      f32x4 v = taps4<W>(win, xv, w, b);
      if (a.act == KDA_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= sigmoidf(v[i]);
      }
      store4<TI, NT>(in_row(y + t * ys, lb), v);
      shift4<W>(win, xv);
    };
    Row4<TI> nx[U];
#pragma unroll
    for (int u = 0; u < U; ++u) nx[u].template load<NT>(in_row(x + (p.a1 - p.a0 > u ? p.a0 + u : p.a1 - 1) * xs, lb));
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j] = row_at<TI, W>(a, p.n, p.q.s, p.a0 - (W - 1) + j, c);
    int t = p.a0;
    for (; t + U <= p.a1; t += U) {
      Row4<TI> cx[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        cx[u] = nx[u];
        nx[u].template load<NT>(in_row(x + (p.a1 - t > U + u ? t + U + u : p.a1 - 1) * xs, lb));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) step(t + u, cx[u]);
    }
#pragma unroll
    for (int u = 0; u < U - 1; ++u)
      if (t + u < p.a1) step(t + u, nx[u]);
    pos = p.a1;
  }
  zero_rows<TI>(y, ys, lb, pos, t1);
}

// Backward. A run owns its tokens' rows of dx, its share of dweight and dbias,
// and the initial-state rows of the sequences that start in it. In each
// sequence it walks its tokens and, where the sequence goes on, W-1 behind
// them, and keeps the W rows whose gradient is still incomplete in `acc`: the
// token t adds w_j dp_t to row t + j of e and completes row t. The last W-1
// rows are completed at the sequence's end, where the final state's gradient
// joins them. An empty sequence's state gradient passes through (threads past
// the runs' blocks).
template <typename TI, int W, bool NT>
__global__ void __launch_bounds__(kThreads) k_short_conv_bwd(ShortConvArgs a, Cover g) {
  constexpr int U = kAhead;
  __shared__ __align__(16) float sm[kRuns][kWaveCh];
  const int64_t rb = blockIdx.x / g.ncb;
  if (rb >= g.nrb) {
    const int64_t id = (static_cast<int64_t>(blockIdx.x) - g.nrb * g.ncb) * kThreads + threadIdx.x;
    const int nvec = a.C / kLaneCh;
    const int64_t row = id / nvec, n = row / (W - 1);
    if (n >= a.N) return;
    const Bounds q = bounds(a, static_cast<int>(n));
    if (q.e > q.s) return;
    const size_t at = static_cast<size_t>(row) * a.C + static_cast<size_t>(id - row * nvec) * kLaneCh;
    f32x4 v = zero4();
    if (a.dfinal) {
      Row4<TI> d;
      d.load(static_cast<const TI*>(a.dfinal) + at);
      v = d.get();
    }
    store4<TI>(static_cast<TI*>(a.dinit) + at, v);
    return;
  }
  const int cb = static_cast<int>(blockIdx.x % g.ncb), lane = threadIdx.x & 63;
  const int run = uniform(threadIdx.x >> 6);
  const int c = cb * kWaveCh + lane * kLaneCh;
  const int64_t first = (rb * kRuns + run) * g.R;
  f32x4 dw[W], db = zero4();
#pragma unroll
  for (int j = 0; j < W; ++j) dw[j] = zero4();
  if (first < a.T && c < a.C) {
    const int T = static_cast<int>(a.T), t0 = static_cast<int>(first);
    const int t1 = T - t0 > g.R ? t0 + g.R : T;
    const uint32_t lb = c * sizeof(TI);
    const TI* x = static_cast<const TI*>(a.x);
    const TI* dy = static_cast<const TI*>(a.dy);
    TI* dx = static_cast<TI*>(a.dx);
    const size_t xs = a.xs, ys = a.C;
    f32x4 w[W], b;
    load_taps4<W>(a, c, w, b);
    int n = seq_of(a, t0), pos = t0;
    Part p;
    while (pos < t1 && next_part(a, t1, pos, n, p)) {
      zero_rows<TI>(dx, ys, lb, pos, p.a0);
      // tokens [a1, stop) behind the run; the initial state's rows are this
      // run's if the sequence starts here
      const int stop = p.q.e - p.a1 > W - 1 ? p.a1 + (W - 1) : p.q.e;
      TI* di = p.a0 == p.q.s && a.dinit ? static_cast<TI*>(a.dinit) + static_cast<size_t>(p.n) * (W - 1) * a.C
                                        : nullptr;
      f32x4 acc[W], win[W - 1];
#pragma unroll
      for (int j = 0; j < W; ++j) acc[j] = zero4();
      // row t - (W-1) of the tokens, or before a0 of the initial state
      auto put = [&](int t, const f32x4& v) {
        const int tt = t - (W - 1);
        if (tt >= p.a0) {
          if (tt < p.a1) store4<TI, NT>(in_row(dx + tt * ys, lb), v);
        } else if (di) {
          store4<TI>(in_row(di + (t - p.q.s) * ys, lb), v);
        }
      };
      auto step = [&](int t, const Row4<TI>& xr, const Row4<TI>& dr, bool own) {
        const f32x4 xv = xr.get();
        f32x4 d = dr.get();
        if (a.act == KDA_ACT_SILU) {
          const f32x4 v = taps4<W>(win, xv, w, b);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float s = sigmoidf(v[i]);
            d[i] *= s * (1.f + v[i] * (1.f - s));
          }
        }
        if (own) {
#pragma unroll
          for (int j = 0; j < W - 1; ++j) dw[j] += win[j] * d;
          dw[W - 1] += xv * d;
          db += d;
        }
        put(t, acc[0] + w[0] * d);
#pragma unroll
        for (int j = 0; j + 1 < W; ++j) acc[j] = acc[j + 1] + w[j + 1] * d;
        acc[W - 1] = zero4();
        shift4<W>(win, xv);
      };
      Row4<TI> nx[U], nd[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int tu = stop - p.a0 > u ? p.a0 + u : stop - 1;
        nx[u].template load<NT>(in_row(x + tu * xs, lb));
        nd[u].template load<NT>(in_row(dy + tu * ys, lb));
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j) win[j] = row_at<TI, W>(a, p.n, p.q.s, p.a0 - (W - 1) + j, c);
      int t = p.a0;
      for (; t + U <= p.a1; t += U) {
        Row4<TI> cx[U], cd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int tu = stop - t > U + u ? t + U + u : stop - 1;
          cx[u] = nx[u];
          cd[u] = nd[u];
          nx[u].template load<NT>(in_row(x + tu * xs, lb));
          nd[u].template load<NT>(in_row(dy + tu * ys, lb));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) step(t + u, cx[u], cd[u], true);
      }
      for (; t < stop; ++t) {
        Row4<TI> xr, dr;
        xr.load(in_row(x + t * xs, lb));
        dr.load(in_row(dy + t * ys, lb));
        step(t, xr, dr, t < p.a1);
      }
      if (stop == p.q.e) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
          f32x4 v = acc[j];
          if (a.dfinal) {
            Row4<TI> d;
            d.load(in_row(static_cast<const TI*>(a.dfinal) + (static_cast<size_t>(p.n) * (W - 1) + j) * ys, lb));
            v += d.get();
          }
          put(stop + j, v);
        }
      }
      pos = p.a1;
    }
    zero_rows<TI>(dx, ys, lb, pos, t1);
  }
  // join the block's runs: one partial row of dweight [C][W], dbias [C]
  float* part = a.partials + static_cast<size_t>(rb) * a.C * (W + 1);
  const int cc = cb * kWaveCh + threadIdx.x;  // a thread per channel
  static_assert(kThreads == kWaveCh, "one channel per thread");
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    if (j) __syncthreads();
    *reinterpret_cast<f32x4*>(&sm[run][lane * kLaneCh]) = j < W ? dw[j < W ? j : 0] : db;
    __syncthreads();
    if (cc < a.C) {
      float t = 0.f;
#pragma unroll
      for (int r = 0; r < kRuns; ++r) t += sm[r][threadIdx.x];
      part[j < W ? static_cast<size_t>(cc) * W + j : static_cast<size_t>(a.C) * W + cc] = t;
    }
  }
}

// Decoding: a block takes one sequence and 1024 channels, four per thread, the
// state's rows in registers over the sequence's tokens.
template <typename TI, int W, bool MANY>
__global__ void __launch_bounds__(kThreads) k_short_conv_update(ShortConvArgs a, int ncb) {
  const int n = blockIdx.x / ncb;
  if (n >= a.N) {
    const unsigned own = static_cast<unsigned>(a.N) * ncb;
    zero_rest(a.y, static_cast<size_t>(a.C) * sizeof(TI), a.cu, a.N, a.T, blockIdx.x - own, gridDim.x - own);
    return;
  }
  const int c = static_cast<int>(blockIdx.x % ncb) * kThreads * kLaneCh + threadIdx.x * kLaneCh;
  Bounds q{n, n + 1};
  if (a.cu) q = uniform_bounds(a, n);
  if (q.s >= q.e) return;
  const int64_t slot = find_slot<MANY>(a.idx, a.cu, a.T, n, a.n_slots);
  if (c >= a.C) return;
  const size_t xs = a.xs, ys = a.C;
  const uint32_t lb = c * sizeof(TI);
  const TI* x = static_cast<const TI*>(a.x);
  TI* y = static_cast<TI*>(a.y);
  if (slot < 0) {  // padded: zeros; a slot it cannot have: NaN
    const float f = slot == kPadded ? 0.f : nan_value();
    for (int t = q.s; t < q.e; ++t) store4<TI>(in_row(y + t * ys, lb), f32x4{f, f, f, f});
    return;
  }
  TI* st = static_cast<TI*>(a.state) + static_cast<size_t>(slot) * (W - 1) * a.C;
  Row4<TI> next, old[W - 1];
  next.load(in_row(x + q.s * xs, lb));
#pragma unroll
  for (int j = 0; j < W - 1; ++j) old[j].load(in_row(static_cast<const TI*>(st + j * ys), lb));
  f32x4 w[W], b, win[W - 1];
  load_taps4<W>(a, c, w, b);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) win[j] = old[j].get();
  for (int t = q.s; t < q.e; ++t) {
    const f32x4 xv = next.get();
    if (t + 1 < q.e) next.load(in_row(x + (t + 1) * xs, lb));
    f32x4 v = taps4<W>(win, xv, w, b);
    if (a.act == KDA_ACT_SILU) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] *= sigmoidf(v[i]);
    }
    store4<TI>(in_row(y + t * ys, lb), v);
    shift4<W>(win, xv);
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store4<TI>(in_row(st + j * ys, lb), win[j]);
}

enum { kFwd, kBwd, kUpdate };

// Runs of a multiple of kAhead tokens, 8 at least, such that the waves fill
// whole rounds of 2048: the backward's registers let two waves per SIMD run at
// once, and a part-filled round costs as much as a full one (forward and
// backward of 9000 x 8192: 192 us with 2272 runs of 128, 163 us with 2016 of
// 144). The forward's registers would let more waves run, which gains nothing:
// a step of 8192 x 8192 takes 144 us, with forwards of 4096 or 8192 waves 148 or
// 157. One round while its runs are at most 160 tokens; from there on longer
// ones change little. Longest run, bf16, microseconds forward / backward:
//                    64           96           128          160          192          320
//   4096 x 8192      30.3 / 61.9  29.2 / 50.2  29.3 / 49.8  29.4 / 50.2  29.3 / 50.2  29.3 / 50.4
//   8192 x 8192      51.4 / 96.2  51.7 / 96.9  51.8 / 96.7  50.2 / 82.7  49.5 / 81.9  49.3 / 82.3
//   9000 x 8192      55.8 / 103   53.8 / 96.3  53.8 / 95.5  50.4 / 91.5  50.2 / 91.2  50.2 / 90.8
//   16384 x 8192     103 / 176    107 / 167    105 / 168    97.2 / 154   97.4 / 154   101 / 147
//   20000 x 4096     70.2 / 114   68.9 / 106   68.6 / 105   67.4 / 103   66.9 / 100   67.1 / 102
Cover cover_of(int C, int64_t T) {
  constexpr int64_t kRound = 2048, kLongest = 160;
  Cover c;
  c.ncb = (C + kWaveCh - 1) / kWaveCh;
  const int64_t work = c.ncb * T;  // tokens that one wave at a time walks
  const int64_t rounds = work / (kRound * kLongest) + 1;
  const int64_t run = (work + kRound * rounds - 1) / (kRound * rounds);
  c.R = run <= 8 ? 8 : static_cast<int>((run + kAhead - 1) / kAhead * kAhead);
  c.nrb = ((T + c.R - 1) / c.R + kRuns - 1) / kRuns;
  return c;
}

template <typename TI, int W>
hipError_t launch_w(int what, const ShortConvArgs& a, hipStream_t s) {
  if (what == kUpdate) {
    const int ncb = (a.C + kThreads * kLaneCh - 1) / (kThreads * kLaneCh);
    const unsigned own = static_cast<unsigned>(a.N) * ncb;  // below 2^24 with the rest's
    const unsigned grid = own + rest_blocks(a.zero_rest, a.T * a.C * static_cast<int64_t>(sizeof(TI)), (1 << 24) - 1 - own);
    if (a.idx && a.N > kScanAlone) k_short_conv_update<TI, W, true><<<grid, kThreads, 0, s>>>(a, ncb);
    else k_short_conv_update<TI, W, false><<<grid, kThreads, 0, s>>>(a, ncb);
    return hipGetLastError();
  }
  const Cover g = cover_of(a.C, a.T);
  const bool ends = what == kFwd ? a.final_state != nullptr : a.dinit != nullptr;
  const int64_t rows = static_cast<int64_t>(a.N) * (W - 1);
  const int64_t tail = ends ? (rows * (a.C / kLaneCh) + kThreads - 1) / kThreads : 0;
  const unsigned grid = static_cast<unsigned>(g.nrb * g.ncb + tail);
  if (grid == 0) return hipSuccess;
  const bool nt = streams_past_caches((what == kFwd ? 2 : 3) * a.T * a.C * static_cast<int64_t>(sizeof(TI)));
  if (what == kFwd) {
    if (nt) k_short_conv<TI, W, true><<<grid, kThreads, 0, s>>>(a, g);
    else k_short_conv<TI, W, false><<<grid, kThreads, 0, s>>>(a, g);
  } else {
    if (nt) k_short_conv_bwd<TI, W, true><<<grid, kThreads, 0, s>>>(a, g);
    else k_short_conv_bwd<TI, W, false><<<grid, kThreads, 0, s>>>(a, g);
  }
  return hipGetLastError();
}
template <typename TI>
hipError_t launch_t(int what, int W, const ShortConvArgs& a, hipStream_t s) {
  return W == 2 ? launch_w<TI, 2>(what, a, s)
                : W == 3 ? launch_w<TI, 3>(what, a, s) : launch_w<TI, 4>(what, a, s);
}
hipError_t launch(int what, int dtype, int W, const ShortConvArgs& a, hipStream_t s) {
  return dtype == 0 ? launch_t<float>(what, W, a, s) : launch_t<bf16>(what, W, a, s);
}

}  // namespace

int64_t short_conv_blocks(int C, int64_t T) { return cover_of(C, T).nrb; }

hipError_t launch_short_conv_fwd(int dtype, int W, const ShortConvArgs& a, hipStream_t s) {
  return launch(kFwd, dtype, W, a, s);
}
hipError_t launch_short_conv_bwd(int dtype, int W, const ShortConvArgs& a, hipStream_t s) {
  return launch(kBwd, dtype, W, a, s);
}
hipError_t launch_short_conv_update(int dtype, int W, const ShortConvArgs& a, hipStream_t s) {
  return launch(kUpdate, dtype, W, a, s);
}

}  // namespace kda
