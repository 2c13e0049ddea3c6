// The short causal convolution in front of the operator: depthwise over the
// channels, W = 2 .. 4 taps, packed sequences, initial and final states; its
// backward; and its decoding form on a pool of states.
//
// With e the W-1 rows of a sequence's state followed by its tokens:
//   p_t = bias + sum_j w_j e_{t+j},  y_t = act(p_t)
//   dp_t = dy_t act'(p_t),  de_r = sum_j w_j dp_{r-j} (+ the final state's
//   gradient on the last W-1 rows),  dw_j = sum_t dp_t e_{t+j}
// All are bound by HBM (about 10 operations per element and direction). A
// thread takes 16 bytes of channels over a run of consecutive tokens, the
// last W-1 rows in registers, so that each row is read once and W-1 rows
// before (and, backward, behind) the run again.
#include "../kda_internal.h"
#include "kda.h"
#include "kda_layer.h"
#include "kda_rows.h"

namespace kda {

namespace {

constexpr int kThreads = 256;

// Threads side by side on the channels of a row (a power of two up to a
// wave); the block's others take further runs.
int channel_lanes(int nvec) {
  int cl = 8;
  while (cl < 64 && cl < nvec) cl *= 2;
  return cl;
}

// How a launch covers [T][C]: `cl` channel lanes, runs of `R` tokens, ncb
// blocks across the channels times nrb along the tokens.
struct Cover {
  int cl, R, ncb;
  int64_t nrb;
};
Cover cover(int nvec, int64_t T, int maxR, int64_t want) {
  Cover c;
  c.cl = channel_lanes(nvec);
  c.ncb = (nvec + c.cl - 1) / c.cl;
  c.R = maxR;
  while (c.R > 8 && nvec * ((T + c.R - 1) / c.R) < want) c.R /= 2;
  const int64_t runs = (T + c.R - 1) / c.R, rpb = kThreads / c.cl;
  c.nrb = (runs + rpb - 1) / rpb;
  return c;
}

// Bounds [s, e) of sequence n, inside [0, T] whatever cu_seqlens holds.
struct Bounds {
  int64_t s, e;
};
__device__ __forceinline__ Bounds bounds(const ShortConvArgs& a, int n) {
  if (!a.cu) return Bounds{0, a.T};
  int64_t s = a.cu[n], e = a.cu[n + 1];
  s = s < 0 ? 0 : (s > a.T ? a.T : s);
  e = e > a.T ? a.T : e;
  return Bounds{s, e < s ? s : e};
}

// Row `tt` of the sequence n that starts at s (tt >= s - (W-1)): a token, or
// a row of the initial state.
template <typename TI, int W>
__device__ __forceinline__ void load_row(const ShortConvArgs& a, int n, int64_t s, int64_t tt, int c,
                                         RowVec<TI>& v) {
  if (tt >= s) {
    v.load(static_cast<const TI*>(a.x) + tt * a.xs + c);
  } else if (a.init) {
    v.load(static_cast<const TI*>(a.init) +
           (static_cast<size_t>(n) * (W - 1) + static_cast<size_t>(W - 1 - (s - tt))) * a.C + c);
  } else {
    v.u = make_uint4(0, 0, 0, 0);
  }
}

// Taps [j][i] of the thread's channels (weight rows [C][W] in order).
template <int N, int W>
__device__ __forceinline__ void load_taps(const ShortConvArgs& a, int c, float (&w)[W][N], float (&b)[N]) {
  float f[N * W];
  load_params<N * W>(a.weight + static_cast<size_t>(c) * W, f);
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][i] = f[i * W + j];
#pragma unroll
  for (int i = 0; i < N; ++i) b[i] = 0.f;
  if (a.bias) load_params<N>(a.bias + c, b);
}

// p = bias + sum of the taps over the window's rows and the newest row x.
template <typename TI, int W, int N = RowVec<TI>::N>
__device__ __forceinline__ void taps(const RowVec<TI> (&win)[W - 1], const RowVec<TI>& x,
                                     const float (&w)[W][N], const float (&b)[N], float (&p)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] = b[i];
#pragma unroll
  for (int j = 0; j < W; ++j) {
    float f[N];
    if (j < W - 1) win[j < W - 1 ? j : 0].get(f);
    else x.get(f);
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] += w[j][i] * f[i];
  }
}
template <typename TI, int W>
__device__ __forceinline__ void shift(RowVec<TI> (&win)[W - 1], const RowVec<TI>& x) {
#pragma unroll
  for (int j = 0; j + 1 < W - 1; ++j) win[j] = win[j + 1];
  win[W - 2] = x;
}

// Row len + i of e for i in [0, W-1): the final state (threads past the runs'
// blocks, one per 16 bytes).
template <typename TI, int W>
__device__ __forceinline__ void copy_final(const ShortConvArgs& a, int64_t id) {
  constexpr int N = RowVec<TI>::N;
  const int nvec = a.C / N;
  const int64_t row = id / nvec;
  const int c = static_cast<int>(id - row * nvec) * N;
  const int n = static_cast<int>(row / (W - 1)), i = static_cast<int>(row % (W - 1));
  if (n >= a.N) return;
  const Bounds q = bounds(a, n);
  RowVec<TI> v;
  load_row<TI, W>(a, n, q.s, q.e - (W - 1) + i, c, v);
  v.store(static_cast<TI*>(a.final_state) + static_cast<size_t>(row) * a.C + c);
}

template <typename TI, int W>
__global__ void __launch_bounds__(kThreads) k_short_conv(ShortConvArgs a, Cover g) {
  using RV = RowVec<TI>;
  constexpr int N = RV::N, U = 4;
  const int64_t rb = blockIdx.x / g.ncb;
  if (rb >= g.nrb) {
    copy_final<TI, W>(a, (static_cast<int64_t>(blockIdx.x) - g.nrb * g.ncb) * kThreads + threadIdx.x);
    return;
  }
  const int vec = static_cast<int>(blockIdx.x % g.ncb) * g.cl + threadIdx.x % g.cl;
  const int64_t t0 = (rb * (kThreads / g.cl) + threadIdx.x / g.cl) * g.R;
  const int64_t t1 = t0 + g.R < a.T ? t0 + g.R : a.T;
  const int c = vec * N;
  if (t0 >= t1 || c >= a.C) return;
  float w[W][N], b[N];
  load_taps<N, W>(a, c, w, b);
  int n = a.cu && a.N > 0 ? find_seq(a.cu, a.N, static_cast<int>(t0)) : 0;
  Bounds q = a.N > 0 ? bounds(a, n) : Bounds{0, 0};
  RV win[W - 1];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) win[j].u = make_uint4(0, 0, 0, 0);
  if (t0 > q.s && t0 < q.e) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_row<TI, W>(a, n, q.s, t0 - (W - 1) + j, c, win[j]);
  }
  const TI* x = static_cast<const TI*>(a.x) + c;
  TI* y = static_cast<TI*>(a.y) + c;
  for (int64_t tb = t0; tb < t1; tb += U) {
    RV xv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) xv[u].load(x + (tb + u < t1 ? tb + u : t1 - 1) * a.xs);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = tb + u;
      if (t >= t1) break;
      bool fresh = t == q.s;
      while (t >= q.e && n + 1 < a.N) {
        q = bounds(a, ++n);
        fresh = true;
      }
      if (fresh && t >= q.s && t < q.e) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) load_row<TI, W>(a, n, q.s, t - (W - 1) + j, c, win[j]);
      }
      float p[N];
      taps<TI, W>(win, xv[u], w, b, p);
      if (a.act == KDA_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] *= sigmoidf(p[i]);
      }
      RV out;
      out.set(p);
      if (t < q.s || t >= q.e) out.u = make_uint4(0, 0, 0, 0);  // a row of no sequence
      out.store(y + static_cast<size_t>(t) * a.C);
      shift<TI, W>(win, xv[u]);
    }
  }
}

// Backward. A run owns its tokens' rows of dx, its share of dweight and dbias,
// and the initial-state rows of the sequences that start in it. Walking its
// tokens and up to W-1 behind them (of the same sequence), it keeps the W
// rows whose gradient is still incomplete in `acc`: the token t adds
// w_j dp_t to row t + j of e and completes row t. The last W-1 rows are
// completed at the sequence's end, where the final state's gradient joins
// them. An empty sequence's state gradient passes through (threads past the
// runs' blocks).
template <typename TI, int W>
__global__ void __launch_bounds__(kThreads) k_short_conv_bwd(ShortConvArgs a, Cover g) {
  using RV = RowVec<TI>;
  constexpr int N = RV::N;
  __shared__ __align__(16) float sm[kThreads * N];
  const int64_t rb = blockIdx.x / g.ncb;
  if (rb >= g.nrb) {
    const int64_t id = (static_cast<int64_t>(blockIdx.x) - g.nrb * g.ncb) * kThreads + threadIdx.x;
    const int nvec = a.C / N;
    const int64_t row = id / nvec;
    const int n = static_cast<int>(row / (W - 1));
    if (n >= a.N) return;
    const Bounds q = bounds(a, n);
    if (q.e > q.s) return;
    const size_t at = static_cast<size_t>(row) * a.C + static_cast<size_t>(id - row * nvec) * N;
    RV v;
    v.u = make_uint4(0, 0, 0, 0);
    if (a.dfinal) v.load(static_cast<const TI*>(a.dfinal) + at);
    v.store(static_cast<TI*>(a.dinit) + at);
    return;
  }
  const int cl0 = threadIdx.x % g.cl, rsub = threadIdx.x / g.cl;
  const int cb = static_cast<int>(blockIdx.x % g.ncb);
  const int c = (cb * g.cl + cl0) * N;
  const int64_t t0 = (rb * (kThreads / g.cl) + rsub) * g.R;
  const int64_t t1 = t0 + g.R < a.T ? t0 + g.R : a.T;
  float w[W][N], b[N], dw[W][N], db[N], acc[W][N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    db[i] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][i] = acc[j][i] = 0.f;
  }
  if (t0 < t1 && c < a.C) {
    load_taps<N, W>(a, c, w, b);
    int n = a.cu && a.N > 0 ? find_seq(a.cu, a.N, static_cast<int>(t0)) : 0;
    Bounds q = a.N > 0 ? bounds(a, n) : Bounds{0, 0};
    const TI* x = static_cast<const TI*>(a.x) + c;
    const TI* dy = static_cast<const TI*>(a.dy) + c;
    TI* dx = static_cast<TI*>(a.dx) + c;
    RV win[W - 1];
    bool fresh = true;  // the window has to be read
    // the gradient of row r (counted from the sequence's state) is complete
    auto emit = [&](int64_t r, const float (&v)[N], bool last) {
      const int64_t tt = q.s + r - (W - 1);
      const bool token = r >= W - 1;
      if (token ? (tt < t0 || tt >= t1) : (!a.dinit || q.s < t0 || q.s >= t1)) return;
      float f[N];
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = v[i];
      if (last && a.dfinal) {
        RV d;
        float e[N];
        d.load(static_cast<const TI*>(a.dfinal) +
               (static_cast<size_t>(n) * (W - 1) + static_cast<size_t>(r - (q.e - q.s))) * a.C + c);
        d.get(e);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] += e[i];
      }
      RV out;
      out.set(f);
      out.store(token ? dx + static_cast<size_t>(tt) * a.C
                      : static_cast<TI*>(a.dinit) + (static_cast<size_t>(n) * (W - 1) + r) * a.C + c);
    };
    for (int64_t t = t0; t < t1 + (W - 1); ++t) {
      if (t >= t1 && (t >= q.e || t >= a.T)) break;  // behind the run: only its last sequence
      while (t >= q.e && n + 1 < a.N) {
        q = bounds(a, ++n);
        fresh = true;
      }
      if (t < q.s || t >= q.e) {  // a row of no sequence
        if (t >= t1) break;
        RV z;
        z.u = make_uint4(0, 0, 0, 0);
        z.store(dx + static_cast<size_t>(t) * a.C);
        continue;
      }
      if (fresh) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) load_row<TI, W>(a, n, q.s, t - (W - 1) + j, c, win[j]);
        fresh = false;
      }
      RV xv, dv;
      xv.load(x + t * a.xs);
      dv.load(dy + static_cast<size_t>(t) * a.C);
      float p[N], d[N];
      dv.get(d);
      if (a.act == KDA_ACT_SILU) {
        taps<TI, W>(win, xv, w, b, p);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float s = sigmoidf(p[i]);
          d[i] *= s * (1.f + p[i] * (1.f - s));
        }
      }
#pragma unroll
      for (int j = 0; j < W; ++j) {
        float f[N];
        if (j < W - 1) win[j < W - 1 ? j : 0].get(f);
        else xv.get(f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          acc[j][i] += w[j][i] * d[i];
          if (t < t1) dw[j][i] += f[i] * d[i];
        }
      }
      if (t < t1) {
#pragma unroll
        for (int i = 0; i < N; ++i) db[i] += d[i];
      }
      emit(t - q.s, acc[0], false);
#pragma unroll
      for (int j = 0; j < W; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) acc[j][i] = j + 1 < W ? acc[j + 1 < W ? j + 1 : 0][i] : 0.f;
      shift<TI, W>(win, xv);
      if (t == q.e - 1) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
          emit(q.e - q.s + j, acc[j], true);
#pragma unroll
          for (int i = 0; i < N; ++i) acc[j][i] = 0.f;
        }
      }
    }
  }
  // join the block's runs: one partial row of dweight [C][W], dbias [C]
  const int cols = g.cl * N, runs = kThreads / g.cl;
  float* part = a.partials + static_cast<size_t>(rb) * a.C * (W + 1);
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    if (j) __syncthreads();
    store_params<N>(sm + rsub * cols + cl0 * N, j < W ? dw[j < W ? j : 0] : db);
    __syncthreads();
    for (int k = threadIdx.x; k < cols; k += kThreads) {
      const int cc = cb * cols + k;
      if (cc >= a.C) break;
      float t = 0.f;
      for (int r = 0; r < runs; ++r) t += sm[r * cols + k];
      part[j < W ? static_cast<size_t>(cc) * W + j : static_cast<size_t>(a.C) * W + cc] = t;
    }
  }
}

// Decoding: a thread takes 16 bytes of channels of one sequence, its state
// rows in registers over the sequence's tokens.
template <typename TI, int W>
__global__ void __launch_bounds__(kThreads) k_short_conv_update(ShortConvArgs a) {
  using RV = RowVec<TI>;
  constexpr int N = RV::N;
  const int nvec = a.C / N;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int n = static_cast<int>(id / nvec), c = static_cast<int>(id - static_cast<int64_t>(n) * nvec) * N;
  if (n >= a.N) return;
  Bounds q{n, n + 1};
  if (a.cu) q = bounds(a, n);
  if (q.s >= q.e) return;
  const int64_t slot = a.idx ? a.idx[n] : n;
  TI* y = static_cast<TI*>(a.y) + c;
  if (slot < 0 || slot >= a.n_slots) {  // a padded sequence
    RV z;
    z.u = make_uint4(0, 0, 0, 0);
    for (int64_t t = q.s; t < q.e; ++t) z.store(y + static_cast<size_t>(t) * a.C);
    return;
  }
  TI* st = static_cast<TI*>(a.state) + static_cast<size_t>(slot) * (W - 1) * a.C + c;
  RV win[W - 1];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) win[j].load(st + static_cast<size_t>(j) * a.C);
  float w[W][N], b[N];
  load_taps<N, W>(a, c, w, b);
  for (int64_t t = q.s; t < q.e; ++t) {
    RV x, out;
    x.load(static_cast<const TI*>(a.x) + t * a.xs + c);
    float p[N];
    taps<TI, W>(win, x, w, b, p);
    if (a.act == KDA_ACT_SILU) {
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] *= sigmoidf(p[i]);
    }
    out.set(p);
    out.store(y + static_cast<size_t>(t) * a.C);
    shift<TI, W>(win, x);
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) win[j].store(st + static_cast<size_t>(j) * a.C);
}

enum { kFwd, kBwd, kUpdate };

int vec_of(int dtype) { return dtype == 0 ? 4 : 8; }

// Runs of up to 64 tokens, shorter while fewer than 2^17 threads (two waves
// per SIMD) would run.
Cover cover_of(int dtype, int C, int64_t T) { return cover(C / vec_of(dtype), T, 64, 1 << 17); }

template <typename TI, int W>
hipError_t launch_w(int what, int dtype, const ShortConvArgs& a, hipStream_t s) {
  const int64_t nvec = a.C / RowVec<TI>::N;
  if (what == kUpdate) {
    const int64_t blocks = (a.N * nvec + kThreads - 1) / kThreads;
    k_short_conv_update<TI, W><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  const Cover g = cover_of(dtype, a.C, a.T);
  const bool ends = what == kFwd ? a.final_state != nullptr : a.dinit != nullptr;
  const int64_t tail = ends ? (a.N * (W - 1) * nvec + kThreads - 1) / kThreads : 0;
  const unsigned grid = static_cast<unsigned>(g.nrb * g.ncb + tail);
  if (grid == 0) return hipSuccess;
  if (what == kFwd) k_short_conv<TI, W><<<grid, kThreads, 0, s>>>(a, g);
  else k_short_conv_bwd<TI, W><<<grid, kThreads, 0, s>>>(a, g);
  return hipGetLastError();
}
template <typename TI>
hipError_t launch_t(int what, int dtype, int W, const ShortConvArgs& a, hipStream_t s) {
  return W == 2 ? launch_w<TI, 2>(what, dtype, a, s)
                : W == 3 ? launch_w<TI, 3>(what, dtype, a, s) : launch_w<TI, 4>(what, dtype, a, s);
}
hipError_t launch(int what, int dtype, int W, const ShortConvArgs& a, hipStream_t s) {
  return dtype == 0 ? launch_t<float>(what, dtype, W, a, s) : launch_t<bf16>(what, dtype, W, a, s);
}

}  // namespace

int64_t short_conv_blocks(int dtype, int C, int64_t T) { return cover_of(dtype, C, T).nrb; }

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
