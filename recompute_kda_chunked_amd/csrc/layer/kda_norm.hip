// The norms around the operator: behind it, per head, with the output gate
// (gated norm), and between two blocks, with the gate, the residual scale and
// the residual stream (block norm); and the sum of per-block parameter
// gradients.
//
// All are bound by HBM: a few operations per element, each input read once
// and each output written once (the backward recomputes the norms from the
// inputs, so nothing is kept from the forward). Sums of squares, gate values
// and parameter gradients are fp32; every output is rounded once.
#include <cfloat>

#include "../kda_internal.h"
#include "kda.h"
#include "kda_layer.h"
#include "kda_rows.h"

namespace kda {

namespace {

// ------------------------------------------------------------ parameter sums

// A block takes CL columns with 1024 / CL row lanes; each lane sums every
// (1024 / CL)-th partial row, then the lanes' sums of a column are added in
// order, first within groups of 16. Few columns take narrow blocks, so that
// enough lanes share the rows.
template <int CL>
__global__ void __launch_bounds__(1024) k_param_reduce(ParamReduceArgs a) {
  constexpr int RL = 1024 / CL;
  __shared__ float sm[RL][CL + 1];
  const int M = a.n0 + a.n1, cl = threadIdx.x % CL, rl = threadIdx.x / CL;
  const int c = blockIdx.x * CL + cl;
  float s = 0.f;
  if (c < M) {
#pragma unroll 8
    for (int64_t r = rl; r < a.nb; r += RL) s += a.partials[r * M + c];
  }
  sm[rl][cl] = s;
  __syncthreads();
  if (rl < RL / 16) {
    s = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) s += sm[rl * 16 + r][cl];
  }
  __syncthreads();
  if (rl < RL / 16) sm[rl][cl] = s;
  __syncthreads();
  if (rl == 0 && c < M) {
    s = 0.f;
#pragma unroll
    for (int r = 0; r < RL / 16; ++r) s += sm[r][cl];
    if (c < a.n0) a.out0[c] = s;
    else if (a.out1) a.out1[c - a.n0] = s;
  }
}

// ------------------------------------------------------------------ gated norm

// Sum over the N lanes that hold one row (N = 8 .. 64, aligned).
template <int N>
__device__ __forceinline__ float row_sum(float x) {
  if constexpr (N == 64) return sum_wave(x);
  else return group_sum<N>(x);
}

// 1 - s for s = sigmoidf(g), as e^-g s: the difference loses its digits where s
// is next to 1 (half of them at g = 9, the last at 17). Where e^-g overflows, 1.
__device__ __forceinline__ float sigmoid_rest(float g, float s) {
  const float e = __expf(-g);
  return e > FLT_MAX ? 1.f : e * s;
}

// act(g) and its derivative.
__device__ __forceinline__ float act_value(int act, float g, float s) {
  return act == KDA_ACT_SILU ? g * s : s;
}
__device__ __forceinline__ float act_slope(int act, float g, float s) {
  return act == KDA_ACT_SILU ? s * (1.f + g * (1.f - s)) : s * sigmoid_rest(g, s);
}

// A row lies across V / N consecutive lanes, one 16-byte vector each, so a
// wave instruction reads 1 KB of adjacent rows.
template <typename TI, int V, bool NT>
__global__ void __launch_bounds__(256) k_gated_norm(GatedNormArgs a) {
  using RV = RowVec<TI>;
  constexpr int N = RV::N, LPR = V / N, RPB = 256 / LPR;
  const int c = (threadIdx.x % LPR) * N;
  float w[N];
  load_params<N>(a.weight + c, w);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + threadIdx.x / LPR; row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * RPB) {
    const size_t at = static_cast<size_t>(row) * V + c;
    RV vo, vg;
    vo.template load<NT>(static_cast<const TI*>(a.o) + at);
    vg.template load<NT>(static_cast<const TI*>(a.gate) + at);
    float o[N], g[N], y[N], ss = 0.f;
    vo.get(o);
    vg.get(g);
#pragma unroll
    for (int i = 0; i < N; ++i) ss += o[i] * o[i];
    const float r = 1.f / sqrtf(row_sum<LPR>(ss) * (1.f / V) + a.eps);
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = o[i] * r * w[i] * act_value(a.act, g[i], sigmoidf(g[i]));
    vo.set(y);
    vo.template store<NT>(static_cast<TI*>(a.y) + at);
  }
}

// With n = o r and dn = dy w act(g): do = r (dn - n mean(dn n)), and
// mean(dn n) = r mean(dn o), so both sums of a row are taken together. A
// lane keeps its channels over all its rows, so dweight adds up in registers;
// the block's row groups are joined through LDS into one partial row.
template <typename TI, int V, bool NT>
__global__ void __launch_bounds__(256) k_gated_norm_bwd(GatedNormArgs a) {
  using RV = RowVec<TI>;
  constexpr int N = RV::N, LPR = V / N, RPB = 256 / LPR;
  __shared__ __align__(16) float sm[RPB][V];
  const int c = (threadIdx.x % LPR) * N, sub = threadIdx.x / LPR;
  float w[N], dw[N];
  load_params<N>(a.weight + c, w);
#pragma unroll
  for (int i = 0; i < N; ++i) dw[i] = 0.f;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + sub; row < a.rows;
       row += static_cast<int64_t>(gridDim.x) * RPB) {
    const size_t at = static_cast<size_t>(row) * V + c;
    RV vo, vg, vd;
    vo.template load<NT>(static_cast<const TI*>(a.o) + at);
    vg.template load<NT>(static_cast<const TI*>(a.gate) + at);
    vd.template load<NT>(static_cast<const TI*>(a.dy) + at);
    float o[N], g[N], d[N], s[N], ss = 0.f, sd = 0.f;
    vo.get(o);
    vg.get(g);
    vd.get(d);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s[i] = sigmoidf(g[i]);
      ss += o[i] * o[i];
      sd += d[i] * w[i] * act_value(a.act, g[i], s[i]) * o[i];
    }
    const float r = 1.f / sqrtf(row_sum<LPR>(ss) * (1.f / V) + a.eps);
    const float m = row_sum<LPR>(sd) * (1.f / V) * r * r;  // r mean(dn n)
    float x[N], y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float av = act_value(a.act, g[i], s[i]), n = o[i] * r;
      x[i] = r * (d[i] * w[i] * av) - m * n;
      y[i] = d[i] * n * w[i] * act_slope(a.act, g[i], s[i]);
      dw[i] += d[i] * n * av;
    }
    vo.set(x);
    vo.template store<NT>(static_cast<TI*>(a.d_o) + at);
    vg.set(y);
    vg.template store<NT>(static_cast<TI*>(a.dgate) + at);
  }
  store_params<N>(&sm[sub][c], dw);
  __syncthreads();
  if (threadIdx.x < V) {
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < RPB; ++r) t += sm[r][threadIdx.x];
    a.partials[static_cast<size_t>(blockIdx.x) * V + threadIdx.x] = t;
  }
}

// ------------------------------------------------------------------ block norm

// Sums of K values over the block, every thread receiving them. Consecutive
// calls alternate between two LDS buffers (`phase`), so one barrier each is
// enough: a buffer is written again only after the barrier of the call in
// between, which every thread reaches after its reads.
template <int K>
__device__ __forceinline__ void block_sum(float (&v)[K], float (&sm)[2][2][8], int& phase) {
  const int nw = blockDim.x >> 6, w = threadIdx.x >> 6;
  float(&b)[2][8] = sm[phase & 1];
  ++phase;
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = sum_wave(v[k]);
  if (nw == 1) return;
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) b[k][w] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float t = b[k][0];
    for (int i = 1; i < nw; ++i) t += b[k][i];
    v[k] = t;
  }
}

// One block per token (a launch of 2^22 blocks takes more in turn), the row's
// NV 16-byte vectors per thread in registers; vector j of thread t is number
// j * threads + t of the row.
template <typename TI, int NV, int GATE, bool POST, bool NT>
__global__ void __launch_bounds__(512) k_block_norm(BlockNormArgs a) {
  using RV = RowVec<TI>;
  constexpr int N = RV::N;
  __shared__ float sm[2][2][8];
  int phase = 0;
  const int nvec = a.D / N;
  const float inv = 1.f / a.D;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t row = static_cast<size_t>(t) * a.D;
    RV vx[NV], vy[NV], vg[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = j * blockDim.x + threadIdx.x;
      vx[j].u = vy[j].u = vg[j].u = make_uint4(0, 0, 0, 0);
      if (v < nvec) {
        vy[j].template load<NT>(static_cast<const TI*>(a.y) + row + v * N);
        vx[j].template load<NT>(static_cast<const TI*>(a.x) + row + v * N);
        if constexpr (GATE == KDA_BLOCK_GATE_CHANNEL) vg[j].template load<NT>(static_cast<const TI*>(a.gate) + row + v * N);
      }
    }
    float gt = 1.f;
    if constexpr (GATE == KDA_BLOCK_GATE_TOKEN) gt = sigmoidf(to_f(static_cast<const TI*>(a.gate)[t]));
    float ry = 1.f;
    if constexpr (POST) {
      float s[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float y[N];
        vy[j].get(y);
#pragma unroll
        for (int i = 0; i < N; ++i) s[0] += y[i] * y[i];
      }
      block_sum<1>(s, sm, phase);
      ry = 1.f / sqrtf(s[0] * inv + a.eps);
    }
    float xo[NV][N], s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = j * blockDim.x + threadIdx.x;
      float x[N], y[N], g[N], w[N];
      vx[j].get(x);
      vy[j].get(y);
      vg[j].get(g);
      if constexpr (POST)
        if (v < nvec) load_params<N>(a.w_post + v * N, w);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float z = y[i] * (a.scale * gt);
        if constexpr (POST) z *= v < nvec ? ry * w[i] : 0.f;
        if constexpr (GATE == KDA_BLOCK_GATE_CHANNEL) z *= sigmoidf(g[i]);
        xo[j][i] = x[i] + z;
        s[0] += xo[j][i] * xo[j][i];
      }
      if (v < nvec) {
        vx[j].set(xo[j]);
        vx[j].template store<NT>(static_cast<TI*>(a.x_out) + row + v * N);
      }
    }
    block_sum<1>(s, sm, phase);
    const float rx = 1.f / sqrtf(s[0] * inv + a.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = j * blockDim.x + threadIdx.x;
      if (v < nvec) {
        float w[N], h[N];
        load_params<N>(a.w_pre + v * N, w);
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = xo[j][i] * rx * w[i];
        vx[j].set(h);
        vx[j].template store<NT>(static_cast<TI*>(a.h) + row + v * N);
      }
    }
  }
}

// The backward of one token, with n_x = x_out r_x and n_y = y r_y:
//   dX = dx_out + r_x (dh w_pre - n_x mean(dh w_pre n_x)) = dx
//   dz = scale sigmoid(gate) dX,  dgate = scale z sigmoid'(gate) dX
//   dy = r_y (dz w_post - n_y mean(dz w_post n_y))
// Three block sums in turn: y^2; x_out^2 with dh w_pre x_out; dz w_post n_y
// with z dX (a per-token gate). A block takes every gridDim-th token and keeps
// its threads' channels of dw_pre and dw_post in registers, one partial row
// per block at the end.
template <typename TI, int NV, int GATE, bool POST, bool NT>
__global__ void __launch_bounds__(512) k_block_norm_bwd(BlockNormArgs a) {
  using RV = RowVec<TI>;
  constexpr int N = RV::N;
  __shared__ float sm[2][2][8];
  int phase = 0;
  const int nvec = a.D / N;
  const float inv = 1.f / a.D;
  float wpre[NV][N], wpost[NV][N], dwpre[NV][N], dwpost[NV][N];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = j * blockDim.x + threadIdx.x;
#pragma unroll
    for (int i = 0; i < N; ++i) wpre[j][i] = wpost[j][i] = dwpre[j][i] = dwpost[j][i] = 0.f;
    if (v < nvec) {
      load_params<N>(a.w_pre + v * N, wpre[j]);
      if constexpr (POST) load_params<N>(a.w_post + v * N, wpost[j]);
    }
  }
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const size_t row = static_cast<size_t>(t) * a.D;
    RV vx[NV], vy[NV], vg[NV], vd[NV], vh[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = j * blockDim.x + threadIdx.x;
      vx[j].u = vy[j].u = vg[j].u = vd[j].u = vh[j].u = make_uint4(0, 0, 0, 0);
      if (v < nvec) {
        vy[j].template load<NT>(static_cast<const TI*>(a.y) + row + v * N);
        vx[j].template load<NT>(static_cast<const TI*>(a.x) + row + v * N);
        if constexpr (GATE == KDA_BLOCK_GATE_CHANNEL) vg[j].template load<NT>(static_cast<const TI*>(a.gate) + row + v * N);
        if (a.dh) vh[j].template load<NT>(static_cast<const TI*>(a.dh) + row + v * N);
        if (a.dx_out) vd[j].template load<NT>(static_cast<const TI*>(a.dx_out) + row + v * N);
      }
    }
    float raw = 0.f, gt = 1.f;
    if constexpr (GATE == KDA_BLOCK_GATE_TOKEN) {
      raw = to_f(static_cast<const TI*>(a.gate)[t]);
      gt = sigmoidf(raw);
    }
    float ry = 1.f;
    if constexpr (POST) {
      float s[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float y[N];
        vy[j].get(y);
#pragma unroll
        for (int i = 0; i < N; ++i) s[0] += y[i] * y[i];
      }
      block_sum<1>(s, sm, phase);
      ry = 1.f / sqrtf(s[0] * inv + a.eps);
    }
    float xo[NV][N], s2[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float x[N], y[N], g[N], dh[N];
      vx[j].get(x);
      vy[j].get(y);
      vg[j].get(g);
      vh[j].get(dh);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float z = y[i] * (a.scale * gt);
        if constexpr (POST) z *= ry * wpost[j][i];
        if constexpr (GATE == KDA_BLOCK_GATE_CHANNEL) z *= sigmoidf(g[i]);
        xo[j][i] = x[i] + z;
        s2[0] += xo[j][i] * xo[j][i];
        s2[1] += dh[i] * wpre[j][i] * xo[j][i];
      }
    }
    block_sum<2>(s2, sm, phase);
    const float rx = 1.f / sqrtf(s2[0] * inv + a.eps);
    const float mx = s2[1] * inv * rx * rx;  // r_x mean(dh w_pre n_x)
    float dz[NV][N], s3[2] = {0.f, 0.f};     // dz before the scale and a per-token gate
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = j * blockDim.x + threadIdx.x;
      float y[N], g[N], d[N], dh[N], dg[N];
      vy[j].get(y);
      vg[j].get(g);
      vd[j].get(d);
      vh[j].get(dh);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float n = xo[j][i] * rx;
        d[i] += rx * (dh[i] * wpre[j][i]) - mx * n;
        dwpre[j][i] += dh[i] * n;
        const float z = POST ? y[i] * ry * wpost[j][i] : y[i];
        float e = d[i];
        if constexpr (GATE == KDA_BLOCK_GATE_CHANNEL) {
          const float s = sigmoidf(g[i]);
          dg[i] = a.scale * z * e * s * sigmoid_rest(g[i], s);
          e *= s;
        }
        dz[j][i] = e;
        s3[0] += e * z;
      }
      if (v < nvec) {
        vd[j].set(d);
        vd[j].template store<NT>(static_cast<TI*>(a.dx) + row + v * N);
        if constexpr (GATE == KDA_BLOCK_GATE_CHANNEL) {
          vg[j].set(dg);
          vg[j].template store<NT>(static_cast<TI*>(a.dgate) + row + v * N);
        }
      }
    }
    // sum of dz w_post n_y and of z dX are one sum, up to factors: with the
    // scale c = scale * (per-token gate), mean(dz w_post n_y) = c mean(e z)
    const float cz = a.scale * gt;
    if constexpr (POST || GATE == KDA_BLOCK_GATE_TOKEN) {
      float s1[1] = {s3[0]};
      block_sum<1>(s1, sm, phase);
      s3[0] = s1[0];
      if constexpr (GATE == KDA_BLOCK_GATE_TOKEN)
        if (threadIdx.x == 0)
          static_cast<TI*>(a.dgate)[t] = from_f<TI>(a.scale * s3[0] * gt * sigmoid_rest(raw, gt));
    }
    const float my = s3[0] * inv * cz * ry;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = j * blockDim.x + threadIdx.x;
      float y[N];
      vy[j].get(y);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float d = cz * dz[j][i];
        if constexpr (POST) {
          const float n = y[i] * ry;
          dwpost[j][i] += d * n;
          y[i] = ry * (d * wpost[j][i]) - my * n;
        } else {
          y[i] = d;
        }
      }
      if (v < nvec) {
        vy[j].set(y);
        vy[j].template store<NT>(static_cast<TI*>(a.dy) + row + v * N);
      }
    }
  }
  float* p = a.partials + static_cast<size_t>(blockIdx.x) * (POST ? 2 : 1) * a.D;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = j * blockDim.x + threadIdx.x;
    if (v < nvec) {
      if constexpr (POST) store_params<N>(p + v * N, dwpost[j]);
      store_params<N>(p + (POST ? a.D : 0) + v * N, dwpre[j]);
    }
  }
}

// A row as threads x values per thread: 8 values while 256 threads hold the
// row so, else 16 (D <= 8192: up to 512 threads).
struct RowShape {
  int values, threads;
  RowShape(int dtype, int D) : values(D <= 2048 ? 8 : 16) {
    const int n = dtype == KDA_F32 ? 4 : 8, nvec = D / n, nv = values / n;
    threads = ((nvec + nv - 1) / nv + 63) / 64 * 64;
  }
};

template <typename TI, int NV, int GATE, bool NT>
hipError_t launch_block_n(bool bwd, int threads, const BlockNormArgs& a, hipStream_t s) {
  const unsigned grid = bwd ? block_norm_blocks(sizeof(TI) == 4 ? KDA_F32 : KDA_BF16, a.D, a.T) : static_cast<unsigned>(a.T < (1 << 22) ? a.T : 1 << 22);
  if (bwd) {
    if (a.w_post) k_block_norm_bwd<TI, NV, GATE, true, NT><<<grid, threads, 0, s>>>(a);
    else k_block_norm_bwd<TI, NV, GATE, false, NT><<<grid, threads, 0, s>>>(a);
  } else {
    if (a.w_post) k_block_norm<TI, NV, GATE, true, NT><<<grid, threads, 0, s>>>(a);
    else k_block_norm<TI, NV, GATE, false, NT><<<grid, threads, 0, s>>>(a);
  }
  return hipGetLastError();
}
template <typename TI, int NV, int GATE>
hipError_t launch_block_g(bool bwd, int threads, const BlockNormArgs& a, hipStream_t s) {
  // x, y and two gradients in; x_out and h, or dx and dy out; the gate and its gradient
  const int64_t rows = bwd ? 4 + !!a.dx_out + !!a.dh : 4;
  const int64_t gates = GATE == KDA_BLOCK_GATE_CHANNEL ? (bwd ? 2 : 1) : 0;
  return streams_past_caches((rows + gates) * a.T * a.D * static_cast<int64_t>(sizeof(TI)))
             ? launch_block_n<TI, NV, GATE, true>(bwd, threads, a, s)
             : launch_block_n<TI, NV, GATE, false>(bwd, threads, a, s);
}
template <typename TI, int NV>
hipError_t launch_block_v(bool bwd, int gate, int threads, const BlockNormArgs& a, hipStream_t s) {
  if (gate == KDA_BLOCK_GATE_TOKEN) return launch_block_g<TI, NV, KDA_BLOCK_GATE_TOKEN>(bwd, threads, a, s);
  if (gate == KDA_BLOCK_GATE_CHANNEL) return launch_block_g<TI, NV, KDA_BLOCK_GATE_CHANNEL>(bwd, threads, a, s);
  return launch_block_g<TI, NV, KDA_BLOCK_GATE_NONE>(bwd, threads, a, s);
}
hipError_t launch_block(int dtype, int gate, bool bwd, const BlockNormArgs& a, hipStream_t s) {
  const RowShape r(dtype, a.D);
  if (dtype == KDA_F32)
    return r.values == 8 ? launch_block_v<float, 2>(bwd, gate, r.threads, a, s)
                         : launch_block_v<float, 4>(bwd, gate, r.threads, a, s);
  return r.values == 8 ? launch_block_v<bf16, 1>(bwd, gate, r.threads, a, s)
                       : launch_block_v<bf16, 2>(bwd, gate, r.threads, a, s);
}

template <typename TI, int V, bool NT>
hipError_t launch_gated_n(bool bwd, const GatedNormArgs& a, int blocks, hipStream_t s) {
  if (bwd) k_gated_norm_bwd<TI, V, NT><<<blocks, 256, 0, s>>>(a);
  else k_gated_norm<TI, V, NT><<<blocks, 256, 0, s>>>(a);
  return hipGetLastError();
}
template <typename TI, int V>
hipError_t launch_gated(bool bwd, const GatedNormArgs& a, int blocks, hipStream_t s) {
  return streams_past_caches((bwd ? 5 : 3) * a.rows * V * static_cast<int64_t>(sizeof(TI)))
             ? launch_gated_n<TI, V, true>(bwd, a, blocks, s)
             : launch_gated_n<TI, V, false>(bwd, a, blocks, s);
}
hipError_t launch_gated_t(int dtype, int V, bool bwd, const GatedNormArgs& a, int blocks, hipStream_t s) {
  if (dtype == KDA_F32)
    return V == 64 ? launch_gated<float, 64>(bwd, a, blocks, s)
                   : V == 128 ? launch_gated<float, 128>(bwd, a, blocks, s)
                              : launch_gated<float, 256>(bwd, a, blocks, s);
  return V == 64 ? launch_gated<bf16, 64>(bwd, a, blocks, s)
                 : V == 128 ? launch_gated<bf16, 128>(bwd, a, blocks, s)
                            : launch_gated<bf16, 256>(bwd, a, blocks, s);
}
int64_t gated_groups(int dtype, int V, int64_t rows) {
  const int rpb = 256 / (V / (dtype == KDA_F32 ? 4 : 8));
  return (rows + rpb - 1) / rpb;
}

}  // namespace

hipError_t launch_param_reduce(const ParamReduceArgs& a, hipStream_t s) {
  const int M = a.n0 + a.n1;
  if (M <= 1024) k_param_reduce<4><<<(M + 3) / 4, 1024, 0, s>>>(a);
  else if (M <= 16384) k_param_reduce<32><<<(M + 31) / 32, 1024, 0, s>>>(a);
  else k_param_reduce<64><<<(M + 63) / 64, 1024, 0, s>>>(a);
  return hipGetLastError();
}

// Blocks of the backward kernels, which loop over rows: enough for every CU
// to hold several, few enough that their partial sums stay small.
int gated_norm_blocks(int dtype, int V, int64_t rows) {
  const int64_t g = gated_groups(dtype, V, rows);
  return static_cast<int>(g < 1024 ? g : 1024);
}
int block_norm_blocks(int dtype, int D, int64_t T) {
  const int values = RowShape(dtype, D).values;
  const int64_t b = 256 * (values == 16 ? 8 : 16) / (RowShape(dtype, D).threads / 64);
  return static_cast<int>(T < b ? T : b);
}

hipError_t launch_gated_norm_fwd(int dtype, int V, const GatedNormArgs& a, hipStream_t s) {
  const int64_t g = gated_groups(dtype, V, a.rows);
  return launch_gated_t(dtype, V, false, a, static_cast<int>(g < 65536 ? g : 65536), s);
}
hipError_t launch_gated_norm_bwd(int dtype, int V, const GatedNormArgs& a, hipStream_t s) {
  return launch_gated_t(dtype, V, true, a, gated_norm_blocks(dtype, V, a.rows), s);
}
hipError_t launch_block_norm_fwd(int dtype, int gate, const BlockNormArgs& a, hipStream_t s) {
  return launch_block(dtype, gate, false, a, s);
}
hipError_t launch_block_norm_bwd(int dtype, int gate, const BlockNormArgs& a, hipStream_t s) {
  return launch_block(dtype, gate, true, a, s);
}

}  // namespace kda
