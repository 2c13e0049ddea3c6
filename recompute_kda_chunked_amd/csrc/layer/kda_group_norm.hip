// Group norm over the channels of each token, with an activation or an
// activated gate, forward and backward.
//
// Bound by HBM: each row read once and written once, the backward's norms
// recomputed from x and the gate. A group of W channels lies across a slot of
// `lp` lanes (a power of two up to a wave, or the whole block), NV 16-byte
// vectors a lane; slots keep their group over all their rows, so weights and
// their gradients stay in registers. Means are taken off before the squares
// are added up. Sums are fp32, every output is rounded once. Measured at 8192 rows
// of 4096 bf16 channels, groups of 512 with a gate: forward 35 us (5.8 TB/s),
// backward 58 (5.8), the rows past the caches; 4097 x 2560 in groups of
// 64 without a gate, in the caches, 15 (2.8): of the two blocks of a row the second
// has 8 of its 32 places in use, and forward each row reads its parameters, 64
// bytes for 16 of x.
#include "../kda_internal.h"
#include "kda.h"
#include "kda_layer.h"
#include "kda_rows.h"
#include "kda_ssm.h"

namespace kda {

namespace {

// How a launch lies over a row: lp lanes a group, gpb groups and rb rows of
// them a block. A group of 65 to 128 vectors takes a wave with two each, as fast as
// a block of its own (8192 x 4096 in 4 groups: 32 us and 31 forward, 70 and 86 back).
struct GroupShape {
  int nv, lp, gpb, rb, threads, gx;
  bool block;
  GroupShape(int dtype, int C, int groups) {
    const int W = C / groups, vecs = W / (dtype == KDA_F32 ? 4 : 8);
    block = vecs > 128;
    if (block) {
      nv = dtype == KDA_F32 ? 4 : 2;
      threads = ((vecs + nv - 1) / nv + 63) / 64 * 64;
      lp = threads;
      gpb = rb = 1;
    } else {
      nv = vecs > 64 ? 2 : 1;
      for (lp = 1; lp * nv < vecs;) lp *= 2;
      gpb = groups < 256 / lp ? groups : 256 / lp;
      rb = 256 / (lp * gpb);
      threads = (lp * gpb * rb + 63) / 64 * 64;
    }
    gx = (groups + gpb - 1) / gpb;
  }
};

// Sums of K values over a slot, every lane receiving them. A slot of the whole
// block alternates between two LDS buffers (`phase`), one barrier each.
template <bool BLOCK, int K>
__device__ __forceinline__ void slot_sum(float (&v)[K], int lp, float (&sm)[2][3][8], int& phase) {
  if constexpr (BLOCK) {
    const int nw = blockDim.x >> 6, w = threadIdx.x >> 6;
    float(&b)[3][8] = sm[phase & 1];
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
  } else {
    auto level = [&](auto move) {
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = move(v[k]);
    };
    if (lp > 1) level([](float x) { return x + dpp_mov<0xB1>(x); });
    if (lp > 2) level([](float x) { return x + dpp_mov<0x4E>(x); });
    if (lp > 4) level([](float x) { return x + dpp_mov<0x141>(x); });
    if (lp > 8) level([](float x) { return x + dpp_mov<0x140>(x); });
    if (lp > 16) level([](float x) {
      const uint32_t b = __float_as_uint(x);
      const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
      return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    });
    if (lp > 32) level([](float x) {
      const uint32_t b = __float_as_uint(x);
      const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
      return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    });
  }
}

template <typename TI, int NV, int GATE, bool BLOCK, bool BWD, bool NT>
__global__ void __launch_bounds__(512) k_group_norm(GroupNormArgs a, int lp, int gpb, int rb) {
  using RV = RowVec<TI>;
  constexpr int N = RV::N;
  __shared__ float sm[2][3][8];
  int phase = 0;
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & (lp - 1), slot = BLOCK ? 0 : threadIdx.x / lp;
  const int rsub = slot / gpb, group = blockIdx.x * gpb + slot % gpb;
  if (rsub >= rb || group >= a.groups) return;
  const int nvec = a.W / N, c0 = group * a.W;
  const float inv = 1.f / a.W;
  bool have[NV];
  int c[NV];
  float w[NV][N], b[NV][N], dw[NV][N], db[NV][N];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = j * lp + lane;
    have[j] = v < nvec;
    c[j] = c0 + v * N;
#pragma unroll
    for (int i = 0; i < N; ++i) w[j][i] = b[j][i] = dw[j][i] = db[j][i] = 0.f;
    if (have[j]) {
      load_params<N>(a.weight + c[j], w[j]);
      if (a.bias) load_params<N>(a.bias + c[j], b[j]);
    }
  }
  const int64_t step = static_cast<int64_t>(gridDim.y) * rb;
  for (int64_t row = static_cast<int64_t>(blockIdx.y) * rb + rsub; row < a.rows; row += step) {
    RV vx[NV], vg[NV], vd[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      vx[j].u = vg[j].u = vd[j].u = make_uint4(0, 0, 0, 0);
      if (have[j]) {
        vx[j].template load<NT>(static_cast<const TI*>(a.x) + row * a.xs + c[j]);
        if constexpr (GATE != KDA_GROUP_GATE_NONE) vg[j].template load<NT>(static_cast<const TI*>(a.gate) + row * a.gs + c[j]);
        if constexpr (BWD) vd[j].template load<NT>(static_cast<const TI*>(a.dy) + row * a.C + c[j]);
      }
    }
    // z, then z - m in its place
    float z[NV][N];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      vx[j].get(z[j]);
      if constexpr (GATE == KDA_GROUP_GATE_FIRST) {
        float g[N];
        vg[j].get(g);
#pragma unroll
        for (int i = 0; i < N; ++i) z[j][i] *= act_value(a.act, g[i], sigmoidf(g[i]));
      }
    }
    if (a.center) {
      float s[1] = {0.f};
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) s[0] += z[j][i];
      slot_sum<BLOCK, 1>(s, lp, sm, phase);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < N; ++i) z[j][i] = have[j] ? z[j][i] - s[0] * inv : 0.f;
    }
    // sums of z^2 and, where the slope at p needs no norm, of dn and dn z
    float s[3] = {0.f, 0.f, 0.f};
    constexpr bool kJoint = BWD && GATE != KDA_GROUP_GATE_NONE;
    float dn[NV][N];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float g[N], d[N];
      vg[j].get(g);
      vd[j].get(d);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        s[0] += z[j][i] * z[j][i];
        if constexpr (kJoint) {
          const float dp = GATE == KDA_GROUP_GATE_AFTER ? d[i] * act_value(a.act, g[i], sigmoidf(g[i])) : d[i];
          dn[j][i] = dp * w[j][i];
          s[1] += dn[j][i];
          s[2] += dn[j][i] * z[j][i];
        }
      }
    }
    if constexpr (kJoint) {
      slot_sum<BLOCK, 3>(s, lp, sm, phase);
    } else {
      float q[1] = {s[0]};
      slot_sum<BLOCK, 1>(q, lp, sm, phase);
      s[0] = q[0];
    }
    const float r = 1.f / sqrtf(s[0] * inv + a.eps);
    if constexpr (!BWD) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float g[N], y[N];
        vg[j].get(g);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float p = z[j][i] * r * w[j][i] + b[j][i];
          if constexpr (GATE == KDA_GROUP_GATE_NONE) y[i] = a.act == KDA_ACT_NONE ? p : act_value(a.act, p, sigmoidf(p));
          else if constexpr (GATE == KDA_GROUP_GATE_AFTER) y[i] = p * act_value(a.act, g[i], sigmoidf(g[i]));
          else y[i] = p;
        }
        vx[j].set(y);
        if (have[j]) vx[j].template store<NT>(static_cast<TI*>(a.y) + row * a.C + c[j]);
      }
    } else {
      if constexpr (!kJoint) {
        float q[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float d[N];
          vd[j].get(d);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float p = z[j][i] * r * w[j][i] + b[j][i];
            if (a.act != KDA_ACT_NONE) d[i] *= act_slope(a.act, p, sigmoidf(p));
            dw[j][i] += d[i] * z[j][i] * r;
            db[j][i] += d[i];
            dn[j][i] = d[i] * w[j][i];
            q[0] += dn[j][i];
            q[1] += dn[j][i] * z[j][i];
          }
        }
        slot_sum<BLOCK, 2>(q, lp, sm, phase);
        s[1] = q[0];
        s[2] = q[1];
      }
      const float md = a.center ? s[1] * inv : 0.f, mz = s[2] * inv * r * r;  // mean(dn), r mean(dn n)
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float g[N], d[N], x[N];
        vg[j].get(g);
        vd[j].get(d);
        vx[j].get(x);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float n = z[j][i] * r;
          float dz = r * (dn[j][i] - md) - mz * n;
          if constexpr (GATE != KDA_GROUP_GATE_NONE) {
            const float sg = sigmoidf(g[i]), av = act_value(a.act, g[i], sg), slope = act_slope(a.act, g[i], sg);
            if constexpr (GATE == KDA_GROUP_GATE_FIRST) {
              dw[j][i] += d[i] * n;
              db[j][i] += d[i];
              g[i] = dz * x[i] * slope;
              dz *= av;
            } else {
              dw[j][i] += d[i] * av * n;
              db[j][i] += d[i] * av;
              g[i] = d[i] * (n * w[j][i] + b[j][i]) * slope;
            }
          }
          x[i] = dz;
        }
        if (have[j]) {
          vx[j].set(x);
          vx[j].template store<NT>(static_cast<TI*>(a.dx) + row * a.C + c[j]);
          if constexpr (GATE != KDA_GROUP_GATE_NONE) {
            vg[j].set(g);
            vg[j].template store<NT>(static_cast<TI*>(a.dgate) + row * a.C + c[j]);
          }
        }
      }
    }
  }
  if constexpr (BWD) {
    float* p = a.partials + (static_cast<size_t>(blockIdx.y) * rb + rsub) * (a.dbias ? 2 : 1) * a.C;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (have[j]) {
        store_params<N>(p + c[j], dw[j]);
        if (a.dbias) store_params<N>(p + a.C + c[j], db[j]);
      }
    }
  }
}

// Blocks along the rows: forward all of them up to 65535 and 2^22 blocks in
// all, backward, where each leaves a partial row, enough to fill the chip: 512, 1024
// or 2048 take 70, 65 and 67 us at 8192 rows of 4096 channels in 8 groups, 113, 71
// and 83 in 2, 102, 108 and 120 at 4096 rows of one group of 8192.
unsigned group_norm_rows(const GroupShape& g, int64_t rows, bool bwd) {
  const int64_t want = (rows + g.rb - 1) / g.rb, fill = (1 << 22) / g.gx;
  const int64_t most = bwd ? (1024 + g.gx - 1) / g.gx : (fill < 65535 ? fill : 65535);
  return static_cast<unsigned>(want < most ? want : most);
}

template <typename TI, int NV, int GATE, bool BLOCK, bool NT>
hipError_t launch_group_n(bool bwd, const GroupShape& g, const GroupNormArgs& a, hipStream_t s) {
  const dim3 grid(g.gx, group_norm_rows(g, a.rows, bwd));
  if (bwd) k_group_norm<TI, NV, GATE, BLOCK, true, NT><<<grid, g.threads, 0, s>>>(a, g.lp, g.gpb, g.rb);
  else k_group_norm<TI, NV, GATE, BLOCK, false, NT><<<grid, g.threads, 0, s>>>(a, g.lp, g.gpb, g.rb);
  return hipGetLastError();
}
template <typename TI, int NV, int GATE, bool BLOCK>
hipError_t launch_group_v(bool bwd, const GroupShape& g, const GroupNormArgs& a, hipStream_t s) {
  const int rows = (bwd ? 3 : 2) + (GATE == KDA_GROUP_GATE_NONE ? 0 : bwd ? 2 : 1);
  return streams_past_caches(rows * a.rows * a.C * static_cast<int64_t>(sizeof(TI)))
             ? launch_group_n<TI, NV, GATE, BLOCK, true>(bwd, g, a, s)
             : launch_group_n<TI, NV, GATE, BLOCK, false>(bwd, g, a, s);
}
template <typename TI, int GATE>
hipError_t launch_group_g(bool bwd, const GroupNormArgs& a, hipStream_t s) {
  const GroupShape g(sizeof(TI) == 4 ? KDA_F32 : KDA_BF16, a.C, a.groups);
  if (g.block) return launch_group_v<TI, sizeof(TI) == 4 ? 4 : 2, GATE, true>(bwd, g, a, s);
  return g.nv == 1 ? launch_group_v<TI, 1, GATE, false>(bwd, g, a, s) : launch_group_v<TI, 2, GATE, false>(bwd, g, a, s);
}
template <typename TI>
hipError_t launch_group_t(bool bwd, int gate, const GroupNormArgs& a, hipStream_t s) {
  if (gate == KDA_GROUP_GATE_NONE) return launch_group_g<TI, KDA_GROUP_GATE_NONE>(bwd, a, s);
  if (gate == KDA_GROUP_GATE_AFTER) return launch_group_g<TI, KDA_GROUP_GATE_AFTER>(bwd, a, s);
  return launch_group_g<TI, KDA_GROUP_GATE_FIRST>(bwd, a, s);
}
hipError_t launch_group(bool bwd, int dtype, int gate, const GroupNormArgs& a, hipStream_t s) {
  return dtype == KDA_F32 ? launch_group_t<float>(bwd, gate, a, s) : launch_group_t<bf16>(bwd, gate, a, s);
}

}  // namespace

int64_t group_norm_partials(int dtype, int C, int groups, int64_t rows) {
  if (rows == 0) return 0;
  const GroupShape g(dtype, C, groups);
  return static_cast<int64_t>(group_norm_rows(g, rows, true)) * g.rb;
}
hipError_t launch_group_norm_fwd(int dtype, int gate, const GroupNormArgs& a, hipStream_t s) {
  return launch_group(false, dtype, gate, a, s);
}
hipError_t launch_group_norm_bwd(int dtype, int gate, const GroupNormArgs& a, hipStream_t s) {
  return launch_group(true, dtype, gate, a, s);
}

}  // namespace kda
