// The recurrent form of the gated delta rule (KDA, its per-head gate, GDN-2):
// one token after another from a state in HBM, for decoding.
//
// Per (sequence, head), with the state S [K][V] in fp32:
//   S~ = Diag(a) S,  u = S~^T e,  d = w - u
//   S  = S~ + kh d^T,  o = S^T qh = S~^T qh + (kh . qh) d
// where a = exp(g); e = beta kh and w = beta v (KDA), or e = b * kh and
// w = (write gate) * v (GDN-2). Taking o from S~ puts both sums over the rows
// of S in one pass, so a token costs one reduction across lanes.
//
// What bounds it: the state's bytes, 4 K V read and written once per
// sequence and head whatever the number of tokens; the rows of a token are
// 1-2% of that at one token per sequence. Every column of S is independent,
// so a wave takes all K rows of CW columns (a lane: 4 columns and every
// (CW / 4)-lane-th group of 4 rows), the tile in registers over all tokens,
// and no wave waits for another. Each wave computes the token's prologue for
// itself (norms, gates; K channels over 64 lanes, passed to its lanes' row
// layout through its own 4 K floats of LDS): its rows come from the caches
// after the first wave's, and a shared copy would need a barrier per token.
// The next token's rows are loaded during a token's step (9 x 12 heads of 5
// tokens: 9.0 -> 8.2 us); computing its prologue there too gained nothing and
// its registers cost a wave per SIMD.
//
// States are loaded and stored past the caches (non-temporal): a model's
// layers together hold more states than the caches, and then 64 sequences x
// 32 heads x D128 take 51 us instead of 57, 16 x 32 heads 14.2 instead of
// 16.7. A single pool that would have stayed in the cache from call to call
// takes 48.7 instead of 41.9.
//
// Sums, gates and the state are fp32 for either dtype; only o is rounded,
// once. The chunked form keeps an fp32 problem's gate in fp64 because it adds
// it up over a chunk; here a gate is used alone, from the fp32 exponential and
// reciprocal (fp32 states after up to 8 tokens: 2.2e-8 of fp64, normalised L2).
#include "../kda_device.h"
#include "../kda_prologue.h"
#include "kda_layer.h"
#include "kda_rows.h"

namespace kda {

namespace {

// CPL consecutive channels of a row from c0 (CPL = D / 64).
template <typename TI, int CPL>
struct RowPart {
  uint32_t u[CPL];
  __device__ __forceinline__ void load(const TI* p) {
    if constexpr (CPL == 1) {
      u[0] = load_bits<TI>(p);
    } else if constexpr (sizeof(TI) == 2) {
      u[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      u[0] = x.x;
      u[1] = x.y;
    }
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (CPL == 2 && sizeof(TI) == 2)
      return __uint_as_float(e ? (u[0] & 0xffff0000u) : (u[0] << 16));
    else
      return bits_to_f<TI>(u[e]);
  }
};

// Sum over the row groups of a wave: the lanes that differ in lane / (CW / 4),
// by rotations within rows of 16 lanes and swaps of rows and halves.
template <int CW>
__device__ __forceinline__ float sum_rows(float x) {
  if constexpr (CW == 16) x += dpp_mov<0x124>(x);
  return sum_row_groups(x);
}

template <typename TI, int D, bool G2, int CW, int NW, bool MANY>
__global__ void __launch_bounds__(64 * NW) k_recurrent(RecurrentArgs a) {
  constexpr int NT = D / CW;            // waves per (sequence, head), CW columns each
  constexpr int CPL = D / 64;           // prologue channels per lane
  constexpr int RS = 4 * 64 / (CW / 4); // rows of one load by the wave's lanes, 4 each
  constexpr int NJ = D / RS;            // groups of 4 rows per lane
  __shared__ __align__(16) float sm[NW][4][D];  // per wave: a, e, kh, qh
  const int nh = blockIdx.x / (NT / NW);
  const int n = nh / a.H, h = nh % a.H;
  if (n >= a.N) {
    const unsigned own = static_cast<unsigned>(a.N) * a.H * (NT / NW);
    zero_rest(a.o, static_cast<size_t>(a.H) * D * sizeof(TI), a.cu, a.N, a.T, blockIdx.x - own, gridDim.x - own);
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
  TI* o = static_cast<TI*>(a.o) + static_cast<size_t>(h) * D;
  const size_t os = static_cast<size_t>(a.H) * D;
  const int cg = lane % (CW / 4), rg = lane / (CW / 4);
  const int col = CW * (static_cast<int>(blockIdx.x % (NT / NW)) * NW + w) + 4 * cg;
  if (slot < 0) {  // padded: zeros; a slot it cannot have: NaN
    const float f = slot == kPadded ? 0.f : nan_value();
    if (rg == 0)
      for (int64_t t = t0; t < t1; ++t) store4<TI>(o + t * os + col, f32x4{f, f, f, f});
    return;
  }

  const int c0 = CPL * lane;
  const size_t hc = static_cast<size_t>(h) * D + c0;
  const float ea = expf(a.A_log[h]);
  float db[CPL];
#pragma unroll
  for (int e = 0; e < CPL; ++e) db[e] = a.gate_head ? a.dt_bias[h] : a.dt_bias[hc + e];

  // a token's rows, loaded one token ahead of their use
  struct Token {
    RowPart<TI, CPL> q, k, g, b;
    uint32_t be, v[4], w[4];
  };
  auto load = [&](int64_t t, Token& x) {
    x.q.load(static_cast<const TI*>(a.q) + t * a.qs + hc);
    x.k.load(static_cast<const TI*>(a.k) + t * a.ks + hc);
    if (a.gate_head) {
      const uint32_t u = load_bits<TI>(static_cast<const TI*>(a.g) + t * a.gs + h);
      if constexpr (CPL == 2 && sizeof(TI) == 2) x.g.u[0] = u | (u << 16);
      else x.g.u[0] = x.g.u[CPL - 1] = u;
    } else {
      x.g.load(static_cast<const TI*>(a.g) + t * a.gs + hc);
    }
    const size_t vc = static_cast<size_t>(h) * D + col;
    if constexpr (G2) {
      x.b.load(static_cast<const TI*>(a.bk) + t * a.bks + hc);
      load4_raw<TI>(static_cast<const TI*>(a.wv) + t * a.wvs + vc, x.w);
    } else {
      x.be = load_bits<TI>(static_cast<const TI*>(a.beta) + t * a.bes + h);
    }
    load4_raw<TI>(static_cast<const TI*>(a.v) + t * a.vs + vc, x.v);
  };
  Token next;
  load(t0, next);

  // rows RS j + 4 rg + r of the lane's four columns
  float* Sp = a.state + (static_cast<size_t>(slot) * a.H + h) * (D * D) + 4 * rg * D + col;
  f32x4 s[NJ][4];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) s[j][r] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(Sp + (RS * j + r) * D));

  for (int64_t t = t0; t < t1; ++t) {
    const Token x = next;
    if (t + 1 < t1) load(t + 1, next);
    const RowPart<TI, CPL>&q = x.q, &k = x.k, &g = x.g, &b = x.b;
    // prologue: this lane's channels, then to the row layout through LDS
    float sq = 0.f, sk = 0.f, qk = 0.f;
#pragma unroll
    for (int e = 0; e < CPL; ++e) {
      sq += q.get(e) * q.get(e);
      sk += k.get(e) * k.get(e);
      qk += q.get(e) * k.get(e);
    }
    sq = sum_wave(sq);
    sk = sum_wave(sk);
    qk = sum_wave(qk);
    const float rq = a.scale * rsqrtf(sq + a.eps), rk = rsqrtf(sk + a.eps);
    const float beta = G2 ? 0.f : sigmoidf(bits_to_f<TI>(x.be));
    const float kq = qk * rq * rk;
#pragma unroll
    for (int e = 0; e < CPL; ++e) {
      const float kh = k.get(e) * rk;
      sm[w][0][c0 + e] = expf(gate_map<float>(a.gate_mode, ea, g.get(e) + db[e], a.lb));
      sm[w][1][c0 + e] = (G2 ? sigmoidf(b.get(e)) : beta) * kh;
      sm[w][2][c0 + e] = kh;
      sm[w][3][c0 + e] = q.get(e) * rq;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();

    f32x4 u = zero4(), oo = zero4();
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int r0 = RS * j + 4 * rg;
      const f32x4 av = *reinterpret_cast<const f32x4*>(&sm[w][0][r0]);
      const f32x4 ev = *reinterpret_cast<const f32x4*>(&sm[w][1][r0]);
      const f32x4 qv = *reinterpret_cast<const f32x4*>(&sm[w][3][r0]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s[j][r] *= av[r];
        u += ev[r] * s[j][r];
        oo += qv[r] * s[j][r];
      }
    }
    f32x4 d = unpack4<TI>(x.v);
    if constexpr (G2) {
      const f32x4 wg = unpack4<TI>(x.w);
#pragma unroll
      for (int r = 0; r < 4; ++r) d[r] *= sigmoidf(wg[r]);
    } else {
      d *= beta;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      d[r] -= sum_rows<CW>(u[r]);
      oo[r] = sum_rows<CW>(oo[r]) + kq * d[r];
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const f32x4 kv = *reinterpret_cast<const f32x4*>(&sm[w][2][RS * j + 4 * rg]);
#pragma unroll
      for (int r = 0; r < 4; ++r) s[j][r] += kv[r] * d;
    }
    if (rg == 0) store4<TI>(o + t * os + col, oo);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }

#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) vstore<true>(reinterpret_cast<f32x4*>(Sp + (RS * j + r) * D), s[j][r]);
}

// Three shapes of one kernel (microseconds per launch, bf16, D = 128, states
// that come from HBM):
//   wide: the waves of a (sequence, head) in one block, 32 columns each.
//   narrow: single waves of 16 columns. A token's step is bound by one wave's
//     instructions (about 1.1 us), and half the columns are half of them:
//     1 sequence x 32 heads, 8 tokens 13.7 -> 11.1, 4 x 32 heads 13.8 -> 11.9.
//     Taken while one such wave per SIMD holds the launch and cu_seqlens says
//     that sequences may have several tokens; with one token its half lines
//     cost more (4 x 32 heads 5.9 -> 7.8). D = 64 has half the rows: no gain
//     (8 x 16 heads, 8 tokens fp32 10.1 either way).
//   wide with one block (D = 128) or four (D = 64) per CU, kept apart by LDS
//     that nothing uses: one token a sequence is a copy of the states, which
//     runs faster with fewer reads and writes interleaved: 128 sequences x 32
//     heads 100.2 -> 94.1, 251 x 32 heads 195.9 -> 182.5 (5.8 TB/s), 256 x 64
//     heads 383 -> 353; D = 64, 512 x 64 heads 201.7 -> 194.4. From 4096
//     (sequence, head) pairs, where every type gains (pairs: apart not / apart):
//       D = 128 bf16  512 16.0 / 16.8  1024 29.1 / 28.9  2048 52.7 / 50.8  4096 101.8 / 95.4  8192 201.7 / 187.0
//       D = 128 fp32  512 14.4 / 17.2  1024 29.0 / 30.9  2048 53.2 / 54.6  4096 103.1 / 101.7  8192 201.1 / 195.2
//       D = 64 bf16   512 7.8 / 7.7  1024 9.1 / 9.1  2048 17.3 / 17.1  4096 29.0 / 28.6  8192 56.1 / 53.7
//     Several tokens need the waves (37 x 64 heads of up to 8: 59.6 -> 84.5).
template <typename TI, int D, bool G2>
hipError_t launch_g(const RecurrentArgs& a, hipStream_t s) {
  const unsigned nh = static_cast<unsigned>(a.N) * static_cast<unsigned>(a.H);
  // blocks of 256 threads, below 2^32 in all
  const unsigned rest = rest_blocks(a.zero_rest, a.T * a.H * D * static_cast<int64_t>(sizeof(TI)), (1 << 24) - 1 - nh);
  if constexpr (D == 128) {
    if (a.cu && nh * (D / 16) <= 1024) {
      k_recurrent<TI, D, G2, 16, 1, false><<<nh * (D / 16) + rest, 64, 0, s>>>(a);
      return hipGetLastError();
    }
  }
  const unsigned apart = !a.cu && nh >= 4096 ? (D == 128 ? 100 : 35) * 1024 : 0;
  if (a.idx && a.N > kScanAlone) k_recurrent<TI, D, G2, 32, D / 32, true><<<nh + rest, 2 * D, apart, s>>>(a);
  else k_recurrent<TI, D, G2, 32, D / 32, false><<<nh + rest, 2 * D, apart, s>>>(a);
  return hipGetLastError();
}
template <typename TI, int D>
hipError_t launch_d(bool gdn2, const RecurrentArgs& a, hipStream_t s) {
  return gdn2 ? launch_g<TI, D, true>(a, s) : launch_g<TI, D, false>(a, s);
}

}  // namespace

hipError_t launch_recurrent(int dtype, int D, bool gdn2, const RecurrentArgs& a, hipStream_t s) {
  if (dtype == 0) return D == 64 ? launch_d<float, 64>(gdn2, a, s) : launch_d<float, 128>(gdn2, a, s);
  return D == 64 ? launch_d<bf16, 64>(gdn2, a, s) : launch_d<bf16, 128>(gdn2, a, s);
}

}  // namespace kda
