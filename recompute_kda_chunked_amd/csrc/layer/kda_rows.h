// Device helpers of the row kernels around the chunked operator: 16-byte
// vectors of a row, and sums over a wave.
#pragma once

#include "../kda_device.h"

namespace kda {

// Sum over the lanes 8, 16 and 32 apart: a rotation by 8 within rows of 16
// lanes, then gfx950's row and half swaps of a value with itself (no LDS
// traffic). Every lane receives the sum.
__device__ __forceinline__ float sum_row_groups(float x) {
  x += dpp_mov<0x128>(x);
  const uint32_t b = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  const uint32_t c = __float_as_uint(x);
  const auto h = __builtin_amdgcn_permlane32_swap(c, c, false, false);
  return __uint_as_float(h[0]) + __uint_as_float(h[1]);
}
// Sum over all 64 lanes.
__device__ __forceinline__ float sum_wave(float x) { return sum_row_groups(group_sum<8>(x)); }

// A load with or without the non-temporal hint (see streams_past_caches).
template <bool NT, typename V>
__device__ __forceinline__ V vload(const V* p) {
  if constexpr (NT) return __builtin_nontemporal_load(p);
  else return *p;
}

// 16 bytes of a row: 8 bf16 or 4 fp32 values.
template <typename TI>
struct RowVec {
  static constexpr int N = 16 / sizeof(TI);
  uint4 u;
  template <bool NT>
  __device__ __forceinline__ void load(const TI* p) {
    u = __builtin_bit_cast(uint4, vload<NT>(reinterpret_cast<const f32x4*>(p)));
  }
  template <bool NT>
  __device__ __forceinline__ void store(TI* p) const {
    vstore<NT>(reinterpret_cast<f32x4*>(p), __builtin_bit_cast(f32x4, u));
  }
  __device__ __forceinline__ void get(float (&f)[N]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(TI) == 2) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        f[i] = __uint_as_float(w[i]);
      }
    }
  }
  // rounds to nearest even
  __device__ __forceinline__ void set(const float (&f)[N]) {
    if constexpr (sizeof(TI) == 2) {
      bf16x8 b;
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = static_cast<bf16>(f[i]);
      u = __builtin_bit_cast(uint4, b);
    } else {
      u = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                     __float_as_uint(f[3]));
    }
  }
};

// N consecutive fp32 parameters from a 16-byte aligned address.
template <int N>
__device__ __forceinline__ void load_params(const float* p, float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(p + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[i + j] = v[j];
  }
}
template <int N>
__device__ __forceinline__ void store_params(float* p, const float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4)
    *reinterpret_cast<f32x4*>(p + i) = f32x4{f[i], f[i + 1], f[i + 2], f[i + 3]};
}

// Whether sequence j has a token in [0, T), where its bounds are clamped to.
__device__ __forceinline__ bool has_tokens(const int32_t* cu, int64_t T, int j) {
  const int64_t s = cu[j] < 0 ? 0 : cu[j], e = cu[j + 1] > T ? T : cu[j + 1];
  return s < e;
}

// The pool slot of sequence n, found by the whole block: kPadded for a negative
// index (a padded sequence), kBadSlot for one past the pool or one that an
// earlier sequence with tokens names too (two writers of one state). Every
// block looks through all earlier indices, the first of them read together with
// its own, so a launch's reads grow with the square of their number, and the
// host refuses more than 65536. MANY, for more than kScanAlone sequences: the
// block's waves share the search (it costs 37 x 64 heads of drafts 0.4 of 59 us,
// so fewer sequences go without). Microseconds without indices / with them:
//   recurrent, 1 head, D = 64   256 6.6 / 6.7   1024 9.8 / 12.8   4096 27 / 35   16384 89 / 165   65536 344 / 1283
//   update, 2048 channels       256 6.6 / 6.5   1024 9.9 / 13.0   4096 24 / 32   16384 109 / 191  65536 437 / 1149
// (each wave on its own, as for fewer: 4096 49 and 54, 16384 375 and 512).
constexpr int64_t kPadded = -1, kBadSlot = -2;
constexpr int kScanAlone = 1024;
template <bool MANY>
__device__ __forceinline__ int64_t find_slot(const int32_t* idx, const int32_t* cu, int64_t T,
                                             int n, int64_t n_slots) {
  if (!idx) return n;
  const int step = MANY ? blockDim.x : 64;
  int j = MANY ? threadIdx.x : threadIdx.x & 63;
  const int32_t own = idx[n], first = idx[j < n ? j : n];
  const int32_t slot = __builtin_amdgcn_readfirstlane(own);
  bool taken = false;
  auto look = [&](int i, int32_t x) {
    if (x == slot && (!cu || has_tokens(cu, T, i))) taken = true;
  };
  if (j < n) look(j, first);
  j += step;
  if constexpr (MANY) {
    for (; j + 3 * step < n; j += 4 * step) {
      int32_t x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) x[u] = idx[j + u * step];
#pragma unroll
      for (int u = 0; u < 4; ++u) look(j + u * step, x[u]);
    }
  }
  for (; j < n; j += step) look(j, idx[j]);
  const bool twice = MANY ? __syncthreads_or(taken) != 0 : __any(taken) != 0;
  if (slot < 0) return kPadded;
  return slot >= n_slots || twice ? kBadSlot : slot;
}

// Zeroes the rows of o [T][row_bytes] that belong to no sequence, those before
// the first one and those from the end of the last one on: the work of block
// `b` of the `nb` that a launch has for it behind the sequences' own. (In those
// it cost the drafts above 0.7 us, their two loads more than the rows.)
__device__ __forceinline__ void zero_rest(void* o, size_t row_bytes, const int32_t* cu, int N,
                                          int64_t T, unsigned b, unsigned nb) {
  int64_t before = cu[0], behind = cu[N];
  before = before < 0 ? 0 : (before > T ? T : before);
  behind = behind < before ? before : (behind > T ? T : behind);
  const int64_t row = static_cast<int64_t>(row_bytes / 16);
  f32x4* p = static_cast<f32x4*>(o);
  const int64_t step = static_cast<int64_t>(nb) * blockDim.x, at = static_cast<int64_t>(b) * blockDim.x + threadIdx.x;
  for (int64_t i = at; i < before * row; i += step) p[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int64_t i = behind * row + at; i < T * row; i += step) p[i] = f32x4{0.f, 0.f, 0.f, 0.f};
}
// Blocks for it: one per 64 KB of o, at most 1024 and at most `room`.
inline unsigned rest_blocks(bool zero, int64_t bytes, int64_t room) {
  if (!zero) return 0;
  const int64_t want = (bytes + 65535) / 65536, most = room < 1024 ? room : 1024;
  return static_cast<unsigned>(want < most ? want : most);
}
__device__ __forceinline__ float nan_value() { return __uint_as_float(0x7fc00000u); }

}  // namespace kda
