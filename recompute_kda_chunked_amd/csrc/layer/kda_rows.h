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
// block looks through all earlier indices, so a launch's reads grow with the
// square of their number, and the host refuses more than 65536: each wave on
// its own up to kScanAlone (four loads at once), the block's waves together
// above. Microseconds without indices / with them:
//   recurrent, 1 head, D = 64   256 6.5 / 6.9   1024 10.0 / 12.0   4096 27 / 33   16384 90 / 159   65536 345 / 1252
//   update, 2048 channels       256 6.6 / 6.7   1024 10.2 / 12.2   4096 24 / 30   16384 110 / 183  65536 433 / 1119
// (each wave on its own one load at a time: 4096 49 and 54, 16384 375 and 512).
constexpr int64_t kPadded = -1, kBadSlot = -2;
constexpr int kScanAlone = 1024;
__device__ __forceinline__ int64_t find_slot(const int32_t* idx, const int32_t* cu, int64_t T,
                                             int n, int64_t n_slots) {
  if (!idx) return n;
  const int32_t slot = __builtin_amdgcn_readfirstlane(idx[n]);
  const bool together = n > kScanAlone;
  const int step = together ? blockDim.x : 64;
  int j = together ? threadIdx.x : threadIdx.x & 63;
  bool taken = false;
  auto look = [&](int i, int32_t x) {
    if (x == slot && (!cu || has_tokens(cu, T, i))) taken = true;
  };
  for (; j + 3 * step < n; j += 4 * step) {
    int32_t x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = idx[j + u * step];
#pragma unroll
    for (int u = 0; u < 4; ++u) look(j + u * step, x[u]);
  }
  for (; j < n; j += step) look(j, idx[j]);
  const bool twice = together ? __syncthreads_or(taken) != 0 : __any(taken) != 0;
  if (slot < 0) return kPadded;
  return slot >= n_slots || twice ? kBadSlot : slot;
}
// The rows in [0, T) that belong to no sequence: those before the first one and
// those from the end of the last one on.
struct Rest {
  int64_t before, behind, T;
  __device__ __forceinline__ Rest(const int32_t* cu, int N, int64_t t) : before(cu[0]), behind(cu[N]), T(t) {
    before = before < 0 ? 0 : (before > T ? T : before);
    behind = behind < before ? before : (behind > T ? T : behind);
  }
  __device__ __forceinline__ int64_t rows() const { return before + T - behind; }
  __device__ __forceinline__ int64_t row(int64_t i) const { return i < before ? i : behind + (i - before); }
};
__device__ __forceinline__ float nan_value() { return __uint_as_float(0x7fc00000u); }

}  // namespace kda
