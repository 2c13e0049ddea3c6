// Tiles and matrix products of the selective scan's kernels.
//
// A tile lies in LDS row by row in 16-byte units, unit u of row r at place
// u ^ (r & 7), so that the reads below (16 rows at one column, or 4 rows of 32
// bytes) spread over the banks. A fragment is one operand of a product over 32
// values of the reduction index: 8 per lane, lane (i, g) = i + 16 g holding row
// (or column) i and the 8 values that group g has; the products take any
// assignment of the 32 values to (g, e) as long as both operands have the same:
//   plain   k = 8 g + e
//   paired  k = 4 g + e (e < 4), 16 + 4 g + e - 4: the one in which two
//           accumulator tiles (lane: rows 4 g .. 4 g + 3 of column i) are an
//           operand as they stand, so that scores never leave the registers.
// For fp32 a product is eight 16x16x4 instructions, each over one e.
#pragma once

#include "../kda_device.h"

namespace kda {

typedef __attribute__((ext_vector_type(8))) float f32x8;
typedef __attribute__((ext_vector_type(4))) short s16x4;

template <typename T>
struct FragOf;
template <>
struct FragOf<bf16> { typedef bf16x8 type; };
template <>
struct FragOf<float> { typedef f32x8 type; };
template <typename T>
using Frag = typename FragOf<T>::type;

__device__ __forceinline__ f32x4 mma32(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma32(f32x8 a, f32x8 b, f32x4 c) {
#pragma unroll
  for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
  return c;
}

// Place of element (row, col) in a tile of COLS columns.
template <typename T, int COLS>
__device__ __forceinline__ int tile_at(int row, int col) {
  constexpr int U = 16 / sizeof(T), M = (COLS / U < 8 ? COLS / U : 8) - 1;
  return row * COLS + (((col / U) ^ (row & M)) * U) + col % U;
}

// A 4 x 16 block per group of 16 lanes, read transposed: lane i of
// the group receives column i of its four rows (gfx950's transposing LDS read).
__device__ __forceinline__ s16x4 tr_read(const bf16* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
}

// Rows r0 .. r0 + 15, reduction over columns k0 .. k0 + 31 (plain).
template <int COLS>
__device__ __forceinline__ bf16x8 frag_row(const bf16* t, int r0, int k0, int lane) {
  return *reinterpret_cast<const bf16x8*>(t + tile_at<bf16, COLS>(r0 + (lane & 15), k0 + 8 * (lane >> 4)));
}
template <int COLS>
__device__ __forceinline__ f32x8 frag_row(const float* t, int r0, int k0, int lane) {
  const int r = r0 + (lane & 15), k = k0 + 8 * (lane >> 4);
  const f32x4 a = *reinterpret_cast<const f32x4*>(t + tile_at<float, COLS>(r, k));
  const f32x4 b = *reinterpret_cast<const f32x4*>(t + tile_at<float, COLS>(r, k + 4));
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
// Columns c0 .. c0 + 15, reduction over rows k0 .. k0 + 31, plain or paired.
template <int COLS, bool PAIRED>
__device__ __forceinline__ bf16x8 frag_col(const bf16* t, int k0, int c0, int lane) {
  const int i = lane & 15, g = lane >> 4, r = k0 + (PAIRED ? 4 : 8) * g + (i >> 2), c = c0 + 4 * (i & 3);
  const s16x4 a = tr_read(t + tile_at<bf16, COLS>(r, c)), b = tr_read(t + tile_at<bf16, COLS>(r + (PAIRED ? 16 : 4), c));
  typedef __attribute__((ext_vector_type(8))) short s16x8;
  return __builtin_bit_cast(bf16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
}
template <int COLS, bool PAIRED>
__device__ __forceinline__ f32x8 frag_col(const float* t, int k0, int c0, int lane) {
  const int i = lane & 15, g = lane >> 4;
  f32x8 f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int k = PAIRED ? (e < 4 ? 4 * g + e : 12 + 4 * g + e) : 8 * g + e;
    f[e] = t[tile_at<float, COLS>(k0 + k, c0 + i)];
  }
  return f;
}
// The same from a row-major matrix in memory, rows `ld` apart (plain).
__device__ __forceinline__ bf16x8 frag_mem(const bf16* m, int r0, int k0, int ld, int lane) {
  return *reinterpret_cast<const bf16x8*>(m + (r0 + (lane & 15)) * ld + k0 + 8 * (lane >> 4));
}
__device__ __forceinline__ f32x8 frag_mem(const float* m, int r0, int k0, int ld, int lane) {
  return *reinterpret_cast<const f32x8*>(m + (r0 + (lane & 15)) * ld + k0 + 8 * (lane >> 4));
}

// Two accumulator tiles as one operand (paired).
template <typename T>
__device__ __forceinline__ Frag<T> pair_frag(const f32x4& a, const f32x4& b) {
  Frag<T> f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[e] = static_cast<T>(a[e]);
    f[4 + e] = static_cast<T>(b[e]);
  }
  return f;
}

// Four consecutive elements of a tile as floats.
template <typename T, int COLS>
__device__ __forceinline__ f32x4 tile_get4(const T* t, int row, int col) {
  uint32_t u[4];
  load4_raw<T>(t + tile_at<T, COLS>(row, col), u);
  return unpack4<T>(u);
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

}  // namespace kda
