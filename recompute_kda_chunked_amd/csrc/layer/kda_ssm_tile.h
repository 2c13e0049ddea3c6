// Tiles and matrix products of the selective scan's kernels.
//
// A tile lies in LDS row by row, its 16-byte units in an order that goes by the
// row. A fragment is one operand of a product over 32
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

// Place of element (row, col) in a tile of COLS columns. The 16-byte units of a
// row change places by row so that both kinds of reads below are free of bank
// conflicts (64 banks of 4 bytes; a pass takes 16 bytes of the lanes i < 8 of
// one g with the lanes i >= 8 of the next, or 8 bytes of two whole g): sixteen
// rows at one unit with the next, and 4 + 4 rows, 8 rows on, at two units.
template <typename T, int COLS>
struct TileFlip {
  static constexpr int U = 16 / sizeof(T), UNITS = COLS / U < 16 ? COLS / U : 16;  // units that change places
  static constexpr int WIN = UNITS * U;
  static __device__ __forceinline__ constexpr int units(int row) {
    const int r = row & 7, far = (row >> 3) & 1;
    if (UNITS == 4) return far << 1;
    if (UNITS == 8) return r ^ (far << 2);
    return sizeof(T) == 2 ? (r << 1) ^ (far << 3) : r ^ (far << 3);
  }
};
template <typename T, int COLS>
__device__ __forceinline__ int tile_at(int row, int col) {
  using F = TileFlip<T, COLS>;
  return row * COLS + (col ^ (F::units(row) * F::U));
}

// A 4 x 16 block per group of 16 lanes, read transposed: lane i of
// the group receives column i of its four rows (gfx950's transposing LDS read).
__device__ __forceinline__ s16x4 tr_read(const bf16* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
}

// Element offsets within a tile are a lane's part with some of its low bits
// flipped by the tile's constant ones, plus constants. The lane's parts, for rows
// and columns that start at multiples of 16:
template <typename T, int COLS>
struct LaneAt {
  static constexpr int WIN = TileFlip<T, COLS>::WIN;
  int row, col, pair, four;
  __device__ __forceinline__ explicit LaneAt(int lane) {
    const int i = lane & 15, g = lane >> 4;
    row = tile_at<T, COLS>(i, 8 * g);
    col = sizeof(T) == 2 ? tile_at<T, COLS>(8 * g + (i >> 2), 4 * (i & 3)) : tile_at<T, COLS>(8 * g, i);
    pair = sizeof(T) == 2 ? tile_at<T, COLS>(4 * g + (i >> 2), 4 * (i & 3)) : tile_at<T, COLS>(4 * g, i);
    four = tile_at<T, COLS>(i, 4 * g);
  }
};
template <typename L>
__device__ __forceinline__ int shifted(int at, int col) {
  return (at ^ (col & (L::WIN - 1))) + (col & ~(L::WIN - 1));
}

// Rows r0 .. r0 + 15, reduction over columns k0 .. k0 + 31 (plain).
template <int COLS>
__device__ __forceinline__ bf16x8 frag_row(const bf16* t, const LaneAt<bf16, COLS>& l, int r0, int k0) {
  return *reinterpret_cast<const bf16x8*>(t + shifted<LaneAt<bf16, COLS>>(l.row, k0) + r0 * COLS);
}
template <int COLS>
__device__ __forceinline__ f32x8 frag_row(const float* t, const LaneAt<float, COLS>& l, int r0, int k0) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(t + shifted<LaneAt<float, COLS>>(l.row, k0) + r0 * COLS);
  const f32x4 b = *reinterpret_cast<const f32x4*>(t + shifted<LaneAt<float, COLS>>(l.row, k0 + 4) + r0 * COLS);
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
// Columns c0 .. c0 + 15, reduction over rows k0 .. k0 + 31, plain or paired.
template <bool PAIRED, int COLS>
__device__ __forceinline__ bf16x8 frag_col(const bf16* t, const LaneAt<bf16, COLS>& l, int k0, int c0) {
  constexpr int FLIP = PAIRED ? 0 : (TileFlip<bf16, COLS>::units(4) ^ TileFlip<bf16, COLS>::units(0)) * 8;  // four rows on
  const int at = shifted<LaneAt<bf16, COLS>>(PAIRED ? l.pair : l.col, c0) + k0 * COLS;
  const int on = shifted<LaneAt<bf16, COLS>>((PAIRED ? l.pair : l.col) ^ FLIP, c0) + (k0 + (PAIRED ? 16 : 4)) * COLS;
  const s16x4 a = tr_read(t + at), b = tr_read(t + on);
  typedef __attribute__((ext_vector_type(8))) short s16x8;
  return __builtin_bit_cast(bf16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
}
template <bool PAIRED, int COLS>
__device__ __forceinline__ f32x8 frag_col(const float* t, const LaneAt<float, COLS>& l, int k0, int c0) {
  f32x8 f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int r = PAIRED ? (e & 3) + 4 * (e & 4) : e;  // past the lane's own row
    f[e] = t[shifted<LaneAt<float, COLS>>((PAIRED ? l.pair : l.col) ^ (4 * (r & 7)), c0) + (k0 + r) * COLS];
  }
  return f;
}
// Row r0 + i of the lane, columns c0 + 4 g .. + 3.
template <typename T, int COLS>
__device__ __forceinline__ f32x4 tile_get4(const T* t, const LaneAt<T, COLS>& l, int r0, int c0) {
  uint32_t u[4];
  load4_raw<T>(t + shifted<LaneAt<T, COLS>>(l.four, c0) + r0 * COLS, u);
  return unpack4<T>(u);
}
// Rows r0 .. r0 + 15, reduction over columns k0 .. k0 + 31 (plain), of a state of
// 64 columns in memory in the order of accumulators: tiles of 16 x 16, by lane,
// lane i + 16 g with columns 4 g .. 4 g + 3 of row i.
__device__ __forceinline__ f32x8 frag_state(const float* m, int r0, int k0, int lane) {
  const int i = lane & 15, g = lane >> 4;
  const float* p = m + (r0 / 4 + k0 / 16 + (g >> 1)) * 256 + 4 * (i + 32 * (g & 1));
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 64);
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
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

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

}  // namespace kda
