// Checks of arguments shared by the entry points of the layer's operators.
#pragma once

#include <cmath>
#include <stddef.h>
#include <stdint.h>

#include "kda.h"

namespace kda {

// Most sequences named by state_indices: every block compares its index with
// all earlier ones (find_slot in kda_rows.h), about 1 ms a head at this many.
constexpr int32_t kMaxIndexed = 65536;

inline bool known_dtype(int dtype) { return dtype == KDA_F32 || dtype == KDA_BF16; }

// A token stride in elements: `row` when 0; otherwise at least a row and,
// with `vec`, a multiple of 16 bytes. A single token's stride is not used.
inline bool stride_ok(int64_t st, int64_t row, int dtype, int64_t T, bool vec) {
  if (st == 0 || T <= 1) return st >= 0;
  if (st < row) return false;
  return !vec || st % (dtype == KDA_F32 ? 4 : 8) == 0;
}
inline int64_t stride_of(int64_t st, int64_t row) { return st ? st : row; }

// Addresses of a tensor; sizes in 128 bits, so that no problem overflows them.
struct Range {
  const void* at;
  unsigned __int128 bytes;
};
inline Range dense(const void* p, int64_t a, int64_t b, size_t elem) {
  return Range{p, static_cast<unsigned __int128>(a) * b * elem};
}
// T rows of `row` elements, `st` apart
inline Range rows_of(const void* p, int64_t T, int64_t st, int64_t row, size_t elem) {
  return Range{p, (static_cast<unsigned __int128>(T - 1) * st + row) * elem};
}
// Whether the state, which sequences write while others still read their
// inputs, shares an address with one of `n` tensors (null ones: none).
inline bool over_any(const Range& state, const Range* others, int n) {
  const unsigned __int128 s = reinterpret_cast<uintptr_t>(state.at);
  for (int i = 0; i < n; ++i) {
    const unsigned __int128 x = reinterpret_cast<uintptr_t>(others[i].at);
    if (x && x < s + state.bytes && s < x + others[i].bytes) return true;
  }
  return false;
}

inline bool bad_eps(float eps) { return !(eps >= 0.f) || !std::isfinite(eps); }

}  // namespace kda
