// shifted.cuh -- 8 neighbouring 16-bit elements of rows that lie at any address:
// odd widths and pitches put most rows off 16-byte boundaries.
//
// A load takes the two 16-byte words that the elements lie in and shifts them
// together; no byte outside of the row is read (pieces at a row's ends go element by
// element, with zeros outside of it). The words overlap those of the neighbouring
// threads, so the second comes from L1. Kernels that may choose lay their pieces out
// by the rows that they write, so that stores are whole words.
#pragma once

#include <cstdint>

namespace sptg {

// Elements between the 16-byte boundary at or below p and p.
__device__ __forceinline__ int shift_of(const void* p) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) >> 1);
}

// Two 16-byte words and the number of elements that a piece of 8 lies into them.
// Their loads need no branch, so that those of several rows are in flight together.
struct ShiftedPiece {
  uint4 a, b;
  int shift;
};

// Whether elements first ... first + 7 of a row, wherever it lies, can be loaded so:
// both words are inside of the row.
__device__ __forceinline__ bool inside_row(int first, int cols) { return first >= 7 && first + 16 <= cols; }

__device__ __forceinline__ ShiftedPiece load_words(const uint16_t* p) {
  ShiftedPiece r;
  r.shift = shift_of(p);
  const uint4* w = reinterpret_cast<const uint4*>(p - r.shift);
  r.a = w[0];
  r.b = w[r.shift ? 1 : 0];
  return r;
}

__device__ __forceinline__ uint4 shifted(const ShiftedPiece& r) {
  const int s = r.shift;
  uint32_t v[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) v[i] = s & 4 ? v[i + 2] : v[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) v[i] = s & 2 ? v[i + 1] : v[i];
  const uint32_t bits = s & 1 ? 16 : 0;
  return make_uint4(__funnelshift_r(v[0], v[1], bits), __funnelshift_r(v[1], v[2], bits),
                    __funnelshift_r(v[2], v[3], bits), __funnelshift_r(v[3], v[4], bits));
}

// Elements first ... first + 7 of a row of `cols` (first may be negative), zeros
// outside of it, one by one: for the ends of rows.
__device__ __forceinline__ uint4 load_elements(const uint16_t* row, int first, int cols) {
  const uint16_t* p = row + first;
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = first + 2 * i;
    const uint32_t lo = e >= 0 && e < cols ? p[2 * i] : 0u;
    const uint32_t hi = e + 1 >= 0 && e + 1 < cols ? p[2 * i + 1] : 0u;
    v[i] = lo | (hi << 16);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// The same, by words where they can be.
__device__ __forceinline__ uint4 load_shifted(const uint16_t* row, int first, int cols) {
  return inside_row(first, cols) ? shifted(load_words(row + first)) : load_elements(row, first, cols);
}

// A row of `cols` elements cut by the boundaries of `out`, a row of the same width:
// pieces of 8 from `body` to `tail`, all inside_row() and on out's boundaries, and
// the elements before and after them, which are left to single threads.
struct CutRow {
  int body, tail, ends;  // ends: how many elements are not in pieces
  __device__ __forceinline__ CutRow(const uint16_t* out, int cols) {
    const int shift = shift_of(out);
    body = min(cols, ((14 + shift) & ~7) - shift);
    tail = body + (max(0, cols - 8 - body) & ~7);
    ends = body + cols - tail;
  }
  __device__ __forceinline__ int end(int i) const { return i < body ? i : tail + i - body; }
};

// The same elements stored: one word where they are one, else as many of 4 bytes as
// lie on their boundaries.
__device__ __forceinline__ void store_shifted(uint16_t* row, int first, int cols, const uint4& v) {
  uint16_t* p = row + first;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (first >= 0 && first + 8 <= cols) {
    const int s = shift_of(p);
    if (s == 0) {
      *reinterpret_cast<uint4*>(p) = v;
    } else if ((s & 1) == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(p)[i] = w[i];
    } else {
      p[0] = static_cast<uint16_t>(w[0]);
#pragma unroll
      for (int i = 0; i < 3; ++i)
        reinterpret_cast<uint32_t*>(p + 1)[i] = __funnelshift_r(w[i], w[i + 1], 16);
      p[7] = static_cast<uint16_t>(w[3] >> 16);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (first + i >= 0 && first + i < cols) p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
}

// Elements `first` to first + 7 of a row; ALIGNED: rows lie on 16-byte boundaries,
// and so do pieces.
template <bool ALIGNED>
__device__ __forceinline__ uint4 load_piece(const uint16_t* row, int first, int cols) {
  if constexpr (ALIGNED) return *reinterpret_cast<const uint4*>(row + first);
  return load_shifted(row, first, cols);
}
template <bool ALIGNED>
__device__ __forceinline__ void store_piece(uint16_t* row, int first, int cols, const uint4& v) {
  if constexpr (ALIGNED)
    *reinterpret_cast<uint4*>(row + first) = v;
  else
    store_shifted(row, first, cols, v);
}

}  // namespace sptg
