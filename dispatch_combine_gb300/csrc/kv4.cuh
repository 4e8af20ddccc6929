// kv4.cuh -- the 4-bit form of the paged key/value cache.
//
// A row of a head is cut into groups of 32 elements.  A group is one fp16 scale
// s = rn(max|v| / 7) and a whole number n - 8 from -7 to 7 for each element,
// v / s rounded to even, held as the nibble n; it stands for (n - 8) * s.  A
// group that holds a NaN or an infinity, or whose scale passes fp16, has the
// scale NaN; one whose scale rounds to zero stands for zeros.
//
// A cache is [num_pages, num_kv_heads, page_size * (D / 2 + D / 16)] bytes: the
// codes of a page's rows of one head, D / 2 bytes each, then their scales, D / 16
// each.  The codes stand as the attention's matrix instructions take them, so
// that its lanes load them in one piece (NB = D / 32 groups; low nibble first):
//   keys:   lane t of four reads bytes [4 NB t, 4 NB (t + 1)) of a row; elements 8t
//           to 8t + 7 of group b are its word b;
//   values: two rows 2i and 2i + 1 stand together; lane g of eight reads bytes
//           [4 NB g, 4 NB (g + 1)) of the pair, whose word b is elements 4g to 4g + 3
//           of group b, of the even row in its low half and of the odd one in its
//           high half.  Lanes that load together take pairs 0 to 3 of eight rows;
//           so that they meet different banks of shared memory, into which whole
//           runs are copied, pair i's bytes are turned by 32 i (D = 128), or the
//           halves of every third and fourth pair changed over (D = 64).
// Scales of keys stand row by row; those of values by pairs of rows, the two of a
// group side by side.
#pragma once

#include "elem.cuh"
#include "kernels.h"

namespace moe {

constexpr int kGroup4 = 32;
__host__ __device__ constexpr int kv4_code_bytes(int D) { return D / 2; }
__host__ __device__ constexpr int kv4_scale_bytes(int D) { return D / 16; }
__host__ __device__ constexpr int kv4_row_bytes(int D) { return D / 2 + D / 16; }

// how the bytes of a pair of value rows are turned
__device__ __forceinline__ int kv4_value_turn(int D, int pair, int at) {
  return D == 128 ? (at + 32 * (pair & 3)) & 127 : at ^ ((pair & 2) << 4);
}
// place among the codes of a key row's word (row r, group b, lane t) and of a
// value row's piece (row r, group b, lane g)
__device__ __forceinline__ int kv4_key_at(int D, int r, int b, int t) {
  return r * kv4_code_bytes(D) + t * (D / 8) + 4 * b;
}
__device__ __forceinline__ int kv4_value_at(int D, int r, int b, int g) {
  const int pair = r >> 1;
  return pair * (2 * kv4_code_bytes(D)) + kv4_value_turn(D, pair, g * (D / 8)) + 4 * b + 2 * (r & 1);
}
// and of the scale of row r's group b among the scales
__device__ __forceinline__ int kv4_key_scale_at(int D, int r, int b) {
  return r * kv4_scale_bytes(D) + 2 * b;
}
__device__ __forceinline__ int kv4_value_scale_at(int D, int r, int b) {
  return (r >> 1) * (2 * kv4_scale_bytes(D)) + 4 * b + 2 * (r & 1);
}

}  // namespace moe
