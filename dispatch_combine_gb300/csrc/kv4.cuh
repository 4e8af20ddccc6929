// kv4.cuh -- the 4-bit form of the paged key/value cache.
//
// A row of a head is cut into groups of 32 elements.  A group is one fp16 scale
// s = rn(max|v| / 7) and a whole number n - 8 from -7 to 7 for each element,
// v / s rounded to even, held as the nibble n; it stands for (n - 8) * s.  A
// group that holds a NaN or an infinity, or whose scale passes fp16, has the
// scale NaN; one whose scale rounds to zero stands for zeros.
//
// A cache is [num_pages, num_kv_heads, page_size * (D / 2 + D / 16)] bytes: the
// codes of a page's rows of one head, D / 2 bytes each, then their scales, D / 32
// each.  Within a row the codes stand as the attention's matrix instructions
// take them, so that its lanes load them in one piece (NB = D / 32 groups;
// element e of group b, low nibble first):
//   keys:   lane t = e / 8 of four reads bytes [4 NB t, 4 NB (t + 1)); the eight
//           elements of group b are its word b;
//   values: lane g = e / 4 of eight reads bytes [2 NB g, 2 NB (g + 1)); the four
//           elements of group b are its 16-bit piece b.
#pragma once

#include "elem.cuh"
#include "kernels.h"

namespace moe {

constexpr int kGroup4 = 32;
__host__ __device__ constexpr int kv4_code_bytes(int D) { return D / 2; }
__host__ __device__ constexpr int kv4_scale_bytes(int D) { return D / 16; }
__host__ __device__ constexpr int kv4_row_bytes(int D) { return D / 2 + D / 16; }

// byte of a key row's word (group b, lane t) and of a value row's piece (b, lane g)
__device__ __forceinline__ int kv4_key_at(int D, int b, int t) { return t * (D / 8) + 4 * b; }
__device__ __forceinline__ int kv4_value_at(int D, int b, int g) { return g * (D / 16) + 2 * b; }

}  // namespace moe
