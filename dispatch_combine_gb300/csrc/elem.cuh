// elem.cuh -- the two 16-bit element types of the block operators (bf16 and
// fp16): packed pairs to and from fp32, and 16-byte vectors of eight.
#pragma once

#include "common.cuh"

namespace moe {

template <int DTYPE>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if (DTYPE == MOE_DTYPE_BF16) return make_float2(bf16lo(v), bf16hi(v));
  return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}

// round to nearest even, lo in the low half
template <int DTYPE>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return DTYPE == MOE_DTYPE_BF16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
}

template <int DTYPE>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2<DTYPE>(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

template <int DTYPE>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<DTYPE>(f[0], f[1]), pack2<DTYPE>(f[2], f[3]), pack2<DTYPE>(f[4], f[5]),
                    pack2<DTYPE>(f[6], f[7]));
}

template <int DTYPE>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
  const uint32_t v = static_cast<const uint16_t *>(p)[i];
  return unpack2<DTYPE>(v).x;
}

}  // namespace moe
