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

// ---- pairs of fp32 in one 64-bit register: one instruction for two elements
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// eight elements as four pairs
template <int DTYPE>
__device__ __forceinline__ void unpack8x2(const uint4 &v, uint64_t (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2<DTYPE>(w[i]);
    f[i] = pack_f32x2(p.x, p.y);
  }
}
template <int DTYPE>
__device__ __forceinline__ uint4 pack8x2(const uint64_t (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack_f32x2(f[i]);
    w[i] = pack2<DTYPE>(p.x, p.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int DTYPE>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
  const uint32_t v = static_cast<const uint16_t *>(p)[i];
  return unpack2<DTYPE>(v).x;
}

}  // namespace moe
