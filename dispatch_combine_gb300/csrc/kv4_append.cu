// kv4_append.cu -- the 4-bit cache as it is written (moe_kv4_append: rotation,
// quantisation, paged write) and read back to 16 bits (moe_kv4_read).
//
//   k' = R(position) k;  per 32 elements s = rn16(max|k'| / 7), n = rn(k' / s) + 8
// Both are bound by HBM: a token's queries, keys and values are read once, and
// what is written of keys and values is 9/32 of it.
#include "kv4.cuh"

namespace moe {
namespace {

constexpr int kUnroll4 = 4;  // units per thread whose loads are in flight together

// Rotation of one pair, every product and sum rounded by itself, so that a key
// near the border between two codes does not depend on what the compiler fuses.
__device__ __forceinline__ float turned_lo(float x, float y, float c, float s) {
  return __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
}
__device__ __forceinline__ float turned_hi(float x, float y, float c, float s) {
  return __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

// The scale of a group with largest magnitude `top` (NaN for one that is not
// finite), as fp16 bits.
__device__ __forceinline__ uint16_t scale4(float top) {
  const float s = __fdiv_rn(top, 7.0f);
  const uint16_t bits = __half_as_ushort(__float2half_rn(s));
  return (bits & 0x7C00u) == 0x7C00u ? uint16_t{0x7E00} : bits;
}
// Eight elements to their nibbles, the first lowest.  The quotient is rounded
// once: of 16-bit values and scales it is exact enough to meet a border only
// where it lies on it.
__device__ __forceinline__ uint32_t codes8(const float (&f)[8], float s) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float n = s > 0.0f ? rintf(__fdiv_rn(f[e], s)) : 0.0f;
    n = fminf(fmaxf(n, -7.0f), 7.0f);
    w |= static_cast<uint32_t>(static_cast<int>(n) + 8) << (4 * e);
  }
  return w;
}

// One CTA per token.  Units: a query head's pairs of 16-byte vectors, as
// kv_append.cu takes them; then the vectors of the key heads and of the value
// heads one by one, so that four neighbouring lanes hold a group of 32 (a key's
// vector fetches the one that it turns with beside itself).
template <int DTYPE>
__global__ void __launch_bounds__(512, 2) kv4_append_kernel(const KvAppendArgs a) {
  pdl_begin();
  __shared__ float s_cos[64], s_sin[64];
  const int t = blockIdx.x;
  const int upr = a.D / 16, vpr = a.D / 8;
  const int nq = a.q ? a.hq * upr : 0, nkv = a.hkv * vpr;
  const int units = nq + 2 * nkv;
  const int32_t slot = a.slots[t];
  const bool bad = slot < -1 || static_cast<int64_t>(slot) >= a.num_slots;
  const bool skip = slot < 0 || bad;
  if (bad && threadIdx.x == 0) set_status(a.status, kStatusBadId);
  const int half = a.rot / 2;
  const int64_t page = slot >> a.page_shift;
  const int in_page = slot & ((1 << a.page_shift) - 1);
  const int64_t page_bytes = static_cast<int64_t>(kv4_row_bytes(a.D)) << a.page_shift;
  bool first = true;
  // (every thread passes the loop once, for the barrier inside; whole warps stay
  // together for the groups' maxima)
  for (int base = threadIdx.x; first || base - (threadIdx.x & 31) < units;
       base += blockDim.x * kUnroll4) {
    uint4 lo[kUnroll4], hi[kUnroll4];
#pragma unroll
    for (int j = 0; j < kUnroll4; ++j) {
      const int u = base + j * blockDim.x;
      lo[j] = hi[j] = make_uint4(0, 0, 0, 0);
      if (u >= units || (skip && u >= nq)) continue;
      if (u < nq) {
        const int head = u / upr, c = u - head * upr;
        const bool rot_half = a.style == MOE_ROPE_HALF && 16 * c < a.rot;
        const int e0 = rot_half ? 8 * c : 16 * c;
        const uint16_t *row = static_cast<const uint16_t *>(a.q) + t * a.q_stride + head * a.D;
        lo[j] = *reinterpret_cast<const uint4 *>(row + e0);
        hi[j] = *reinterpret_cast<const uint4 *>(row + e0 + (rot_half ? half : 8));
      } else {
        const bool is_k = u < nq + nkv;
        const int i = u - nq - (is_k ? 0 : nkv);
        const int head = i / vpr, e0 = 8 * (i - head * vpr);
        const uint16_t *row =
            (is_k ? static_cast<const uint16_t *>(a.k) + t * a.k_stride
                  : static_cast<const uint16_t *>(a.v) + t * a.v_stride) + head * a.D;
        lo[j] = *reinterpret_cast<const uint4 *>(row + e0);
        if (is_k && a.style == MOE_ROPE_HALF && e0 < a.rot)
          hi[j] = *reinterpret_cast<const uint4 *>(row + (e0 < half ? e0 + half : e0 - half));
      }
    }
    if (first) {  // with the first units on their way
      first = false;
      for (int i = threadIdx.x; i < half; i += blockDim.x) {
        // turns = position * inv_freq / 2 pi, its fraction in fp64, sine and cosine
        // rounded once from fp64: a key near a border goes where 64 bits put it
        const double turns = static_cast<double>(a.positions[t]) * static_cast<double>(a.inv_freq[i]) *
                             0.15915494309189535;
        double sn, cs;
        sincospi(2.0 * (turns - rint(turns)), &sn, &cs);
        s_sin[i] = static_cast<float>(sn);
        s_cos[i] = static_cast<float>(cs);
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kUnroll4; ++j) {
      const int u = base + j * blockDim.x;
      if (u - (threadIdx.x & 31) >= units) continue;  // the whole warp
      const bool is_q = u < nq, is_k = !is_q && u < nq + nkv;
      const int i = is_q ? u : u - nq - (is_k ? 0 : nkv);
      const int per = is_q ? upr : vpr;
      const int head = i / per, c = i - head * per;
      float x[8], y[8];
      unpack8<DTYPE>(lo[j], x);
      unpack8<DTYPE>(hi[j], y);
      if (is_q) {
        const bool rot_half = a.style == MOE_ROPE_HALF && 16 * c < a.rot;
        const int e0 = rot_half ? 8 * c : 16 * c, e1 = e0 + (rot_half ? half : 8);
        if (16 * c < a.rot) {
          if (rot_half) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float cs = s_cos[e0 + e], sn = s_sin[e0 + e];
              const float p = turned_lo(x[e], y[e], cs, sn);
              y[e] = turned_hi(x[e], y[e], cs, sn);
              x[e] = p;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const int k = (e0 + e) / 2;
              const float p = turned_lo(x[e], x[e + 1], s_cos[k], s_sin[k]);
              x[e + 1] = turned_hi(x[e], x[e + 1], s_cos[k], s_sin[k]);
              x[e] = p;
              const float r = turned_lo(y[e], y[e + 1], s_cos[k + 4], s_sin[k + 4]);
              y[e + 1] = turned_hi(y[e], y[e + 1], s_cos[k + 4], s_sin[k + 4]);
              y[e] = r;
            }
          }
          lo[j] = pack8<DTYPE>(x);
          hi[j] = pack8<DTYPE>(y);
        }
        uint16_t *row = static_cast<uint16_t *>(a.q_out) + t * a.q_out_stride + head * a.D;
        *reinterpret_cast<uint4 *>(row + e0) = lo[j];
        *reinterpret_cast<uint4 *>(row + e1) = hi[j];
      }
      const int e0 = 8 * c;
      if (is_k && e0 < a.rot) {
        if (a.style == MOE_ROPE_HALF) {
          const bool up = e0 >= half;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int k = e0 + e - (up ? half : 0);
            x[e] = up ? turned_hi(y[e], x[e], s_cos[k], s_sin[k])
                      : turned_lo(x[e], y[e], s_cos[k], s_sin[k]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const int k = (e0 + e) / 2;
            const float p = turned_lo(x[e], x[e + 1], s_cos[k], s_sin[k]);
            x[e + 1] = turned_hi(x[e], x[e + 1], s_cos[k], s_sin[k]);
            x[e] = p;
          }
        }
      }
      // the group's largest magnitude; as bits, so that an infinity or a NaN wins
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      if (is_q || u >= units || skip) continue;
      const uint16_t s16 = scale4(__uint_as_float(top));
      const uint32_t w = codes8(x, __half2float(__ushort_as_half(s16)));
      const int b = c >> 2, part = c & 3;  // group, and eight elements of it
      uint8_t *at = static_cast<uint8_t *>(is_k ? a.k_cache : a.v_cache) +
                    (page * a.hkv + head) * page_bytes;
      if (is_k) {
        *reinterpret_cast<uint32_t *>(at + kv4_key_at(a.D, in_page, b, part)) = w;
      } else {
        *reinterpret_cast<uint16_t *>(at + kv4_value_at(a.D, in_page, b, 2 * part)) =
            static_cast<uint16_t>(w);
        *reinterpret_cast<uint16_t *>(at + kv4_value_at(a.D, in_page, b, 2 * part + 1)) =
            static_cast<uint16_t>(w >> 16);
      }
      if (part == 0)
        *reinterpret_cast<uint16_t *>(at + (kv4_code_bytes(a.D) << a.page_shift) +
                                      (is_k ? kv4_key_scale_at(a.D, in_page, b)
                                            : kv4_value_scale_at(a.D, in_page, b))) = s16;
    }
  }
}

// Eight elements (16 bytes of output) per thread and unit; the units of a row's
// keys, then of its values.
template <int DTYPE>
__global__ void __launch_bounds__(256) kv4_read_kernel(const Kv4ReadArgs a) {
  pdl_begin();
  const int vpr = a.D / 8, per_row = 2 * a.hkv * vpr;
  const int64_t units = static_cast<int64_t>(a.n) * per_row;
  const int64_t page_bytes = static_cast<int64_t>(kv4_row_bytes(a.D)) << a.page_shift;
  const int mask = (1 << a.page_shift) - 1;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; u < units;
       u += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int i = static_cast<int>(u / per_row);
    const int j = static_cast<int>(u - static_cast<int64_t>(i) * per_row);
    const int32_t slot = a.slots[i];
    const int32_t dst = a.dst_slots ? a.dst_slots[i] : i;
    if (slot < -1 || slot >= a.num_slots || (a.dst_slots && (dst < -1 || dst >= a.dst_num_slots))) {
      if (j == 0) set_status(a.status, kStatusBadId);
      continue;
    }
    if (slot < 0 || dst < 0) continue;
    const bool is_k = j < a.hkv * vpr;
    const int h = (j - (is_k ? 0 : a.hkv * vpr)) / vpr, c = j % vpr;
    const int b = c >> 2, part = c & 3;
    const uint8_t *at = (is_k ? a.k_cache : a.v_cache) +
                        (static_cast<int64_t>(slot >> a.page_shift) * a.hkv + h) * page_bytes;
    const int r = slot & mask;
    uint32_t w;
    if (is_k)
      w = *reinterpret_cast<const uint32_t *>(at + kv4_key_at(a.D, r, b, part));
    else
      w = *reinterpret_cast<const uint16_t *>(at + kv4_value_at(a.D, r, b, 2 * part)) |
          static_cast<uint32_t>(
              *reinterpret_cast<const uint16_t *>(at + kv4_value_at(a.D, r, b, 2 * part + 1)))
              << 16;
    const float s = __half2float(__ushort_as_half(*reinterpret_cast<const uint16_t *>(
        at + (kv4_code_bytes(a.D) << a.page_shift) +
        (is_k ? kv4_key_scale_at(a.D, r, b) : kv4_value_scale_at(a.D, r, b)))));
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      f[e] = static_cast<float>(static_cast<int>((w >> (4 * e)) & 15u) - 8) * s;
    uint16_t *out = static_cast<uint16_t *>(is_k ? a.k_out : a.v_out);
    if (a.dst_slots)
      out += (((static_cast<int64_t>(dst >> a.page_shift) * a.hkv + h) << a.page_shift) + (dst & mask)) * a.D;
    else
      out += i * (is_k ? a.k_stride : a.v_stride) + h * a.D;
    *reinterpret_cast<uint4 *>(out + 8 * c) = pack8<DTYPE>(f);
  }
}

}  // namespace

cudaError_t launch_kv4_append(const KvAppendArgs &a, int dtype, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const int units = ((a.q ? a.hq : 0) + 4 * a.hkv) * (a.D / 16);
  int threads = (units + kUnroll4 * 32 - 1) / (kUnroll4 * 32) * 32;
  if (threads > 512) threads = 512;
  if (dtype == MOE_DTYPE_BF16)
    MOE_LAUNCH_PDL(kv4_append_kernel<MOE_DTYPE_BF16>, static_cast<unsigned>(a.T), threads, 0, s, a);
  else
    MOE_LAUNCH_PDL(kv4_append_kernel<MOE_DTYPE_FP16>, static_cast<unsigned>(a.T), threads, 0, s, a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4ReadArgs &a, int dtype, cudaStream_t s) {
  if (a.n == 0) return cudaSuccess;
  const int64_t units = static_cast<int64_t>(a.n) * a.hkv * (a.D / 4);
  const int64_t ctas = (units + 255) / 256, most = static_cast<int64_t>(num_sms()) * 64;
  const unsigned grid = static_cast<unsigned>(ctas < most ? ctas : most);
  if (dtype == MOE_DTYPE_BF16)
    MOE_LAUNCH_PDL(kv4_read_kernel<MOE_DTYPE_BF16>, grid, 256, 0, s, a);
  else
    MOE_LAUNCH_PDL(kv4_read_kernel<MOE_DTYPE_FP16>, grid, 256, 0, s, a);
  return cudaGetLastError();
}

}  // namespace moe
