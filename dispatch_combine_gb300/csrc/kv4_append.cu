// kv4_append.cu -- the 4-bit cache as it is written (moe_kv4_append: rotation,
// quantisation, paged write) and read back to 16 bits (moe_kv4_read).
//
//   k' = R(position) k;  per 32 elements s = rn16(max|k'| / 7), n = rn(k' / s) + 8
// Both are bound by HBM where there are many rows: a token's queries, keys and values
// are read once, and what is written of keys and values is 9/32 of it.  16384 tokens
// of 64 + 8 heads of 128 appended and read back (690 MB) take 119 us, 0.86 of the
// measured copy bandwidth; 131072 rows of 8 heads of 128 read back into a 16-bit
// cache (689 MB, 538 of them written) 117 us, 0.87.  Few rows cost their launch: 64 tokens appended and
// read back 5.2 us.
//   What the append was bound by first was arithmetic: with sines in 64 bits and
// divisions as they are written (119 us now) it was 216, with either of the two
// replaced 194.
#include "kv4.cuh"

namespace moe {
namespace {

// Sine and cosine of a position's angle.  A key near the border between two codes
// goes where 64 bits put it only if both are as good as fp32 can hold them, and the
// 64-bit units of a GB300 would take longer over them than the memory over
// everything else.  So the angle is a whole number of 2^-64 turns (exact as positions
// multiply; the frequency's own rounding to 53 bits is the only error), its upper six
// bits pick a tabled angle a, the rest is d, |d| <= 2 pi / 128, and
//   sin(a + d) = sin a + (cos a sin d + sin a (cos d - 1)),  cos likewise,
// with the table and d in two fp32 numbers each and short Taylor series.  The error
// before the one rounding to fp32 is 2e-10 (1 in 900 is not the nearest number).
struct Sine {
  float high, low;  // of sin(2 pi k / 64)
};
__device__ const Sine kSines[80] = {
    {0.0e+00f, 0.0e+00f}, {9.801714e-02f, -8.933932e-10f}, {1.9509032e-01f, -1.6704714e-09f}, {2.9028466e-01f, 1.3815665e-08f},
    {3.8268343e-01f, 6.2233507e-09f}, {4.7139674e-01f, -7.4252537e-09f}, {5.5557024e-01f, -1.1769521e-08f}, {6.343933e-01f, 9.379558e-09f},
    {7.0710677e-01f, 1.21016175e-08f}, {7.7301043e-01f, 2.0642553e-08f}, {8.314696e-01f, 1.6870263e-08f}, {8.819213e-01f, -2.7002963e-08f},
    {9.238795e-01f, 2.830749e-08f}, {9.5694035e-01f, -1.7184508e-08f}, {9.8078525e-01f, 2.9739473e-08f}, {9.951847e-01f, 7.109666e-09f},
    {1.0e+00f, 0.0e+00f}, {9.951847e-01f, 7.109666e-09f}, {9.8078525e-01f, 2.9739473e-08f}, {9.5694035e-01f, -1.7184508e-08f},
    {9.238795e-01f, 2.830749e-08f}, {8.819213e-01f, -2.7002963e-08f}, {8.314696e-01f, 1.6870263e-08f}, {7.7301043e-01f, 2.0642553e-08f},
    {7.0710677e-01f, 1.21016175e-08f}, {6.343933e-01f, 9.379558e-09f}, {5.5557024e-01f, -1.1769521e-08f}, {4.7139674e-01f, -7.4252537e-09f},
    {3.8268343e-01f, 6.2233507e-09f}, {2.9028466e-01f, 1.3815665e-08f}, {1.9509032e-01f, -1.6704714e-09f}, {9.801714e-02f, -8.933932e-10f},
    {0.0e+00f, 0.0e+00f}, {-9.801714e-02f, 8.933932e-10f}, {-1.9509032e-01f, 1.6704714e-09f}, {-2.9028466e-01f, -1.3815665e-08f},
    {-3.8268343e-01f, -6.2233507e-09f}, {-4.7139674e-01f, 7.4252537e-09f}, {-5.5557024e-01f, 1.1769521e-08f}, {-6.343933e-01f, -9.379558e-09f},
    {-7.0710677e-01f, -1.21016175e-08f}, {-7.7301043e-01f, -2.0642553e-08f}, {-8.314696e-01f, -1.6870263e-08f}, {-8.819213e-01f, 2.7002963e-08f},
    {-9.238795e-01f, -2.830749e-08f}, {-9.5694035e-01f, 1.7184508e-08f}, {-9.8078525e-01f, -2.9739473e-08f}, {-9.951847e-01f, -7.109666e-09f},
    {-1.0e+00f, 0.0e+00f}, {-9.951847e-01f, -7.109666e-09f}, {-9.8078525e-01f, -2.9739473e-08f}, {-9.5694035e-01f, 1.7184508e-08f},
    {-9.238795e-01f, -2.830749e-08f}, {-8.819213e-01f, 2.7002963e-08f}, {-8.314696e-01f, -1.6870263e-08f}, {-7.7301043e-01f, -2.0642553e-08f},
    {-7.0710677e-01f, -1.21016175e-08f}, {-6.343933e-01f, -9.379558e-09f}, {-5.5557024e-01f, 1.1769521e-08f}, {-4.7139674e-01f, 7.4252537e-09f},
    {-3.8268343e-01f, -6.2233507e-09f}, {-2.9028466e-01f, -1.3815665e-08f}, {-1.9509032e-01f, 1.6704714e-09f}, {-9.801714e-02f, 8.933932e-10f},
    {0.0e+00f, 0.0e+00f}, {9.801714e-02f, -8.933932e-10f}, {1.9509032e-01f, -1.6704714e-09f}, {2.9028466e-01f, 1.3815665e-08f},
    {3.8268343e-01f, 6.2233507e-09f}, {4.7139674e-01f, -7.4252537e-09f}, {5.5557024e-01f, -1.1769521e-08f}, {6.343933e-01f, 9.379558e-09f},
    {7.0710677e-01f, 1.21016175e-08f}, {7.7301043e-01f, 2.0642553e-08f}, {8.314696e-01f, 1.6870263e-08f}, {8.819213e-01f, -2.7002963e-08f},
    {9.238795e-01f, 2.830749e-08f}, {9.5694035e-01f, -1.7184508e-08f}, {9.8078525e-01f, 2.9739473e-08f}, {9.951847e-01f, 7.109666e-09f},
};
__device__ __forceinline__ uint64_t turns64(float inv_freq) {  // per position, modulo 1
  const double g = static_cast<double>(inv_freq) * 0.15915494309189535;
  return __double2ull_rn((g - floor(g)) * 18446744073709551616.0);
}
// sin (cos: sign -1) of a + d from sin a, cos a (cos a, sin a)
__device__ __forceinline__ float turned(const Sine &a, const Sine &b, float sign, float d, float dl,
                                        float sd, float cd) {
  const float bh = sign * b.high, bl = sign * b.low;
  const float t = __fmul_rn(bh, d);
  const float rest = __fadd_rn(fmaf(a.high, cd, fmaf(bl, d, fmaf(bh, sd, a.low))), fmaf(bh, d, -t));
  const float u = __fadd_rn(a.high, t);
  return __fadd_rn(u, __fadd_rn(__fsub_rn(t, __fsub_rn(u, a.high)), rest));
}
__device__ __forceinline__ void sine_cosine(uint64_t turns, float *sn, float *cs) {
  const uint64_t up = turns + (uint64_t{1} << 57);
  const int k = static_cast<int>(up >> 58);
  const int part = static_cast<int>(static_cast<uint32_t>(up >> 26) ^ 0x80000000u);
  // part * 2^-38 turns, as d + dl
  const float h = static_cast<float>(part);
  const float l = static_cast<float>(part - __float2int_rn(h));
  constexpr double kUnit = 6.283185307179586 / 274877906944.0;
  constexpr float kHigh = static_cast<float>(kUnit), kLow = static_cast<float>(kUnit - kHigh);
  const float d = __fmul_rn(h, kHigh);
  const float dl = fmaf(l, kHigh, fmaf(h, kLow, fmaf(h, kHigh, -d)));
  const float z = d * d;
  const float sd = fmaf(d * z, fmaf(z, 1.0f / 120, -1.0f / 6), dl);  // sin d - d
  const float cd = fmaf(-d, dl, z * fmaf(z, fmaf(z, -1.0f / 720, 1.0f / 24), -0.5f));
  const Sine s = kSines[k], c = kSines[k + 16];
  *sn = turned(s, c, 1.0f, d, dl, sd, cd);
  *cs = turned(c, s, -1.0f, d, dl, sd, cd);
}

__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The scale of a group with largest magnitude `top` (NaN for one that is not
// finite), as fp16 bits.
__device__ __forceinline__ uint16_t scale4(float top) {
  const float s = __fdiv_rn(top, 7.0f);
  const uint16_t bits = __half_as_ushort(__float2half_rn(s));
  return (bits & 0x7C00u) == 0x7C00u ? uint16_t{0x7E00} : bits;
}
// Eight elements to their nibbles, the first lowest.  The quotient f / s is
// rounded once (Markstein's theorem: a quotient from the rounded reciprocal,
// corrected by its exact remainder): of 16-bit values and scales it meets a border
// between two codes only where it lies on it.
__device__ __forceinline__ uint32_t codes8(float (&f)[8], float s) {
  if (!(s > 0.0f)) return 0x88888888u;
  if (s < 6.103515625e-5f)  // a subnormal scale may be far off max|v| / 7
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = fminf(fmaxf(f[e], -7.0f * s), 7.0f * s);
  const float inv = __frcp_rn(s);
  // 2^23 + 2^22 + 8 + n: the number's last bits are the nibble
  constexpr uint32_t kMagic = 0x4B400000u;
  uint32_t w = 0;
#pragma unroll
  for (int e = 7; e >= 0; --e) {
    const float q0 = __fmul_rn(f[e], inv);
    const float q = fmaf(fmaf(-q0, s, f[e]), inv, q0);
    w = w * 16 + __float_as_uint(__fadd_rn(q, 12582920.0f));
  }
  return w - kMagic * 0x11111111u;
}

// Where the angle of pair i stands among a token's 64: lanes with neighbouring
// eights of them load four at a time from different banks.
__device__ __forceinline__ int angle_at(int i) {
  return ((i >> 2) & 1) * 32 + (i >> 3) * 4 + (i & 3);
}
// The eight from i on (i % 8 == 0) as pairs
__device__ __forceinline__ void angles8(const float *p, int i, uint64_t (&v)[4]) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(p + (i >> 1));
  const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(p + 32 + (i >> 1));
  v[0] = a.x;
  v[1] = a.y;
  v[2] = b.x;
  v[3] = b.y;
}

// A CTA of eight warps has 8 / W tokens, W warps each.  Units of a token: its
// query heads' pairs of 16-byte vectors (the two that turn with one another, or
// neighbours), then the vectors of its key heads and value heads one by one, so that
// four neighbouring lanes hold a group of 32 (a key's vector fetches the one that it
// turns with beside itself).
constexpr int kUnits = 4;  // of a thread, whose loads are in flight together
template <int DTYPE, int D, int W>
__global__ void __launch_bounds__(256, 4) kv4_append_kernel(const KvAppendArgs a) {
  pdl_begin();
  constexpr int TOKENS = 8 / W, UPR = D / 16, VPR = D / 8;
  __shared__ __align__(16) float s_cos[TOKENS][64], s_sin[TOKENS][64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = warp / W;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * TOKENS + mine;
  const int half = a.rot / 2, first = (warp % W) * 32 + lane;
  const bool turn_half = a.style == MOE_ROPE_HALF;
  const int nq = a.q && t < a.T ? a.hq * UPR : 0;
  const uint16_t *q = static_cast<const uint16_t *>(a.q) + t * a.q_stride;
  uint4 lo[kUnits], hi[kUnits];
  auto load_q = [&](int base) {
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int u = base + j * (32 * W), c = u % UPR;
      if (u >= nq) break;
      const bool far = turn_half && 16 * c < a.rot;
      const uint16_t *row = q + u / UPR * D + (far ? 8 * c : 16 * c);
      lo[j] = *reinterpret_cast<const uint4 *>(row);
      hi[j] = *reinterpret_cast<const uint4 *>(row + (far ? half : 8));
    }
  };
  load_q(first);
  for (int i = threadIdx.x; i < TOKENS * half; i += 256) {  // with the first units on their way
    const int tok = i / half, k = i - tok * half;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * TOKENS + tok;
    if (at < a.T) {
      float sn, cs;
      const float freq = a.inv_freq[k];
      sine_cosine(turns64(freq) * static_cast<uint64_t>(static_cast<int64_t>(a.positions[at])), &sn,
                  &cs);
      if (!isfinite(freq)) sn = cs = NAN;
      s_cos[tok][angle_at(k)] = cs;
      s_sin[tok][angle_at(k)] = sn;
    }
  }
  __syncthreads();
  const float *cosines = s_cos[mine], *sines = s_sin[mine];
  uint16_t *q_out = static_cast<uint16_t *>(a.q_out) + t * a.q_out_stride;
  for (int base = first; base < nq;) {
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int u = base + j * (32 * W), c = u % UPR;
      if (u >= nq) break;
      const bool far = turn_half && 16 * c < a.rot;
      const int e0 = far ? 8 * c : 16 * c;
      if (far) {
        uint64_t x[4], y[4], cs[4], sn[4];
        unpack8x2<DTYPE>(lo[j], x);
        unpack8x2<DTYPE>(hi[j], y);
        angles8(cosines, e0, cs);
        angles8(sines, e0, sn);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t p = sub_f32x2(mul_f32x2(x[e], cs[e]), mul_f32x2(y[e], sn[e]));
          y[e] = fma_f32x2(y[e], cs[e], mul_f32x2(x[e], sn[e]));
          x[e] = p;
        }
        lo[j] = pack8x2<DTYPE>(x);
        hi[j] = pack8x2<DTYPE>(y);
      } else if (16 * c < a.rot) {
        float x[8], y[8];
        unpack8<DTYPE>(lo[j], x);
        unpack8<DTYPE>(hi[j], y);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const int i = angle_at((e0 + e) / 2), k = angle_at((e0 + e) / 2 + 4);
          const float p = fmaf(x[e], cosines[i], -(x[e + 1] * sines[i]));
          x[e + 1] = fmaf(x[e + 1], cosines[i], x[e] * sines[i]);
          x[e] = p;
          const float r = fmaf(y[e], cosines[k], -(y[e + 1] * sines[k]));
          y[e + 1] = fmaf(y[e + 1], cosines[k], y[e] * sines[k]);
          y[e] = r;
        }
        lo[j] = pack8<DTYPE>(x);
        hi[j] = pack8<DTYPE>(y);
      }
      uint16_t *row = q_out + u / UPR * D + e0;
      *reinterpret_cast<uint4 *>(row) = lo[j];
      *reinterpret_cast<uint4 *>(row + (far ? half : 8)) = hi[j];
    }
    base += kUnits * 32 * W;
    if (base < nq) load_q(base);
  }

  // ---- keys and values
  if (t >= a.T) return;
  const int32_t slot = a.slots[t];
  const bool bad = slot < -1 || static_cast<int64_t>(slot) >= a.num_slots;
  if (bad && first == 0) set_status(a.status, kStatusBadId);
  if (slot < 0 || bad) return;
  const int nkv = a.hkv * VPR;
  const int page_bytes = kv4_row_bytes(D) << a.page_shift;
  const int64_t page_at = static_cast<int64_t>(slot >> a.page_shift) * a.hkv * page_bytes;
  const int in_page = slot & ((1 << a.page_shift) - 1);
  const int scales_at = kv4_code_bytes(D) << a.page_shift;
  const uint16_t *kr = static_cast<const uint16_t *>(a.k) + t * a.k_stride;
  const uint16_t *vr = static_cast<const uint16_t *>(a.v) + t * a.v_stride;
  for (int base = first; base - lane < 2 * nkv; base += kUnits * 32 * W) {  // whole warps
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int u = base + j * (32 * W), e0 = 8 * (u % VPR);
      if (u >= 2 * nkv) {
        lo[j] = make_uint4(0, 0, 0, 0);
        continue;
      }
      const uint16_t *row = u < nkv ? kr + 8 * u : vr + 8 * (u - nkv);
      lo[j] = *reinterpret_cast<const uint4 *>(row);
      if (u < nkv && turn_half && e0 < a.rot)
        hi[j] = *reinterpret_cast<const uint4 *>(row + (e0 < half ? half : -half));
    }
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int u = base + j * (32 * W), c = u % VPR, e0 = 8 * c;
      if (u - lane >= 2 * nkv) break;
      const bool is_k = u < nkv;
      float x[8];
      unpack8<DTYPE>(lo[j], x);
      if (is_k && e0 < a.rot) {
        if (turn_half) {
          // every product and sum rounded by itself, so that a key near a border does
          // not depend on what is fused
          uint64_t xx[4], y[4], cs[4], sn[4];
          const bool up = e0 >= half;
          unpack8x2<DTYPE>(hi[j], y);
          angles8(cosines, up ? e0 - half : e0, cs);
          angles8(sines, up ? e0 - half : e0, sn);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint64_t one = mul_f32x2(pack_f32x2(x[2 * e], x[2 * e + 1]), cs[e]);
            const uint64_t two = mul_f32x2(y[e], sn[e]);
            xx[e] = up ? add_f32x2(one, two) : sub_f32x2(one, two);
            const float2 r = unpack_f32x2(xx[e]);
            x[2 * e] = r.x;
            x[2 * e + 1] = r.y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const int k = angle_at((e0 + e) / 2);
            const float p = __fsub_rn(__fmul_rn(x[e], cosines[k]), __fmul_rn(x[e + 1], sines[k]));
            x[e + 1] = __fadd_rn(__fmul_rn(x[e + 1], cosines[k]), __fmul_rn(x[e], sines[k]));
            x[e] = p;
          }
        }
      }
      float top = max_nan(fabsf(x[0]), fabsf(x[1]));
      top = max_nan(top, fabsf(x[2]), fabsf(x[3]));
      top = max_nan(top, fabsf(x[4]), fabsf(x[5]));
      top = max_nan(top, fabsf(x[6]), fabsf(x[7]));
      top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
      if (u >= 2 * nkv) continue;
      const uint16_t s16 = scale4(top);
      const uint32_t w = codes8(x, __half2float(__ushort_as_half(s16)));
      const int b = c >> 2, part = c & 3;  // group, and eight elements of it
      const int head = (is_k ? u : u - nkv) / VPR;
      uint8_t *at = static_cast<uint8_t *>(is_k ? a.k_cache : a.v_cache) + page_at +
                    static_cast<int64_t>(head) * page_bytes;
      if (is_k) {
        *reinterpret_cast<uint32_t *>(at + kv4_key_at(D, in_page, b, part)) = w;
      } else {
        *reinterpret_cast<uint16_t *>(at + kv4_value_at(D, in_page, b, 2 * part)) =
            static_cast<uint16_t>(w);
        *reinterpret_cast<uint16_t *>(at + kv4_value_at(D, in_page, b, 2 * part + 1)) =
            static_cast<uint16_t>(w >> 16);
      }
      if (part == 0)
        *reinterpret_cast<uint16_t *>(at + scales_at + (is_k ? kv4_key_scale_at(D, in_page, b)
                                                             : kv4_value_scale_at(D, in_page, b))) =
            s16;
    }
  }
}

// n - 8 of a word's nibbles, times s0 (the first four) or s1, rounded once
template <int DTYPE>
__device__ __forceinline__ uint4 values8(uint32_t w, __half s0, __half s1) {
  const __half2 s = __halves2half2(s0, s1);
  uint32_t h[4];  // pairs (e, e + 4): 1024 + n, minus 1032, exact in fp16
  const uint32_t half_of[2] = {w, w >> 8};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t bits = half_of[e >> 1] & (e & 1 ? 0x00F000F0u : 0x000F000Fu);
    bits |= 0x64006400u;
    const __half2 n = *reinterpret_cast<const __half2 *>(&bits);
    // an odd pair stands 16 times as high: 1024 + 16 n
    const __half2 d = e & 1 ? __hfma2(n, __float2half2_rn(0.0625f), __float2half2_rn(-72.0f))
                            : __hsub2(n, __float2half2_rn(1032.0f));
    const __half2 p = DTYPE == MOE_DTYPE_FP16 ? __hmul2(d, s) : d;
    h[e] = *reinterpret_cast<const uint32_t *>(&p);
  }
  if (DTYPE == MOE_DTYPE_FP16)
    return make_uint4(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410),
                      __byte_perm(h[0], h[1], 0x7632), __byte_perm(h[2], h[3], 0x7632));
  const float2 sf = __half22float2(s);
  const uint64_t ss = pack_f32x2(sf.x, sf.y);
  float f[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 n = __half22float2(*reinterpret_cast<const __half2 *>(&h[e]));
    const float2 v = unpack_f32x2(mul_f32x2(pack_f32x2(n.x, n.y), ss));
    f[e] = v.x;
    f[e + 4] = v.y;
  }
  return pack8<DTYPE>(f);
}
__device__ __forceinline__ __half half_of(uint32_t w, int high) {
  return __ushort_as_half(static_cast<uint16_t>(high ? w >> 16 : w));
}
template <int N>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t (&w)[N]) {
  if constexpr (N == 4)
    *reinterpret_cast<uint4 *>(w) = *reinterpret_cast<const uint4 *>(p);
  else if constexpr (N == 2)
    *reinterpret_cast<uint2 *>(w) = *reinterpret_cast<const uint2 *>(p);
  else
    w[0] = *reinterpret_cast<const uint32_t *>(p);
}

// A warp reads one head's keys or values, kReadRows rows at a time: a lane has
// what a lane of the attention has of a row, so that codes and scales come in one
// load each (keys: 8 elements of every group, four lanes a row; values: 4 of every
// group, eight lanes a row, and the row's half of its pair's words).  The slots of
// the next rows are on their way while these are read.  131072 rows of 8 heads of
// 128: 117 us; 182 with a thread for every 8 elements and one load for each of their
// parts, 137 with 16 rows a warp (spills), 174 with 6 CTAs an SM.
constexpr int kReadRows = 8, kReadWarps = 8, kReadCtas = 4;  // CTAs of an SM
template <int DTYPE, int D, bool IS_K>
__device__ __forceinline__ void read_head(const Kv4ReadArgs &a, int h, int64_t block, int64_t step) {
  constexpr int NB = D / kGroup4, LANES = IS_K ? 4 : 8, SIDE = 32 / LANES, U = kReadRows / SIDE;
  const int lane = threadIdx.x & 31, side = lane % LANES, row0 = lane / LANES;
  const int mask = (1 << a.page_shift) - 1;
  const int page_bytes = kv4_row_bytes(D) << a.page_shift;
  const int scales_at = kv4_code_bytes(D) << a.page_shift;
  const int64_t page_stride = static_cast<int64_t>(a.hkv) * page_bytes;
  const int num_slots = static_cast<int>(a.num_slots), num_dst = static_cast<int>(a.dst_num_slots);
  const uint8_t *cache = (IS_K ? a.k_cache : a.v_cache) + static_cast<int64_t>(h) * page_bytes;
  uint16_t *out = static_cast<uint16_t *>(IS_K ? a.k_out : a.v_out) + 32 / LANES * side;
  const int64_t stride = IS_K ? a.k_stride : a.v_stride;
  const int64_t blocks = (static_cast<int64_t>(a.n) + kReadRows - 1) / kReadRows;
  int32_t slot[U], dst[U];
  auto fetch = [&](int64_t of) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = of * kReadRows + u * SIDE + row0;
      slot[u] = i < a.n ? a.slots[i] : -1;
      dst[u] = a.dst_slots && i < a.n ? a.dst_slots[i] : 0;
    }
  };
  if (block < blocks) fetch(block);
  for (; block < blocks; block += step) {
    constexpr int NS = IS_K ? NB / 2 : NB;
    uint32_t w[U][NB], s[U][NS], odd = 0;
    uint16_t *to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      to[u] = nullptr;
      if (slot[u] < -1 || slot[u] >= num_slots ||
          (a.dst_slots && (dst[u] < -1 || dst[u] >= num_dst))) {
        if (h == 0 && IS_K && side == 0) set_status(a.status, kStatusBadId);
        continue;
      }
      if (slot[u] < 0 || dst[u] < 0) continue;
      const uint8_t *at = cache + (slot[u] >> a.page_shift) * page_stride;
      const int r = slot[u] & mask;
      if (IS_K) {
        load_words<NB>(at + kv4_key_at(D, r, 0, side), w[u]);
        load_words<NS>(at + scales_at + kv4_key_scale_at(D, r, 0), s[u]);
      } else {
        odd |= (r & 1) << u;
        load_words<NB>(at + kv4_value_at(D, r & ~1, 0, side), w[u]);
        load_words<NS>(at + scales_at + kv4_value_scale_at(D, r & ~1, 0), s[u]);
      }
      if (a.dst_slots)
        to[u] = out + (((static_cast<int64_t>(dst[u] >> a.page_shift) * a.hkv + h) << a.page_shift) +
                       (dst[u] & mask)) * D;
      else
        to[u] = out + (block * kReadRows + u * SIDE + row0) * stride + h * D;
    }
    fetch(block + step);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!to[u]) continue;
      if (IS_K) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const __half sb = half_of(s[u][(b / 2) % NS], b & 1);
          *reinterpret_cast<uint4 *>(to[u] + 32 * b) = values8<DTYPE>(w[u][b], sb, sb);
        }
      } else {
#pragma unroll
        for (int b = 0; b < NB; b += 2) {
          const int high = odd >> u & 1;
          const uint4 v = values8<DTYPE>(__byte_perm(w[u][b], w[u][b + 1], high ? 0x7632 : 0x5410),
                                         half_of(s[u][b % NS], high), half_of(s[u][(b + 1) % NS], high));
          *reinterpret_cast<uint2 *>(to[u] + 32 * b) = make_uint2(v.x, v.y);
          *reinterpret_cast<uint2 *>(to[u] + 32 * b + 32) = make_uint2(v.z, v.w);
        }
      }
    }
  }
}

template <int DTYPE, int D>
__global__ void __launch_bounds__(kReadWarps * 32, kReadCtas) kv4_read_kernel(const Kv4ReadArgs a) {
  pdl_begin();
  const int kinds = 2 * a.hkv;
  const int warps = gridDim.x * kReadWarps, at = blockIdx.x * kReadWarps + (threadIdx.x >> 5);
  const int step = max(warps / kinds, 1);  // warps of a kind: they take its rows in turn
  for (int k = at; k < step * kinds; k += warps) {
    const int kind = k % kinds;
    if (kind < a.hkv)
      read_head<DTYPE, D, true>(a, kind, k / kinds, step);
    else
      read_head<DTYPE, D, false>(a, kind - a.hkv, k / kinds, step);
  }
}

template <int DTYPE, int D>
cudaError_t append(const KvAppendArgs &a, cudaStream_t s) {
  // Warps of a token: eight while the CTAs are one wave, then fewer, whose units in
  // flight are more.  us with 8, 4, 2 of them, 64 + 8 heads of 128 and the rows read
  // back: 304 tokens 6.0, 6.4, 8.4; 608 8.3, 8.0, 9.5; 1216 16.0, 14.7, 15.0; 2432
  // 26.2, 23.9, 24.3; 16384 141, 122, 119.  28 + 4 heads of 64: 152 tokens 4.5, 4.8,
  // 5.1; 608 5.7, 5.4, 5.4; 4096 24.0, 18.4, 15.0.
  const unsigned T = static_cast<unsigned>(a.T);
  if (a.T < 4 * num_sms())
    MOE_LAUNCH_PDL(kv4_append_kernel<DTYPE, D, 8>, T, 256, 0, s, a);
  else if (a.T < 12 * num_sms())
    MOE_LAUNCH_PDL(kv4_append_kernel<DTYPE, D, 4>, (T + 1) / 2, 256, 0, s, a);
  else
    MOE_LAUNCH_PDL(kv4_append_kernel<DTYPE, D, 2>, (T + 3) / 4, 256, 0, s, a);
  return cudaGetLastError();
}
template <int DTYPE, int D>
cudaError_t read(const Kv4ReadArgs &a, cudaStream_t s) {
  const int64_t tasks = (static_cast<int64_t>(a.n) + kReadRows - 1) / kReadRows * 2 * a.hkv;
  const int64_t ctas = (tasks + kReadWarps - 1) / kReadWarps, most = num_sms() * kReadCtas;
  MOE_LAUNCH_PDL(kv4_read_kernel<DTYPE, D>, static_cast<unsigned>(ctas < most ? ctas : most),
                 kReadWarps * 32, 0, s, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_append(const KvAppendArgs &a, int dtype, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  if (dtype == MOE_DTYPE_BF16)
    return a.D == 64 ? append<MOE_DTYPE_BF16, 64>(a, s) : append<MOE_DTYPE_BF16, 128>(a, s);
  return a.D == 64 ? append<MOE_DTYPE_FP16, 64>(a, s) : append<MOE_DTYPE_FP16, 128>(a, s);
}

cudaError_t launch_kv4_read(const Kv4ReadArgs &a, int dtype, cudaStream_t s) {
  if (a.n == 0) return cudaSuccess;
  if (dtype == MOE_DTYPE_BF16)
    return a.D == 64 ? read<MOE_DTYPE_BF16, 64>(a, s) : read<MOE_DTYPE_BF16, 128>(a, s);
  return a.D == 64 ? read<MOE_DTYPE_FP16, 64>(a, s) : read<MOE_DTYPE_FP16, 128>(a, s);
}

}  // namespace moe
