// kv4_attention.cu -- attention over the 4-bit paged cache (moe_kv4_attention).
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q.k_j),
//   k = (n - 8) s and v likewise, a scale s for every 32 elements of a row, so
//   q.k = sum over groups b of s_b (sum_{d in b} q_d n_d - 8 sum_{d in b} q_d)
//   sum_j p_j v_j[d] = sum_j (p_j s_jb) n_jd - 8 sum_j (p_j s_jb),  d in b.
// The codes go into the matrix instructions as they stand: a nibble alone in its
// half of a register is the fp16 number n 2^-24 (a subnormal), one nibble further
// up n 2^-20, so decoding is one AND per two elements.  The powers of two come
// off the scale of the scores and of the output, the offset of 8 off the
// accumulators' start (keys) and off one more product with a constant (values).
// Nothing of the cache is rounded on the way: scales and codes are exact.
//
// Keys are the rows (M = 16) of the instruction and query rows its columns (N =
// 8), so that 8 query heads of a key head, the usual number, fill it.  Every warp
// is a worker on its own (attention.cuh): it streams steps of 32 keys through a
// private ring in shared memory (cp.async).
//
// Rounded to fewer bits: queries to fp16 after taking out each row's power of two
// (its largest element is put at 2^14: bf16 ones lose nothing above 2^-28 of it);
// probabilities times the value scales to fp16 for the product with V (the tensor
// cores take 16-bit operands).  Where the output is bf16, whose own rounding is
// eight times coarser, the probabilities are rounded first and multiplied two at a
// time; for fp16 outputs the product is taken in fp32 and rounded once (error
// against 64 bits 1.6 times that of the output's rounding with two, 37 sequences of
// up to 6 tokens and 4099 rows).
#include <algorithm>

#include "attention.cuh"
#include "kv4.cuh"

#ifndef KCENT
#define KCENT true
#define INL __forceinline__
#define W1 12
#define W2 8
#define ASMV asm
#endif
namespace moe {
namespace {

struct Steps4 {
  static constexpr int kKeys = 32, kUnitCost = 2;
  static __device__ __forceinline__ int cost(int) { return 1; }
  static __device__ __forceinline__ int steps_up(int x, int) { return x; }
};

constexpr int kMostWarps4 = 16;  // of a CTA

// Probabilities are 2^(score + c0), c0 = kOff - ev - max, where the value scales
// are below 2^(ev + 1): 2^(kOff + kLag) at most, and with a scale below 2^15.5.
// Past kMost the rounding of c0 could carry them out of fp16; such rows are NaN.
struct Prob4 {
  static constexpr float kOff = 9.0f, kLag = 5.0f, kMost = 16777216.0f;
};

template <int D, int WARPS>
struct Cfg4 {
  static constexpr int NB = D / kGroup4;
  static constexpr int CB = kv4_code_bytes(D), SB = kv4_scale_bytes(D);  // of a row
  static constexpr int CODES = Steps4::kKeys * CB;  // bytes of a step's keys or values
  static constexpr int SCALES = Steps4::kKeys * SB;
  static constexpr int STAGE = 2 * (CODES + SCALES);  // key codes, values', key scales, values'
  static constexpr int STAGES = std::min(8, 216 * 1024 / (WARPS * STAGE));
  static constexpr int WARP_BYTES = STAGES * STAGE;
  static constexpr int SMEM_BYTES = WARPS * WARP_BYTES;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// N 32-bit words of shared memory
template <int N>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&v)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr));
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[0]) : "r"(addr));
}
__device__ __forceinline__ void sts_zero16(uint32_t addr) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(static_cast<uint16_t>(0)) : "memory");
}
__device__ __forceinline__ void mma4(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                     uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1,
                                     float c2, float c3) {
  ASMV(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma4(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                     uint32_t a3, uint32_t b0, uint32_t b1) {
  ASMV(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed8x8(uint32_t v) {
  uint32_t r;
  ASMV("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float2 half2_at(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u;  // n 2^-24, n 2^-20
constexpr uint32_t kEight = 0x00080008u, kEightHigh = 0x00800080u;

// One stretch, by one warp.  `slot`: first row of its partial result; `split`:
// pieces that the query heads of a key head are cut into.
template <int DTYPE, int D, int NT, int WARPS>
__device__ INL void attend(const AttnArgs &g, const Stretch &x, int split,
                                       int64_t slot, uint32_t ring) {
  using C = Cfg4<D, WARPS>;
  constexpr int NB = C::NB;
  constexpr bool ONCE = DTYPE == MOE_DTYPE_FP16;
  constexpr bool CENTRED = KCENT || NT > 1;
  const PrefixAttnArgs &a = g.a;
  const int lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3;
  const int rows = x.ntok * g.G;
  // ---- the ring.  A step is two runs of 16 rows, each in one page; lane i keeps
  // the page of run `page0 + i`.
  const int kvh = x.head / split, heads = a.hkv / split;
  const int spp = a.page_shift - 4;  // log2 of runs per page
  const int page_bytes = kv4_row_bytes(D) << a.page_shift;
  const int64_t page_stride = static_cast<int64_t>(heads) * page_bytes;
  const int runs = (x.kv_len + 15) >> 4, run_end = min(runs, 2 * x.s1);
  constexpr int RC = 16 * C::CB, RS = 16 * C::SB;  // bytes of a run's codes, scales
  const uint8_t *kl = static_cast<const uint8_t *>(a.k_cache) +
                      static_cast<int64_t>(kvh) * page_bytes + lane * 16;
  const uint8_t *vl = static_cast<const uint8_t *>(a.v_cache) +
                      static_cast<int64_t>(kvh) * page_bytes + lane * 16;
  // scales: the lanes of a run's keys, of the next run's, then those of values
  constexpr int SL = RS / 16;
  const int s_run = (lane / SL) & 1;
  const uint8_t *sl = (lane < 2 * SL ? kl : vl) + (C::CB << a.page_shift) - (lane / SL) * RS;
  int page0 = 2 * x.s0, page = 0;
  auto fetch_pages = [&](int run) {
    page0 = run;
    page = 0;
    if (run + lane < run_end) {
      page = x.pages[(run + lane) >> spp];
      if (page < 0 || page >= a.num_pages) {
        set_status(a.status, kStatusBadId);
        page = 0;
      }
    }
  };
  fetch_pages(page0);
  uint32_t into = ring;
  auto load = [&](int s) {  // past the end: an empty group
    if (s < x.s1) {
      const int run = 2 * s;
      if (run - page0 >= 32) fetch_pages(run);
      const int mask = (1 << spp) - 1;
      const int64_t at0 = __shfl_sync(0xffffffffu, page, run - page0) * page_stride;
      const int64_t at1 = __shfl_sync(0xffffffffu, page, run - page0 + 1) * page_stride;
      const int r0 = run & mask, r1 = (run + 1) & mask;
      const uint32_t dst = into + lane * 16;
      const uint32_t n1 = run + 1 < runs ? 16 : 0;  // the second run may be past the end
      const uint8_t *k0 = kl + at0 + r0 * RC, *k1 = kl + at1 + r1 * RC;
      const uint8_t *v0 = vl + at0 + r0 * RC, *v1 = vl + at1 + r1 * RC;
#pragma unroll
      for (int i = 0; i < RC / 512; ++i) {
        cp_async16(dst + i * 512, k0 + i * 512);
        cp_async16(dst + RC + i * 512, k1 + i * 512, n1);
        cp_async16(dst + C::CODES + i * 512, v0 + i * 512);
        cp_async16(dst + C::CODES + RC + i * 512, v1 + i * 512, n1);
      }
      if (lane < 4 * SL)
        cp_async16(dst + 2 * C::CODES, sl + (s_run ? at1 + r1 * RS : at0 + r0 * RS),
                   s_run ? n1 : 16);
      into = into + C::STAGE == ring + C::WARP_BYTES ? ring : into + C::STAGE;
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < C::STAGES - 1; ++i) load(x.s0 + i);

  // ---- queries: row r is head r % G of token r / G.  Column gr of block nt.
  uint32_t q[NT][NB][4];
  // -8 times the groups' sums: the second operand of one more product, with the
  // groups' scales along the contraction; slots 0 to NB - 1 hold them rounded to
  // fp16, NB to 2 NB - 1 what that left
  uint32_t start[NT];
  uint64_t sl2[NT];        // of the two columns, as everything below
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = nt * 8 + gr, i = r / g.G, hd = r - i * g.G;
    const bool live = r < rows;
    const uint16_t *src = static_cast<const uint16_t *>(a.q) + (x.tok0 + i) * a.q_stride +
                          (x.head * g.G + hd) * D + 8 * t;
    float top = 0.0f;
    uint4 raw[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      raw[b] = live ? *reinterpret_cast<const uint4 *>(src + 32 * b) : make_uint4(0, 0, 0, 0);
      float f[8];
      unpack8<DTYPE>(raw[b], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // the row is divided by 2^e: its largest element comes to [2^14, 2^15)
    int e = static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14;
    e = min(max(e, -24), 100);
    const float down = __uint_as_float((127 - e) << 23);
    float sums[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float f[8];
      unpack8<DTYPE>(raw[b], f);
      // pairs (j, j + 4), the odd j's nibbles standing 16 times as high
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float m = j & 1 ? down * 0.0625f : down;
        q[nt][b][j] = pack_f16x2(f[j] * m, f[j + 4] * m);
        const float2 held = half2_at(q[nt][b][j]);
        sum += (held.x + held.y) * (j & 1 ? 16.0f : 1.0f);
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      sums[b] = sum * (-8.0f / 512.0f);  // 2^15 up, away from fp16's subnormals
    }
    // slots 2t and 2t + 1, of the row itself: column gr
    const int b0 = (2 * t) % NB;
    float pair[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      pair[c] = sums[c];
#pragma unroll
      for (int b = 2; b < NB; ++b)
        if (b == b0 + c) pair[c] = sums[b];
    }
    const uint32_t high = pack_f16x2(pair[0], pair[1]);
    const float2 held = half2_at(high);
    const uint32_t rest = pack_f16x2(pair[0] - held.x, pair[1] - held.y);
    start[nt] = 2 * t < NB ? high : 2 * t < 2 * NB ? rest : 0u;
    // 2^(e + 24) in two factors
    const float up = a.scale * kLog2e * __uint_as_float((127 + e) << 23) * 16777216.0f;
    sl2[nt] = pack_f32x2(__shfl_sync(0xffffffffu, up, 8 * t),
                         __shfl_sync(0xffffffffu, up, 8 * t + 4));
  }

  float o[NT][NB][2][4], z[NT][CENTRED ? 1 : NB][4];
  uint64_t c0[NT], l[NT];
  float ev = 0.0f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[nt][b][0][e] = o[nt][b][1][e] = 0.0f;
        if (b == 0 || !CENTRED) z[nt][CENTRED ? 0 : b][e] = 0.0f;
      }
    c0[nt] = l[nt] = 0;
  }
  const int all_seen = min(x.kv_len, x.lim0);  // keys that every token sees
  uint32_t from = ring;
#pragma unroll 1
  for (int s = x.s0; s < x.s1; ++s) {
    cp_async_wait<C::STAGES - 2>();
    __syncwarp();  // and the stage of the step before is free
    load(s + C::STAGES - 1);
    const int key0 = s * Steps4::kKeys;
    const uint32_t sk = from;
    from = from + C::STAGE == ring + C::WARP_BYTES ? ring : from + C::STAGE;
    const uint32_t sv = sk + C::CODES, ss = sv + C::CODES;
    if (key0 + Steps4::kKeys > x.kv_len) {  // scales past the length: whatever lies there, zero
      const int r = x.kv_len - key0;
      if (lane >= r)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          sts_zero16(ss + kv4_key_scale_at(D, lane, b));
          sts_zero16(ss + C::SCALES + kv4_value_scale_at(D, lane, b));
        }
      __syncwarp();
    }
    // ---- scores: keys gr and gr + 8 of either half, columns 2t and 2t + 1
    float sc[2][NT][4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t k0[NB], k1[NB], w0[NB / 2], w1[NB / 2];
      const uint32_t at = sk + (half * 16 + gr) * C::CB + t * (D / 8);
      lds<NB>(at, k0);
      lds<NB>(at + 8 * C::CB, k1);
      const uint32_t as = ss + (half * 16 + gr) * C::SB;
      lds<NB / 2>(as, w0);
      lds<NB / 2>(as + 8 * C::SB, w1);
      const uint32_t a0 = NB == 4 && (t & 1) ? w0[NB / 2 - 1] : w0[0];
      const uint32_t a1 = NB == 4 && (t & 1) ? w1[NB / 2 - 1] : w1[0];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma4(sc[half][nt], a0, a1, 0, 0, start[nt], 0, 0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[half][nt][e] *= 1.0f / 32768.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float2 p0 = half2_at(w0[b / 2]), p1 = half2_at(w1[b / 2]);
        const float s0 = b & 1 ? p0.y : p0.x, s1 = b & 1 ? p1.y : p1.x;
        const uint32_t x0 = k0[b], x1 = k1[b], y0 = x0 >> 8, y1 = x1 >> 8;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float d[4];
          mma4(d, x0 & kLow, x1 & kLow, x0 & kHigh, x1 & kHigh, q[nt][b][0], q[nt][b][1], 0.0f,
               0.0f, 0.0f, 0.0f);
          mma4(d, y0 & kLow, y1 & kLow, y0 & kHigh, y1 & kHigh, q[nt][b][2], q[nt][b][3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[half][nt][e] = fmaf(d[e], e < 2 ? s0 : s1, sc[half][nt][e]);
        }
      }
    }
    if (key0 + Steps4::kKeys > all_seen) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // columns past the rows see everything there is
          const int r = nt * 8 + 2 * t + c;
          const int lim = (r < rows ? min(x.kv_len, x.lim0 + r / g.G) : x.kv_len) - key0 - gr;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (half * 16 >= lim) sc[half][nt][c] = -INFINITY;
            if (half * 16 + 8 >= lim) sc[half][nt][2 + c] = -INFINITY;
          }
        }
    }
    // ---- exponents.  The running maximum moves when a score passes it by the lag,
    // and the exponent of the value scales when one passes it (the test is of the
    // top bit of fp16 exponents: 2 or more).
    uint64_t ex[2][NT][2];
    float most = -INFINITY;
    auto exponents = [&]() {
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            ex[half][nt][r] = fma_f32x2(
                pack_f32x2(sc[half][nt][2 * r], sc[half][nt][2 * r + 1]), sl2[nt], c0[nt]);
            const float2 f = unpack_f32x2(ex[half][nt][r]);
            most = fmaxf(most, fmaxf(f.x, f.y));
          }
    };
    exponents();
    uint32_t any[NB];  // half of the lanes would do
    lds<NB>(ss + C::SCALES + (lane & 15) * (2 * C::SB), any);
    uint32_t two = any[0];
#pragma unroll
    for (int b = 1; b < NB; ++b) two |= any[b];
    if (__any_sync(0xffffffffu, most > Prob4::kOff + Prob4::kLag - ev || (two & 0x40004000u) ||
                                    s == x.s0)) {
      float big = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float2 p = half2_at(any[b]);
        big = fmaxf(big, fmaxf(p.x, p.y));
      }
      const unsigned top_s = __reduce_max_sync(0xffffffffu, __float_as_uint(big));
      const float ev1 = fmaxf(ev, static_cast<float>(static_cast<int>(top_s >> 23) - 127));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 m = unpack_f32x2(sl2[nt]), was = unpack_f32x2(c0[nt]);
        float is[2], f[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float top = fmaxf(fmaxf(sc[0][nt][c], sc[0][nt][2 + c]),
                            fmaxf(sc[1][nt][c], sc[1][nt][2 + c]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          const float u = c ? m.y : m.x, old = c ? was.y : was.x;
          // each column by its own scores, so that no head's bits depend on another's
          is[c] = old + (ev - ev1);
          if (s == x.s0 || fmaf(top, u, old) > Prob4::kOff + Prob4::kLag - ev)
            is[c] = fmaf(-fmaxf(top, -Prob4::kMost / u), u, Prob4::kOff - ev1);
          f[c] = ex2(is[c] - old);
          if (s == x.s0) f[c] = 0.0f;
        }
        c0[nt] = pack_f32x2(is[0], is[1]);
        l[nt] = mul_f32x2(l[nt], pack_f32x2(f[0], f[1]));
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[nt][b][0][e] *= f[e & 1];
            o[nt][b][1][e] *= f[e & 1];
            if (!CENTRED) z[nt][CENTRED ? 0 : b][e] *= f[e & 1];
          }
      }
      ev = ev1;
      exponents();
    }
    // ---- probabilities, as the second operand: keys along the contraction
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t p[NT][2];
      float pe[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float2 f = unpack_f32x2(ex[half][nt][r]);
          pe[nt][2 * r] = ex2(f.x);
          pe[nt][2 * r + 1] = ex2(f.y);
          l[nt] = add_f32x2(l[nt], pack_f32x2(pe[nt][2 * r], pe[nt][2 * r + 1]));
          if (!ONCE) p[nt][r] = transposed8x8(pack_f16x2(pe[nt][2 * r], pe[nt][2 * r + 1]));
        }
      // value scales of pairs: of keys 2t, 2t + 1 and 2t + 8, 2t + 9; where
      // probabilities take them before they are rounded, those that hold keys gr and
      // gr + 8
      uint32_t sp[2][NB];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        lds<NB>(ss + C::SCALES + (half * 8 + 4 * k + (ONCE ? gr >> 1 : t)) * (2 * C::SB), sp[k]);
      // ---- product with V: elements 4 gr + 2 hh and + 1 of group b, as rows gr and
      // gr + 8; keys 2t, 2t + 1, 2t + 8, 2t + 9 (kv4_value_at)
      uint32_t v[2][NB];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        lds<NB>(sv + (half * 8 + 4 * j + t) * (2 * C::CB) + kv4_value_turn(D, t, gr * (D / 8)), v[j]);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t x0 = v[0][b], y0 = x0 >> 8, x1 = v[1][b], y1 = x1 >> 8;
        uint32_t f[2][4] = {{x0 & kLow, x0 & kHigh, x1 & kLow, x1 & kHigh},
                            {y0 & kLow, y0 & kHigh, y1 & kLow, y1 & kHigh}};
        if (CENTRED)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            f[i / 4][i & 3] = hsub2(f[i / 4][i & 3], i & 1 ? kEightHigh : kEight);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t p0, p1;
          if constexpr (ONCE) {
            const float2 w0 = half2_at(sp[0][b]), w1 = half2_at(sp[1][b]);
            const float s0 = gr & 1 ? w0.y : w0.x, s1 = gr & 1 ? w1.y : w1.x;
            p0 = transposed8x8(pack_f16x2(pe[nt][0] * s0, pe[nt][1] * s0));
            p1 = transposed8x8(pack_f16x2(pe[nt][2] * s1, pe[nt][3] * s1));
          } else {
            p0 = hmul2(p[nt][0], sp[0][b]);
            p1 = hmul2(p[nt][1], sp[1][b]);
          }
#pragma unroll
          for (int hh = 0; hh < 2; ++hh)
            mma4(o[nt][b][hh], f[hh][0], f[hh][1], f[hh][2], f[hh][3], p0, p1);
          if (!CENTRED) mma4(z[nt][CENTRED ? 0 : b], kEight, kEight, kEight, kEight, p0, p1);
        }
      }
    }
  }
  cp_async_wait<0>();
  __syncwarp();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float2 sums = unpack_f32x2(l[nt]), offs = unpack_f32x2(c0[nt]);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float sum = c ? sums.y : sums.x;
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      const int r = nt * 8 + 2 * t + c;
      if (r >= rows) continue;
      const float off = c ? offs.y : offs.x;
      if (off < -Prob4::kMost) sum = NAN;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const float low = inv * 16777216.0f, high = inv * 1048576.0f;
      float *dst = g.part_o + (slot + r) * D + 4 * gr;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float eight = z[nt][CENTRED ? 0 : b][c] * low;
        *reinterpret_cast<float4 *>(dst + 32 * b) = make_float4(
            fmaf(o[nt][b][0][c], low, -eight), fmaf(o[nt][b][0][2 + c], high, -eight),
            fmaf(o[nt][b][1][c], low, -eight), fmaf(o[nt][b][1][2 + c], high, -eight));
      }
      if (gr == 0) g.part_lse[slot + r] = sum == 0.0f ? -INFINITY : log2f(sum) - off;
    }
  }
}

template <int DTYPE, int D, int NT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 1)
    kv4_attention_kernel(const AttnArgs g, const int split) {
  using C = Cfg4<D, WARPS>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ ScanShared<WARPS * 32> scan;
  const int warp = threadIdx.x >> 5;
  pdl_begin();
  const OwnScan own = scan_own<Steps4>(g, scan);
  const int64_t workers = gridDim.x * WARPS;
  const int64_t piece = max(quotient(own.total + workers - 1, workers), static_cast<int64_t>(1));
  if (blockIdx.x == 0) write_meta<Steps4>(g, own);
  // consecutive pieces on different SMs
  const int worker = warp * gridDim.x + blockIdx.x;
  const int64_t lo = worker * piece, hi = min(lo + piece, own.total);
  if (lo >= own.total) return;
  OwnWalk<Steps4> walk;
  walk.begin(g, scan, lo, hi);
  Stretch x;
  while (walk.next(g, &x)) {
    if ((threadIdx.x & 31) == 0) mark_span(g, x.unit, x, worker);
    attend<DTYPE, D, NT, WARPS>(g, x, split, (x.unit + worker) * g.own.rows,
                                smem_u32(smem) + warp * C::WARP_BYTES);
  }
}

// The plan: query rows of a unit, and the scratch.
struct Plan4 {
  int split, blocks8, warps;  // blocks of 8 rows in a unit
  int64_t units;
  size_t span, lse, o, bytes;
};
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

Plan4 plan(AttnArgs &g, int T, int B, int max_q, int hq, int hkv, int D) {
  const int most_rows = D == 128 ? 16 : 32;
  const int G = hq / hkv, nq = std::max(1, std::min(max_q, T));
  Plan4 p = {};
  // more query heads than a unit has rows: equal parts of them
  int Gs = std::min(G, most_rows);
  while (G % Gs != 0) --Gs;
  p.split = G / Gs;
  const int64_t rows = static_cast<int64_t>(nq) * Gs;
  p.blocks8 = rows <= 8 ? 1 : rows <= 16 || D == 128 ? 2 : 4;
  p.warps = p.blocks8 == 1 ? 16 : 8;
  g.G = Gs;
  g.own.tok = static_cast<int>(std::min<int64_t>(std::max(1, 8 * p.blocks8 / Gs), nq));
  g.own.rows = g.own.tok * Gs;
  g.own_rows_kernel = B > 0;
  g.r_on = g.own_rows_kernel;
  g.r_most = kMaxCtas * kMostWarps4;
  // blocks of all sequences: the tokens may lie in any of them, max_q in each
  const int64_t blocks = std::min<int64_t>(
      B + T / g.own.tok, static_cast<int64_t>(B) * ((nq + g.own.tok - 1) / g.own.tok));
  p.units = blocks * (hq / Gs);
  const size_t parts = (static_cast<size_t>(p.units) + kMaxCtas * kMostWarps4) * g.own.rows;
  p.span = up256(sizeof(SeqMeta) * static_cast<size_t>(B));
  p.lse = up256(p.span + sizeof(int2) * static_cast<size_t>(p.units));
  p.o = up256(p.lse + 4 * parts);
  p.bytes = up256(p.o + 4 * parts * D);
  return p;
}

template <int DTYPE, int D, int NT, int WARPS>
cudaError_t run(const AttnArgs &g, int split, int ctas, cudaStream_t s) {
  using C = Cfg4<D, WARPS>;
  auto kernel = kv4_attention_kernel<DTYPE, D, NT, WARPS>;
  const cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (err != cudaSuccess) return err;
  MOE_LAUNCH_PDL(kernel, ctas, WARPS * 32, C::SMEM_BYTES, s, g, split);
  return cudaGetLastError();
}
template <int DTYPE, int D>
cudaError_t run_d(const AttnArgs &g, const Plan4 &p, int ctas, cudaStream_t s) {
  if (p.blocks8 == 1) return run<DTYPE, D, 1, W1>(g, p.split, ctas, s);
  if constexpr (D == 64)
    if (p.blocks8 == 4) return run<DTYPE, D, 4, 8>(g, p.split, ctas, s);
  return run<DTYPE, D, 2, W2>(g, p.split, ctas, s);
}

}  // namespace

size_t kv4_attention_scratch_bytes(int T, int B, int max_q, int hq, int hkv, int D, bool smaller) {
  AttnArgs g = {};
  size_t bytes = plan(g, T, B, max_q, hq, hkv, D).bytes;
  // What no smaller call passes: up to a unit's most rows a smaller max_q can have
  // more units, past them none.
  for (int q = std::min(max_q - 1, 32); smaller && q > 0; --q)
    bytes = std::max(bytes, plan(g, T, B, q, hq, hkv, D).bytes);
  return bytes;
}

cudaError_t launch_kv4_attention(const PrefixAttnArgs &a, int dtype, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  AttnArgs g = {};
  g.a = a;
  const int ctas = std::min(num_sms(), kMaxCtas);
  const Plan4 p = plan(g, a.T, a.B, a.max_q, a.hq, a.hkv, a.D);
  g.a.hkv = a.hkv * p.split;  // units are counted by parts of a key head's queries
  g.meta = reinterpret_cast<SeqMeta *>(a.scratch);
  g.span = reinterpret_cast<int2 *>(a.scratch + p.span);
  g.part_lse = reinterpret_cast<float *>(a.scratch + p.lse);
  g.part_o = reinterpret_cast<float *>(a.scratch + p.o);
  if (g.r_on) {
    cudaError_t err;
    if (dtype == MOE_DTYPE_BF16)
      err = a.D == 64 ? run_d<MOE_DTYPE_BF16, 64>(g, p, ctas, s)
                      : run_d<MOE_DTYPE_BF16, 128>(g, p, ctas, s);
    else
      err = a.D == 64 ? run_d<MOE_DTYPE_FP16, 64>(g, p, ctas, s)
                      : run_d<MOE_DTYPE_FP16, 128>(g, p, ctas, s);
    if (err != cudaSuccess) return err;
  }
  return launch_attention_join(g, dtype, ctas, s);
}

}  // namespace moe
