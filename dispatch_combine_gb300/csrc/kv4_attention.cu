// kv4_attention.cu -- attention over the 4-bit paged cache (moe_kv4_attention).
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q.k_j),
//   k = (n - 8) s and v likewise, a scale s for every 32 elements of a row, so
//   q.k = sum over groups b of s_b (sum_{d in b} q_d n_d - 8 sum_{d in b} q_d)
//   sum_j p_j v_j[d] = sum_j (p_j s_jb) n_jd - 8 sum_j (p_j s_jb),  d in b.
// The codes go into the matrix instructions as they stand: a nibble alone in its
// half of a register is the fp16 number n 2^-24 (a subnormal), one nibble further
// up n 2^-20, so decoding is one AND per two elements, and the powers of two come
// off the scale of the scores and of the output.  The offset of 8 comes off the
// scores in one product of the key's scales with -8 sum q, and off the values' numbers
// before theirs (exact).  Nothing of the cache is rounded on the way but value scales far
// below the largest of their group (kLeastScale4).
//
// Keys are the rows (M = 16) of the instruction and query rows its columns (N =
// 8), so that 8 query heads of a key head, the usual number, fill it.  Units are a
// sequence's block of tokens x a key head, with up to 16 rows, and stand in a line
// that is cut into a piece for each warp (attention.cuh): every warp is a worker on
// its own and streams steps of keys through a private ring in shared memory
// (cp.async).  A unit that one warp has whole leaves as it should be; of others every
// warp keeps its part (normalised, with its log-sum-exp), which a second kernel joins.
//
// Bound by HBM where contexts are long: 16 sequences of up to 131072 rows (8 key heads
// of 128, 8 query heads each; 1.30 GB) take 200 us, 0.96 of the measured copy
// bandwidth; without the arithmetic 198.  64 of up to 8192 (364 MB) take 71: 2.5 until the
// first rows are asked for, 57 while they stream (0.93), 4 in which workers end one after
// the other, 7 for the join.  Several queries of a sequence are bound by the
// arithmetic (520 instructions for 32 keys x 8 rows of 128): 37 sequences of up to
// 4099, 6 tokens of 7 heads of 64 each (20 MB) 23.7 us.  A unit has 16 rows: 64 sequences
// of up to 8192 rows, 64 + 8 heads of 128, take 81 us with 2 tokens each and 195 with 8, and
// 103 with one token of 128 heads.
//   Other ways, each measured against this one as it then was (64 sequences, or 16
// where it says so): the offset of the values by one more product instead of a
// subtraction 81 -> 85 us; 16 warps (128 registers, spills) 73 -> 83, 10 or 11 warps
// 75 to 79; the scores of the next step ahead of this one's softmax 212 -> 225 (16
// sequences); bulk copies issued by single lanes 217 -> 237 (16); neighbouring pieces
// on one SM, joined in shared memory 72 -> 84.
//
// Rounded to fewer bits: queries to fp16 after taking out each row's power of two
// (its largest element is put at 2^14 to 2^15, elements at odd places 2^4 lower than
// others: those above 2^-24 of the largest, with bf16 2^-27, keep all their bits);
// probabilities times the value scales to fp16 for the product with V (the tensor
// cores take 16-bit operands).  Where the output is bf16, whose own rounding is
// eight times coarser, the probabilities are rounded first and multiplied two at a
// time; for fp16 outputs the product is taken in fp32 and rounded once (error
// against 64 bits 1.6 times that of the output's rounding with two, 37 sequences of
// up to 6 tokens and 4099 rows).
#include <algorithm>
#include <atomic>
#include <cfloat>

#include "attention.cuh"
#include "kv4.cuh"

namespace moe {
namespace {

// A step is NH runs of 16 keys.  What is done once a step (the copies' addresses,
// the test for the maximum) is a third of the instructions at 32 keys, and longer
// straight code fills the waits of the two or three warps that a scheduler has: 16
// sequences of up to 131072 rows took 215 us with 32 keys, 202 with 64; 37 sequences,
// 6 tokens of 7 heads of 64: 28.7 with 32 keys and 12 warps, 28.4 with 64 and 12, 25.2
// with 64 and 8 (fewer parts to join).  Two blocks of query rows of 128 leave no
// registers for 64.  A unit costs its start besides: 64 sequences of up to 8192 rows, 16
// query heads to each of 8 key heads: 112 us counting 2 steps of 32 for it, 105 counting 4
// (102.8 as it is now).
template <int NH>
struct Steps4 {
  static constexpr int kKeys = 16 * NH, kUnitCost = NH == 4 ? 2 : 4;
  static __device__ __forceinline__ int cost(int) { return 1; }
  static __device__ __forceinline__ int steps_up(int x, int) { return x; }
};

constexpr int kMostWarps4 = 12;  // of a CTA

// Probabilities are 2^(score + c0), c0 = kOff - max: 2^(kOff + kLag) at most, and twice
// that with a value scale, which is taken times a power of two that puts it below 2.
// Past kMost the rounding of c0 could carry them out of fp16; such rows are NaN.
struct Prob4 {
  static constexpr float kOff = 9.0f, kLag = 5.0f, kMost = 16777216.0f;
};
// Each group's value scales are taken times a power of two of their own, which puts the
// largest that a warp meets at a unit's first step below 1 and moves when a larger one
// would be 2 or more.  So what fp16 loses of a product of probability and scale is
// measured by the group's own values: 2^-33 of the largest probability times that scale, and
// 2^-24 of that scale.  Scales below kLeastScale4 count as that.  (From 1 to 2 at the first
// step most units would meet a larger one later: 64 sequences of up to 8192 rows, 128 + 8
// heads of 128, 102.4 us so, 105.5 with it.)
//   One power of two for all values, and never below 1, lost small values beside a key that
// took the weight: 100.7 us there, with 64 + 8 heads of 128 in fp16 72.5 (75.6 now), others
// within 1 %.
constexpr float kLeastScale4 = 1.0f / 65536.0f;

template <int D, int NH, int WARPS>
struct Cfg4 {
  static constexpr int KEYS = 16 * NH;
  static constexpr int NB = D / kGroup4;
  static constexpr int CB = kv4_code_bytes(D), SB = kv4_scale_bytes(D);  // of a row
  static constexpr int CODES = KEYS * CB;  // bytes of a step's keys or values
  static constexpr int SCALES = KEYS * SB;
  static constexpr int STAGE = 2 * (CODES + SCALES);  // key codes, values', key scales, values'
  // One step on its way while one is read: the SM's other warps fill the rest.  37 sequences
  // of up to 4099, 6 tokens of 7 heads of 64: 23.7 us, three 24.3, four 24.5; 64 of up to
  // 8192, 2 tokens of 8 heads of 128: 80.1, 81.7, 82.7.
  static constexpr int STAGES = 2;
  static constexpr int WARP_BYTES = STAGES * STAGE;
  static constexpr int SMEM_BYTES = WARPS * WARP_BYTES;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
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
template <int N>
__device__ __forceinline__ void sts(uint32_t addr, const uint32_t (&v)[N]) {
  if constexpr (N == 4)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3])
                 : "memory");
  else
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(v[0]), "r"(v[1]) : "memory");
}
__device__ __forceinline__ void sts_zero16(uint32_t addr) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(static_cast<uint16_t>(0)) : "memory");
}
__device__ __forceinline__ void mma4(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                     uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1,
                                     float c2, float c3) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma4(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                     uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
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

// Where a token's head goes.
struct Row4 {
  uint16_t *o;
  float *lse;
};
template <int D>
__device__ __forceinline__ Row4 row_at(const PrefixAttnArgs &a, int64_t t, int h) {
  return {static_cast<uint16_t *>(a.o) + t * a.o_stride + static_cast<int64_t>(h) * D,
          a.lse ? a.lse + t * a.hq + h : nullptr};
}

// A unit's normalised rows and their log2-sum-exps from shared memory, by a warp (out
// of line: the registers of the loop over keys are not these stores'): to a partial
// result, or to where they belong.
template <int D>
__device__ __noinline__ void keep_part(const float *o, const float *lse, float *part, int rows,
                                       int lse_at) {
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int i = lane; i < rows * (D / 4); i += 32)
    *reinterpret_cast<float4 *>(part + 4 * i) = *reinterpret_cast<const float4 *>(o + 4 * i);
  if (lane < rows) part[lse_at + lane] = lse[lane];
}
template <int DTYPE, int D>
__device__ __noinline__ void write_rows(const AttnArgs &g, const float *o, const float *lse, int tok0,
                                        int head0, int rows, int lim0, int kv_len) {
  constexpr int LANES = D / 8;  // of a row
  const int lane = threadIdx.x & 31, d = lane % LANES * 8;
#pragma unroll 2
  for (int r = lane / LANES; r < rows; r += 32 / LANES) {
    const int i = r * g.tpt >> 16;
    const Row4 row = row_at<D>(g.a, tok0 + i, head0 + r - i * g.G);
    float v[8], at = lse[r];
    *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(o + r * D + d);
    *reinterpret_cast<float4 *>(v + 4) = *reinterpret_cast<const float4 *>(o + r * D + d + 4);
    // nothing in the sum: zeros, unless keys are seen, all below the range
    if (at == -INFINITY && min(kv_len, lim0 + i) > 0) {
      at = NAN;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = NAN;
    }
    *reinterpret_cast<uint4 *>(row.o + d) = pack8<DTYPE>(v);
    if (row.lse && d == 0) *row.lse = at * 0.6931471805599453f;
  }
}

// One stretch, by one warp: a whole unit to its rows, else to `part` as a partial
// result (rows of D, then their log-sum-exps).  `split`: parts that the query heads of
// a key head are cut into.
template <int DTYPE, int D, int NT, int NH, int WARPS>
__device__ __forceinline__ void attend(const AttnArgs &g, const Stretch &x, int split,
                                       float *part, uint8_t *space) {
  const uint32_t ring = smem_u32(space);
  using C = Cfg4<D, NH, WARPS>;
  constexpr int NB = C::NB;
  constexpr bool ONCE = DTYPE == MOE_DTYPE_FP16;
  const PrefixAttnArgs &a = g.a;
  const int lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3;
  const int rows = x.ntok * g.G;
  // row r is head r % G of token r / G (exact for the few rows there are)
  auto token_of = [&](int r) { return r * g.tpt >> 16; };
  // ---- the ring.  A step is NH runs of 16 rows, each in one page; lane i keeps
  // the page of run `page0 + i`.
  const int kvh = x.head / split, heads = a.hkv / split;
  const int spp = a.page_shift - 4;  // log2 of runs per page
  const int page_bytes = kv4_row_bytes(D) << a.page_shift;
  const int64_t page_stride = static_cast<int64_t>(heads) * page_bytes;
  const int runs = (x.kv_len + 15) >> 4, run_end = min(runs, NH * x.s1);
  constexpr int RC = 16 * C::CB, RS = 16 * C::SB;  // bytes of a run's codes, scales
  const int64_t head_at = static_cast<int64_t>(kvh) * page_bytes;
  const uint8_t *kc = static_cast<const uint8_t *>(a.k_cache) + head_at;
  const uint8_t *vc = static_cast<const uint8_t *>(a.v_cache) + head_at;
  constexpr int SL = RS / 16;  // lanes that copy a run's scales
  int page0 = NH * x.s0, page = 0;
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
      const int run = NH * s, mask = (1 << spp) - 1;
      if (run + NH - page0 > 32) fetch_pages(run);
      const uint32_t dst = into + lane * 16;
#pragma unroll
      for (int j = 0; j < NH; ++j) {
        const int64_t at = __shfl_sync(0xffffffffu, page, run - page0 + j) * page_stride +
                           ((run + j) & mask) * RC + lane * 16;
        const uint32_t n = j == 0 || run + j < runs ? 16 : 0;  // a run may be past the end
#pragma unroll
        for (int i = 0; i < RC / 512; ++i) {
          cp_async16(dst + j * RC + i * 512, kc + at + i * 512, n);
          cp_async16(dst + C::CODES + j * RC + i * 512, vc + at + i * 512, n);
        }
      }
      // scales: the lanes of each run's keys, then those of their values
#pragma unroll
      for (int c0 = 0; c0 < 2 * NH * SL; c0 += 32) {
        const int c = c0 + lane, j = c / SL % NH;
        const int64_t p = __shfl_sync(0xffffffffu, page, run - page0 + j);
        if (c < 2 * NH * SL)
          cp_async16(dst + 2 * C::CODES + c0 * 16,
                     (c < NH * SL ? kc : vc) + (C::CB << a.page_shift) + p * page_stride +
                         ((run + j) & mask) * RS + c % SL * 16,
                     run + j < runs ? 16 : 0);
      }
      into = into + C::STAGE == ring + C::WARP_BYTES ? ring : into + C::STAGE;
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < C::STAGES - 1; ++i) load(x.s0 + i);

  // ---- queries: row nt * 8 + gr, column gr of block nt
  uint32_t q[NT][NB][4];
  // -8 times the groups' sums: the second operand of one more product, with the
  // groups' scales along the contraction; slots 0 to NB - 1 hold them rounded to
  // fp16, NB to 2 NB - 1 what that left
  uint32_t start[NT];
  uint64_t sl2[NT];        // of the two columns, as everything below
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = nt * 8 + gr, i = token_of(r), hd = r - i * g.G;
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

  float o[NT][NB][2][4];
  uint64_t c0[NT], l[NT];
  uint32_t lift[NB];  // the power of two of each group's value scales, twice
#pragma unroll
  for (int b = 0; b < NB; ++b) lift[b] = 0x78007800u;  // 2^15, the most
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][b][0][e] = o[nt][b][1][e] = 0.0f;
    c0[nt] = l[nt] = 0;
  }
  const int all_seen = min(x.kv_len, x.lim0);  // keys that every token sees
  uint32_t from = ring;
#pragma unroll 1
  for (int s = x.s0; s < x.s1; ++s) {
    cp_async_wait<C::STAGES - 2>();
    __syncwarp();  // and the stage of the step before is free
    load(s + C::STAGES - 1);
    const int key0 = s * C::KEYS;
    const uint32_t sk = from;
    from = from + C::STAGE == ring + C::WARP_BYTES ? ring : from + C::STAGE;
    const uint32_t sv = sk + C::CODES, ss = sv + C::CODES;
    if (key0 + C::KEYS > x.kv_len) {  // scales past the length: whatever lies there, zero
      for (int r = x.kv_len - key0 + lane; r < C::KEYS; r += 32)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          sts_zero16(ss + kv4_key_scale_at(D, r, b));
          sts_zero16(ss + C::SCALES + kv4_value_scale_at(D, r, b));
        }
      __syncwarp();
    }
    // ---- scores: keys gr and gr + 8 of either half, columns 2t and 2t + 1
    float sc[NH][NT][4];
#pragma unroll
    for (int half = 0; half < NH; ++half) {
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
          const uint32_t *qb = q[nt][b];
          mma4(d, x0 & kLow, x1 & kLow, x0 & kHigh, x1 & kHigh, qb[0], qb[1], 0.0f, 0.0f, 0.0f, 0.0f);
          mma4(d, y0 & kLow, y1 & kLow, y0 & kHigh, y1 & kHigh, qb[2], qb[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[half][nt][e] = fmaf(d[e], e < 2 ? s0 : s1, sc[half][nt][e]);
        }
      }
    }
    if (key0 + C::KEYS > all_seen) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // columns past the rows see everything there is
          const int r = nt * 8 + 2 * t + c;
          const int lim = (r < rows ? min(x.kv_len, x.lim0 + token_of(r)) : x.kv_len) - key0 - gr;
#pragma unroll
          for (int half = 0; half < NH; ++half) {
            if (half * 16 >= lim) sc[half][nt][c] = -INFINITY;
            if (half * 16 + 8 >= lim) sc[half][nt][2 + c] = -INFINITY;
          }
        }
      // Values that stand for NaN are nothing to rows that do not see them (0 NaN would
      // be): their scales go, and the scores of those that do see them are the NaN.
      uint32_t w[NB];
      const uint32_t at = ss + C::SCALES + lane % (8 * NH) * (2 * C::SB);
      lds<NB>(at, w);
      bool even = false, odd = false;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        even |= (w[b] & 0x7C00u) == 0x7C00u;
        odd |= (w[b] & 0x7C000000u) == 0x7C000000u;
      }
      const unsigned evens = __ballot_sync(0xffffffffu, even), odds = __ballot_sync(0xffffffffu, odd);
      if (evens | odds) {
        const uint32_t keep = (even ? 0u : 0xFFFFu) | (odd ? 0u : 0xFFFF0000u);
#pragma unroll
        for (int b = 0; b < NB; ++b) w[b] &= keep;
        if (lane < 8 * NH) sts<NB>(at, w);
        __syncwarp();
        const unsigned mine = (gr & 1 ? odds : evens) >> (gr >> 1);
#pragma unroll
        for (int half = 0; half < NH; ++half)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((mine >> (8 * half + 4 * (e >> 1)) & 1) && sc[half][nt][e] != -INFINITY)
                sc[half][nt][e] = NAN;
      }
    }
    // ---- exponents.  The running maximum moves when a score passes it by the lag,
    // and a group's power of two when a scale times it is 2 or more (the top bit of an
    // fp16 exponent; NaN, too).
    uint64_t ex[NH][NT][2];
    float most = -INFINITY;
    auto exponents = [&]() {
#pragma unroll
      for (int half = 0; half < NH; ++half)
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
    uint32_t any[NB], lifted[NB], two = 0;
    const uint32_t any_at = ss + C::SCALES + lane % (8 * NH) * (2 * C::SB);
    lds<NB>(any_at, any);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      lifted[b] = hmul2(any[b], lift[b]);
      two |= lifted[b];
    }
    if (__any_sync(0xffffffffu, most > Prob4::kOff + Prob4::kLag || (two & 0x40004000u) || s == x.s0)) {
      float to[NB];  // of the accumulators, by groups
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float2 p = half2_at(any[b]);
        const float big = fmaxf(fmaxf(p.x, p.y), kLeastScale4);  // NaN is none
        const uint32_t top_s = __reduce_max_sync(0xffffffffu, __float_as_uint(big)) & 0x7F800000u;
        const float was = half2_at(lift[b]).x;
        const float is = fminf(was, __uint_as_float((253u << 23) - top_s));  // 1 / (2 top_s)
        to[b] = is * __uint_as_float((254u << 23) - __float_as_uint(was));
        lift[b] = pack_f16x2(is, is);
        lifted[b] = hmul2(any[b], lift[b]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 m = unpack_f32x2(sl2[nt]), was = unpack_f32x2(c0[nt]);
        float is[2], f[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float top = -INFINITY;
#pragma unroll
          for (int half = 0; half < NH; ++half)
            top = fmaxf(top, fmaxf(sc[half][nt][c], sc[half][nt][2 + c]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          const float u = c ? m.y : m.x, old = c ? was.y : was.x;
          // each column by its own scores, so that no head's bits depend on another's
          is[c] = old;
          if (s == x.s0 || fmaf(top, u, old) > Prob4::kOff + Prob4::kLag)
            is[c] = fmaf(-fmaxf(top, fmaxf(-Prob4::kMost / u, -FLT_MAX)), u, Prob4::kOff);
          f[c] = ex2(is[c] - old);
          if (s == x.s0) f[c] = 0.0f;
        }
        c0[nt] = pack_f32x2(is[0], is[1]);
        l[nt] = mul_f32x2(l[nt], pack_f32x2(f[0], f[1]));
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[nt][b][0][e] *= f[e & 1] * to[b];
            o[nt][b][1][e] *= f[e & 1] * to[b];
          }
      }
      exponents();
    }
    // the scales as they are used (every lane has read its own: the vote needed them)
    if (lane < 8 * NH) sts<NB>(any_at, lifted);
    __syncwarp();
    // ---- probabilities, as the second operand: keys along the contraction
#pragma unroll
    for (int half = 0; half < NH; ++half) {
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
        }
      }
    }
  }
  cp_async_wait<0>();
  __syncwarp();
  // ---- the rows leave through the ring, where they come to lie in order (and the
  // accumulators' registers are free for the stores)
  float *held = reinterpret_cast<float *>(space);
  static_assert(8 * NT * (D + 1) * sizeof(float) <= C::WARP_BYTES, "rows and their sums in the ring");
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
      const float lse = sum == 0.0f ? -INFINITY : log2f(sum) - off;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      float *row = held + r * D + 4 * gr;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const float down = __uint_as_float((254u << 23) - __float_as_uint(half2_at(lift[b]).x));
        const float low = inv * 16777216.0f * down, high = inv * 1048576.0f * down;
        *reinterpret_cast<float4 *>(row + 32 * b) =
            make_float4(o[nt][b][0][c] * low, o[nt][b][0][2 + c] * high, o[nt][b][1][c] * low,
                        o[nt][b][1][2 + c] * high);
      }
      if (gr == 0) held[8 * NT * D + r] = lse;
    }
  }
  __syncwarp();
  if (part)
    keep_part<D>(held, held + 8 * NT * D, part, rows, g.own.rows * D);
  else
    write_rows<DTYPE, D>(g, held, held + 8 * NT * D, x.tok0, x.head * g.G, rows, x.lim0, x.kv_len);
  __syncwarp();  // before the next stretch's copies
}

// scan_own by every warp for itself, up to kWarpScan sequences a lane: no barriers, and
// nothing goes through shared memory; `gaps`: there may be tokens that no unit has.  One token over 1000 rows 10.7 -> 9.5 us, 37
// sequences of up to 4099 15.3 -> 14.3 (one token of 28 heads of 64 each), 64 of up to 8192
// 70.9 and 71.0, 128 of up to 1024 32.8 -> 32.9, 256 47.0 -> 49.2.
constexpr int kWarpScan = 2;
template <class K>
__device__ __forceinline__ OwnScan scan_warp(const AttnArgs &g, int per, bool *gaps) {
  const int lane = threadIdx.x & 31;
  OwnScan r = {};
  r.b_lo = lane * per;
  r.b_hi = min(r.b_lo + per, g.a.B);
  int64_t mine = 0;
  bool bad_off = false, bad = false, gap = false;
#pragma unroll 1
  for (int b = r.b_lo; b < r.b_hi; ++b) {
    const Seq s = read_seq<K>(g, b, &bad_off, &bad);
    mine += s.cost;
    gap |= s.nq > 0 && s.steps == 0;
    gap |= (b == 0 && s.q0 > 0) || (b == g.a.B - 1 && s.q0 + s.nq < g.a.T);
  }
  if (g.a.B == 0) {  // no sequence reads the one offset that there is
    const int q0 = g.a.q_offsets[0];
    bad_off = q0 < 0 || q0 > g.a.T;
  }
  *gaps = __any_sync(0xffffffffu, gap) || g.a.B == 0;
  int64_t cost = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t c = __shfl_up_sync(0xffffffffu, cost, off);
    if (lane >= off) cost += c;
  }
  r.drop = __any_sync(0xffffffffu, bad_off);
  r.bad = bad || bad_off;
  r.before = cost - mine;
  r.total = r.drop ? 0 : __shfl_sync(0xffffffffu, cost, 31);
  return r;
}

// Walks the units in [lo, hi) of their line, a whole warp, sequence by sequence from
// the one where the scan has lo.  (The walk of attention.cuh looks at 32
// sequences at a time, which a few units a worker do not pay back: 64 sequences of up
// to 8192 rows 71.6 us with it, 70.4 so; one token over 1000 rows 11.2 and 10.8.)
template <class K>
struct Walk4 {
  int64_t lo, hi, start, unit_cost;
  int b, j;
  Seq s;

  // from the sequence before `first`, whose units start at `at`
  __device__ __forceinline__ void begin(int first, int64_t at, int64_t lo_, int64_t hi_) {
    lo = lo_;
    hi = hi_;
    b = first - 1;
    start = at;
    s.cost = 0;
    s.units = j = 0;
    unit_cost = 1;
  }
  __device__ __forceinline__ bool next(const AttnArgs &g, Stretch *out) {
    while (true) {
      while (j < s.units) {
        const int at = j++;
        const int64_t from = start + at * unit_cost;
        if (from >= hi) return false;
        out->s0 = step_at<K>(lo - from, s.steps, 0);
        out->s1 = step_at<K>(hi - from, s.steps, 0);
        if (out->s0 >= out->s1) continue;
        out->n = s.steps;
        const int block = at / g.a.hkv, i0 = block * g.own.tok;
        out->head = at - block * g.a.hkv;
        out->tok0 = s.q0 + i0;
        out->ntok = min(g.own.tok, s.nq - i0);
        out->lim0 = s.len - s.nq + i0 + 1;
        out->kv_len = s.len;
        out->pages = g.a.page_table + static_cast<int64_t>(b) * g.a.max_pages;
        return true;
      }
      start += s.cost;
      if (++b >= g.a.B || start >= hi) return false;
      bool x = false, y = false;
      s = read_seq<K>(g, b, &x, &y);
      if (s.cost == 0) s.units = 0;
      unit_cost = s.steps + K::kUnitCost;
      j = lo <= start ? 0 : static_cast<int>(min(quotient(lo - start, unit_cost), int64_t{s.units}));
    }
  }
};

// Tokens that no unit has, of sequences without rows and of no sequence, by a CTA.
template <int D>
__device__ __forceinline__ void clear_token(const PrefixAttnArgs &a, int64_t t) {
  uint4 *row = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o) + t * a.o_stride);
  for (int i = threadIdx.x; i < a.hq * (D / 8); i += blockDim.x) row[i] = make_uint4(0, 0, 0, 0);
  if (a.lse)
    for (int h = threadIdx.x; h < a.hq; h += blockDim.x) a.lse[t * a.hq + h] = -INFINITY;
}

// A unit that a worker began and did not end: its parts are the worker's tail part
// and the head parts of the `parts - 1` workers after it.  (parts 0: there is none.)
struct Begun {
  int parts, head, tok0, ntok, lim0, kv_len;
};
// A short form of it where there are at most kFewUnits: the unit's number and its parts.
constexpr int kFewUnits = 64;
__device__ __forceinline__ int short_form(const PrefixAttnArgs &a, const Begun &u) {
  return u.parts * kFewUnits + (u.tok0 * a.hkv + u.head) % kFewUnits;
}
// A worker has at most two parts: of a unit begun before it, of one that goes on after.
enum { kTail = 0, kHead = 1 };
__host__ __device__ constexpr int part_floats(int rows, int D) {  // 16-byte aligned rows
  return rows * D + (rows + 3) / 4 * 4;
}
template <int D>
__device__ __forceinline__ float *part_at(const AttnArgs &g, int worker, int which) {
  return g.part_o + static_cast<int64_t>(2 * worker + which) * part_floats(g.own.rows, D);
}

template <int DTYPE, int D, int NT, int NH, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 1)
    kv4_attention_kernel(const __grid_constant__ AttnArgs g, const int split, Begun *begun, int *few) {
  using C = Cfg4<D, NH, WARPS>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ ScanShared<WARPS * 32> scan;
  const PrefixAttnArgs &a = g.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // lengths, offsets and page numbers on their way to L2 while the kernels before
  // this one end (who writes them does it there, too)
  const int at = blockIdx.x * (WARPS * 32) + threadIdx.x, lines = gridDim.x * (WARPS * 32);
  auto prefetch = [&](const int32_t *p, int64_t n) {
    for (int64_t i = at; i * 32 < n; i += lines)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p + i * 32));
  };
  prefetch(a.kv_lens, a.B);
  if (a.q_offsets) prefetch(a.q_offsets, a.B + 1);
  prefetch(a.page_table, static_cast<int64_t>(a.B) * a.max_pages);
  pdl_begin();
  // the line's length, and where this thread's sequences start in it
  const bool by_warp = a.B <= 32 * kWarpScan;
  const int per = by_warp ? (a.B + 31) >> 5 : (a.B + WARPS * 32 - 1) / (WARPS * 32);
  OwnScan own;
  bool gaps = true;
  if (by_warp) {
    own = scan_warp<Steps4<NH>>(g, per, &gaps);
  } else {
    own = scan_own<Steps4<NH>>(g, scan);
  }
  if (blockIdx.x == 0 && own.bad) set_status(a.status, kStatusBadId);
  const int64_t workers = gridDim.x * WARPS;
  const int64_t piece = max(quotient(own.total + workers - 1, workers), static_cast<int64_t>(1));
  // consecutive pieces on different SMs
  const int worker = warp * gridDim.x + blockIdx.x;
  const int64_t lo = worker * piece, hi = min(lo + piece, own.total);
  Begun goes_on = {0, 0, 0, 0, 0, 0};
  if (lo < hi) {
    // the last thread of the scan whose sequences start at or before lo
    int i = 0;
    int64_t at = 0;
    if (by_warp) {
      i = 31 - __clz(__ballot_sync(0xffffffffu, own.before <= lo));
      at = __shfl_sync(0xffffffffu, own.before, i);
    } else {
      for (int k = lane; k < WARPS * 32; k += 32)
        if (scan.before[k] <= lo) i = k;
      i = __reduce_max_sync(0xffffffffu, i);
      at = scan.before[i];
    }
    Walk4<Steps4<NH>> walk;
    walk.begin(i * per, at, lo, hi);
    Stretch x;
    while (walk.next(g, &x)) {
      float *part = x.s0 > 0 ? part_at<D>(g, worker, kHead)
                    : x.s1 < x.n ? part_at<D>(g, worker, kTail) : nullptr;
      attend<DTYPE, D, NT, NH, WARPS>(g, x, split, part, smem + warp * C::WARP_BYTES);
      if (x.s0 == 0 && x.s1 < x.n)  // the worker's last: steps that follow, a piece each worker
        goes_on = {1 + static_cast<int>(quotient(x.n - x.s1 + piece - 1, piece)), x.head, x.tok0,
                   x.ntok, x.lim0, x.kv_len};
      if (x.s1 < x.n) break;
    }
  }
  if (lane == 0) {
    begun[worker] = goes_on;
    if (few) few[worker] = short_form(a, goes_on);
  }
  if (own.drop || !gaps) return;  // offsets within [0, T] from here on
  bool p = false, q = false;
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const Seq s = read_seq<Steps4<NH>>(g, b, &p, &q);
    if (s.steps == 0)
      for (int i = 0; i < s.nq; ++i) clear_token<D>(a, s.q0 + i);
  }
  if (a.q_offsets) {
    const int before = a.q_offsets[0], after = a.q_offsets[a.B];
    for (int t = blockIdx.x; t < before; t += gridDim.x) clear_token<D>(a, t);
    for (int t = after + blockIdx.x; t < a.T; t += gridDim.x) clear_token<D>(a, t);
  }
}

// Of a row's parts those of the workers sub, sub + EVERY, ... after the first, by a
// warp: their sum (rows of D from `parts` on, log2-sum-exps from `lses` on, both the first
// worker's tail part) as o and l, to the power of two `ref`.
template <int D, int EVERY>
__device__ __forceinline__ void add_parts(const float *parts, const float *lses, int two, int n, int sub,
                                          float (&o)[D / 32], float *sum, float *ref) {
  constexpr int E = D / 32, kBatch = 8;
  const int lane = threadIdx.x & 31, count = EVERY == 1 ? n : (n - sub + EVERY - 1) / EVERY;
  auto ahead = [&](int i) {
    const int k = EVERY == 1 ? i : sub + i * EVERY;
    return k == 0 ? 0 : k * two + two / 2;
  };
  static_assert(kTail == 0 && kHead == 1, "a worker's head part follows its tail part");
  float x[kBatch][E], l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
  auto fetch = [&](int k) {
#pragma unroll
    for (int c = 0; c < kBatch; ++c)
      if (k + c < count) {
        const float *src = parts + ahead(k + c) + lane * E;
        if constexpr (E == 4)
          *reinterpret_cast<float4 *>(x[c]) = *reinterpret_cast<const float4 *>(src);
        else
          *reinterpret_cast<float2 *>(x[c]) = *reinterpret_cast<const float2 *>(src);
      }
  };
  float mine = lane < count ? lses[ahead(lane)] : -INFINITY;
  fetch(0);  // before the maximum is known
  float top = mine;
  for (int i = lane + 32; i < count; i += 32) top = fmaxf(top, lses[ahead(i)]);
#pragma unroll
  for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  top = top == -INFINITY ? 0.0f : top;
#pragma unroll 1
  for (int k = 0; k < count; k += kBatch) {
    if (k && (k & 31) == 0) mine = k + lane < count ? lses[ahead(k + lane)] : -INFINITY;
    const float weight = ex2(mine - top);
#pragma unroll
    for (int c = 0; c < kBatch; ++c) {
      const float w = __shfl_sync(0xffffffffu, weight, (k + c) & 31);
      l += w;
      if (k + c < count)  // a part that weighs nothing, too: it may be NaN
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(w, x[c][e], o[e]);
    }
    if (k + kBatch < count) fetch(k + kBatch);
  }
  *sum = l;
  *ref = top;
}
template <int DTYPE, int D>
__device__ __forceinline__ void write_joined(const AttnArgs &g, const Begun &u, int r,
                                             const float (&o)[D / 32], float l, float ref) {
  const int lane = threadIdx.x & 31, i = r * g.tpt >> 16;
  const Row4 row = row_at<D>(g.a, u.tok0 + i, u.head * g.G + r - i * g.G);
  const float inv = l != 0.0f ? 1.0f / l : min(u.kv_len, u.lim0 + i) > 0 ? NAN : 0.0f;
  if constexpr (D == 128)
    *reinterpret_cast<uint2 *>(row.o + 4 * lane) =
        make_uint2(pack2<DTYPE>(o[0] * inv, o[1] * inv), pack2<DTYPE>(o[2] * inv, o[3] * inv));
  else
    *reinterpret_cast<uint32_t *>(row.o + 2 * lane) = pack2<DTYPE>(o[0] * inv, o[1] * inv);
  if (row.lse && lane == 0)
    *row.lse = l != 0.0f ? (ref + log2f(l)) * 0.6931471805599453f : isnan(inv) ? inv : -INFINITY;
}

// The units that several workers had: a CTA joins those that its workers began, a warp a
// row (of 8, blockIdx.y says which).  Two workers a CTA: 37 sequences of up to 4099 rows, 6
// tokens of 7 heads of 64: 24.8 us with one, 24.3 with two, 25.5 with four; 64 of up to 8192
// (heads of 128) 71.3, 71.2, 72.0.
constexpr int kJoinWorkers = 2;
template <int DTYPE, int D>
__global__ void __launch_bounds__(256, D == 128 ? 3 : 4) kv4_join_kernel(const AttnArgs g, const Begun *begun) {
  pdl_begin();
  const int lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5);
  Begun of = {0, 0, 0, 0, 0, 0};
  if (lane < kJoinWorkers) of = begun[blockIdx.x * kJoinWorkers + lane];
  unsigned todo = __ballot_sync(0xffffffffu, of.parts != 0 && r < of.ntok * g.G);
#pragma unroll 1
  for (; todo; todo &= todo - 1) {
    const int k = __ffs(todo) - 1;
    auto take = [&](int v) { return __shfl_sync(0xffffffffu, v, k); };
    const Begun u = {take(of.parts), take(of.head), take(of.tok0),
                     take(of.ntok),  take(of.lim0), take(of.kv_len)};
    const float *tail = part_at<D>(g, blockIdx.x * kJoinWorkers + k, kTail);
    float o[D / 32], l, ref;
    add_parts<D, 1>(tail + r * D, tail + g.own.rows * D + r, 2 * part_floats(g.own.rows, D), u.parts, 0,
                    o, &l, &ref);
    write_joined<DTYPE, D>(g, u, r, o, l, ref);
  }
}

// The same where a batch has few units, which may have many parts each: blockIdx.x is a
// unit's number, blockIdx.y its row, whose parts the CTA's warps take in turn.  One token
// over 1000 rows (16 parts; 8 + 8 x 8 heads of 128) 11.4 us with it, 10.8 without, over
// 2000 11.6 and 12.0, over 8000 14.6 and 20.8, over 131072 44 and 58.
template <int DTYPE, int D>
__global__ void __launch_bounds__(256) kv4_join_few_kernel(const AttnArgs g, const Begun *begun,
                                                           const int *few, const int workers) {
  pdl_begin();
  constexpr int E = D / 32, kWarps = 8;
  __shared__ __align__(16) float s_o[kWarps][D];
  __shared__ float s_ref[kWarps], s_l[kWarps];
  __shared__ int s_worker, s_parts;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.y;
  bool found = false;
#pragma unroll
  for (int k = 0; k < kMaxCtas * kMostWarps4; k += 4 * 256) {
    const int i = k + 4 * threadIdx.x;
    if (i >= workers) continue;  // a multiple of 4
    const int4 w = *reinterpret_cast<const int4 *>(few + i);
    const int of[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (of[c] >= kFewUnits && of[c] % kFewUnits == static_cast<int>(blockIdx.x)) {
        found = true;
        s_worker = i + c;
        s_parts = of[c] / kFewUnits;
      }
  }
  if (!__syncthreads_or(found)) return;  // no unit, or one that a worker has whole
  const int worker = s_worker;
  const Begun u = begun[worker];
  float o[E], l, ref;
  add_parts<D, kWarps>(part_at<D>(g, worker, kTail) + r * D,
                       part_at<D>(g, worker, kTail) + g.own.rows * D + r,
                       2 * part_floats(g.own.rows, D), s_parts, warp, o, &l, &ref);
  if (r >= u.ntok * g.G) return;  // the whole CTA
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
  if (lane == 0) {
    s_ref[warp] = l == 0.0f ? -INFINITY : ref;
    s_l[warp] = l;
  }
  __syncthreads();
  if (warp > 0) return;
  ref = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) ref = fmaxf(ref, s_ref[w]);
  ref = ref == -INFINITY ? 0.0f : ref;
  l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
#pragma unroll 1
  for (int w = 0; w < kWarps; ++w) {
    const float weight = ex2(s_ref[w] - ref);
    l = fmaf(weight, s_l[w], l);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(weight, s_o[w][lane * E + e], o[e]);
  }
  write_joined<DTYPE, D>(g, u, r, o, l, ref);
}

// The plan: query rows of a unit.
struct Plan4 {
  int split, blocks8;  // parts of a key head's queries, blocks of 8 rows in a unit
};
constexpr int kMostRows4 = 16;  // of a unit
Plan4 plan(AttnArgs &g, int T, int max_q, int hq, int hkv) {
  const int G = hq / hkv, nq = std::max(1, std::min(max_q, T));
  Plan4 p = {};
  // more query heads than a unit has rows: equal parts of them
  int Gs = std::min(G, kMostRows4);
  while (G % Gs != 0) --Gs;
  p.split = G / Gs;
  p.blocks8 = static_cast<int64_t>(nq) * Gs <= 8 ? 1 : 2;
  g.G = Gs;
  g.tpt = (65536 + Gs - 1) / Gs;  // r * tpt >> 16 = r / Gs
  g.own.tok = std::min(std::max(1, 8 * p.blocks8 / Gs), nq);
  g.own.rows = g.own.tok * Gs;
  return p;
}
constexpr size_t kBegunBytes = (sizeof(Begun) * kMaxCtas * kMostWarps4 + 255) / 256 * 256;
constexpr size_t kFewBytes = (sizeof(int) * kMaxCtas * kMostWarps4 + 255) / 256 * 256;

template <int DTYPE, int D, int NT, int NH, int WARPS>
cudaError_t run(const AttnArgs &g, int split, Begun *begun, int ctas, cudaStream_t s) {
  using C = Cfg4<D, NH, WARPS>;
  static_assert(WARPS <= kMostWarps4 && WARPS % 4 == 0, "slots of partial results");
  auto kernel = kv4_attention_kernel<DTYPE, D, NT, NH, WARPS>;
  // once for a device (0.7 us a call)
  static std::atomic<uint64_t> known{0};
  int device = 0;
  cudaError_t err = cudaGetDevice(&device);
  if (err != cudaSuccess) return err;
  const uint64_t bit = device < 64 ? uint64_t{1} << device : 0;
  if ((known.load(std::memory_order_relaxed) & bit) == 0) {
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (err != cudaSuccess) return err;
    known.fetch_or(bit, std::memory_order_relaxed);
  }
  const int64_t units = static_cast<int64_t>(g.a.T) * g.a.hkv;  // at most, and their parts:
  const int64_t parts = (static_cast<int64_t>(g.a.max_pages) << g.a.page_shift) / C::KEYS;
  int *few = nullptr;
  if (units <= kFewUnits && parts > 20) few = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(begun) + kBegunBytes);
  MOE_LAUNCH_PDL(kernel, ctas, WARPS * 32, C::SMEM_BYTES, s, g, split, begun, few);
  if (few)
    MOE_LAUNCH_PDL(kv4_join_few_kernel<DTYPE, D>, dim3(static_cast<unsigned>(units), g.own.rows), 256, 0, s,
                   g, begun, few, ctas * WARPS);
  else
    MOE_LAUNCH_PDL(kv4_join_kernel<DTYPE, D>, dim3(ctas * WARPS / kJoinWorkers, (g.own.rows + 7) / 8), 256,
                   0, s, g, begun);
  return cudaGetLastError();
}
template <int DTYPE, int D>
cudaError_t run_d(const AttnArgs &g, const Plan4 &p, Begun *begun, int ctas, cudaStream_t s) {
  if (p.blocks8 == 1) return run<DTYPE, D, 1, 4, 12>(g, p.split, begun, ctas, s);
  return run<DTYPE, D, 2, D == 128 ? 2 : 4, 8>(g, p.split, begun, ctas, s);
}

}  // namespace

size_t kv4_attention_scratch_bytes(int T, int max_q, int hq, int hkv, int D) {
  AttnArgs g = {};
  plan(g, T, max_q, hq, hkv);
  return kBegunBytes + kFewBytes +
         sizeof(float) * kMaxCtas * kMostWarps4 * 2 * static_cast<size_t>(part_floats(g.own.rows, D));
}

cudaError_t launch_kv4_attention(const PrefixAttnArgs &a, int dtype, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  AttnArgs g = {};
  g.a = a;
  const int ctas = std::min(num_sms(), kMaxCtas);
  const Plan4 p = plan(g, a.T, a.max_q, a.hq, a.hkv);
  g.a.hkv = a.hkv * p.split;  // units are counted by parts of a key head's queries
  Begun *begun = reinterpret_cast<Begun *>(a.scratch);
  g.part_o = reinterpret_cast<float *>(a.scratch + kBegunBytes + kFewBytes);
  if (dtype == MOE_DTYPE_BF16)
    return a.D == 64 ? run_d<MOE_DTYPE_BF16, 64>(g, p, begun, ctas, s)
                     : run_d<MOE_DTYPE_BF16, 128>(g, p, begun, ctas, s);
  return a.D == 64 ? run_d<MOE_DTYPE_FP16, 64>(g, p, begun, ctas, s)
                   : run_d<MOE_DTYPE_FP16, 128>(g, p, begun, ctas, s);
}

}  // namespace moe
