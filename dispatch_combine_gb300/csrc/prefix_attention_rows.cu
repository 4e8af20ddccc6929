// prefix_attention_rows.cu -- shared-prefix attention for few query rows.
//
// With up to 16 rows (tokens x query heads of a key head) per unit, or 32 at D =
// 64, the work is reading keys and values: at D = 128 a slice of 16 keys is 8 KB
// and 32 small MMAs.  So every warp works for itself: it owns a piece of the
// line, streams its slices through a private ring in shared memory
// (cp.async, the next slices always in flight), and keeps queries, scores,
// probabilities and accumulators in registers (mma.sync m16n8k16, which a
// few rows fill better than a 128-row tensor-memory tile).  Warps never wait
// for one another; eight of them per SM keep up to 128 KB in flight.  Bound by
// HBM: 64 sequences of up to 8192 rows (1.23 GB of cache in 190 us) run at 0.95
// of the measured copy bandwidth, 256 of up to 512 (287 MB) in 64 us with the
// join, one token over 131072 shared rows (537 MB) in 96 us.
//
// Layouts.  K and V slices are copied as they lie in a page (16 rows of one
// head, contiguous), 16-byte chunk c of row r at chunk c ^ 4 (r & 1) for K and
// c ^ (r & 7) for V, so that the reads below meet no bank conflict.  The order
// of the contraction over D is free as long as Q and K agree: a lane's
// operands for two MMAs are one 16-byte chunk of a K row (lane g, t of key g:
// dims 32 j + 8 t .. + 7).
#include "attention.cuh"

namespace moe {
namespace {

// WARPS per CTA: 8, or 2 beside the tiles kernel for a small batch, where a
// small CTA starts sooner (37 tokens, 4 key heads of 7 at D = 64, prefix 128, own
// rows up to 777: 17.2 us, 18.4 with 8).  Every CTA reads the batch's lengths
// once, so large batches want large CTAs (4096 sequences of up to 512 over 1024,
// 16 + 2 heads: 318 and 285 us); from 64 to 256 sequences the two are within 1 us.
template <int D, int WARPS>
struct RowCfg {
  static constexpr int SLICE = kSlice * D * 2;     // bytes of K or of V
  static constexpr int STAGES = D == 128 ? 3 : 6;  // 24 KB per warp
  static constexpr int WARP_BYTES = STAGES * 2 * SLICE;
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
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t &a, uint32_t &b, uint32_t &c,
                                          uint32_t &d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr));
}
template <int DTYPE>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if (DTYPE == MOE_DTYPE_BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One stretch, by one warp.  `slot`: first row of its partial result.
template <int DTYPE, int D, int MT, int WARPS>
__device__ __forceinline__ void attend(const AttnArgs &g, const Stretch &x, int64_t slot,
                                       uint32_t ring) {
  using C = RowCfg<D, WARPS>;
  const PrefixAttnArgs &a = g.a;
  const int lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3;
  const int rows = x.ntok * g.G;
  // ---- queries: row r is head r % G of token r / G
  uint4 q[MT][2][D / 32];
  int lim[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = m * 16 + h * 8 + gr;
      const int i = r / g.G, hd = r - i * g.G;
      const bool live = r < rows;
      const uint16_t *src = static_cast<const uint16_t *>(a.q) + (x.tok0 + i) * a.q_stride +
                            (x.head * g.G + hd) * D + 8 * t;
#pragma unroll
      for (int j = 0; j < D / 32; ++j)
        q[m][h][j] = live ? *reinterpret_cast<const uint4 *>(src + 32 * j) : make_uint4(0, 0, 0, 0);
      lim[m][h] = live ? min(x.kv_len, x.lim0 + i) : x.kv_len;
    }
  // ---- the ring.  A slice lies in one page (pages hold 16 rows or more);
  // lane i keeps the page of slice `page0 + i`.
  const uint8_t *kc = static_cast<const uint8_t *>(a.k_cache);
  const uint8_t *vc = static_cast<const uint8_t *>(a.v_cache);
  const int spp = a.page_shift - 4;  // log2 of slices per page
  int page0 = x.s0, page = 0;
  auto fetch_pages = [&](int s) {
    page0 = s;
    page = 0;
    if (s + lane < x.s1) {
      page = x.pages[(s + lane) >> spp];
      if (page < 0 || page >= a.num_pages) {
        set_status(a.status, kStatusBadId);
        page = 0;
      }
    }
  };
  fetch_pages(x.s0);
  auto load = [&](int s) {  // slice s into its stage; past the end: an empty group
    if (s < x.s1) {
      if (s - page0 == 32) fetch_pages(s);
      const int64_t p = __shfl_sync(0xffffffffu, page, s - page0);
      const int64_t row =
          ((p * a.hkv + x.head) << a.page_shift) + ((s & ((1 << spp) - 1)) << 4);
      const int stage = (s - x.s0) % C::STAGES;
      const uint32_t dk = ring + stage * 2 * C::SLICE, dv = dk + C::SLICE;
      const int valid = x.kv_len - s * kSlice;  // rows past it read as zero
#pragma unroll
      for (int i = 0; i < C::SLICE / 512; ++i) {
        const int c = i * 32 + lane, r = c / (D / 8), ch = c % (D / 8);
        const uint32_t n = r < valid ? 16u : 0u;
        const int64_t off = row * (D * 2) + c * 16;
        cp_async16(dk + r * (D * 2) + ((ch ^ ((r & 1) * 4)) << 4), kc + off, n);
        cp_async16(dv + r * (D * 2) + ((ch ^ (r & 7)) << 4), vc + off, n);
      }
    }
    cp_async_commit();
  };
  float o[MT][D / 8][4], mx[MT][2], l[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[m][n][e] = 0.0f;
    mx[m][0] = mx[m][1] = -INFINITY;
    l[m][0] = l[m][1] = 0.0f;
  }
  const float sl2 = a.scale * kLog2e;
  const float lag = score_lag<DTYPE>(sl2);
  const int all_seen = min(x.kv_len, x.lim0);  // keys that every token sees
#pragma unroll 1
  for (int s = x.s0 - (C::STAGES - 1); s < x.s1; ++s) {
    if (s >= x.s0) {  // the first passes only fill the ring
    cp_async_wait<C::STAGES - 2>();
    __syncwarp();
    const int stage = (s - x.s0) % C::STAGES;
    const uint32_t sk = ring + stage * 2 * C::SLICE, sv = sk + C::SLICE;
    // ---- scores
    float sc[MT][2][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[m][n][e] = 0.0f;
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint4 k = lds128(sk + (n * 8 + gr) * (D * 2) + (((4 * j + t) ^ ((gr & 1) * 4)) << 4));
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          mma16816<DTYPE>(sc[m][n], q[m][0][j].x, q[m][1][j].x, q[m][0][j].y, q[m][1][j].y, k.x,
                          k.y);
          mma16816<DTYPE>(sc[m][n], q[m][0][j].z, q[m][1][j].z, q[m][0][j].w, q[m][1][j].w, k.z,
                          k.w);
        }
      }
    if ((s + 1) * kSlice > all_seen) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (s * kSlice + n * 8 + 2 * t + (e & 1) >= lim[m][e >> 1]) sc[m][n][e] = -INFINITY;
    }
    // ---- the running maximum moves when a score passes it by `lag`
    bool moves = false;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        moves |= fmaxf(fmaxf(sc[m][0][2 * h], sc[m][0][2 * h + 1]),
                       fmaxf(sc[m][1][2 * h], sc[m][1][2 * h + 1])) - mx[m][h] > lag;
    if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float top = fmaxf(fmaxf(sc[m][0][2 * h], sc[m][0][2 * h + 1]),
                            fmaxf(sc[m][1][2 * h], sc[m][1][2 * h + 1]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          top = in_range<DTYPE>(top, sl2);
          if (top > mx[m][h]) {
            const float f = rescale<DTYPE>(mx[m][h], top, sl2);
            mx[m][h] = top;
            l[m][h] *= f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              o[m][n][2 * h] *= f;
              o[m][n][2 * h + 1] *= f;
            }
          }
        }
    }
    // ---- probabilities, rounded to the cache's type for the product with V
    uint32_t p[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float c0 = prob_offset<DTYPE>(mx[m][h], sl2);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float e0 = ex2(fmaf(sc[m][n][2 * h], sl2, c0));
          const float e1 = ex2(fmaf(sc[m][n][2 * h + 1], sl2, c0));
          l[m][h] += e0 + e1;
          p[m][2 * n + h] = pack2<DTYPE>(e0, e1);
        }
      }
    // ---- product with V: matrices (keys 0-7, 8-15) x (dims 16 n, 16 n + 8)
    const int vr = lane & 15, vch = lane >> 4;
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
      uint32_t b0, b1, b2, b3;
      ldsm_x4_t(sv + vr * (D * 2) + (((2 * n + vch) ^ (vr & 7)) << 4), b0, b1, b2, b3);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        mma16816<DTYPE>(o[m][2 * n], p[m][0], p[m][1], p[m][2], p[m][3], b0, b1);
        mma16816<DTYPE>(o[m][2 * n + 1], p[m][0], p[m][1], p[m][2], p[m][3], b2, b3);
      }
    }
    __syncwarp();  // the stage of the last slice is free again
    }
    load(s + C::STAGES - 1);
  }
  cp_async_wait<0>();
  __syncwarp();
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float sum = l[m][h];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int r = m * 16 + h * 8 + gr;
      if (r >= rows) continue;
      const PartEnd end = end_part<DTYPE>(mx[m][h], sum, sl2);
      float *dst = g.part_o + (slot + r) * D + 2 * t;
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2 *>(dst + 8 * n) =
            make_float2(o[m][n][2 * h] * end.inv, o[m][n][2 * h + 1] * end.inv);
      if (t == 0) g.part_lse[slot + r] = end.lse;  // in powers of two
    }
}

template <int DTYPE, int D, int MT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, kRowWarps / WARPS)
    attention_rows_kernel(const AttnArgs g, const int beside) {
  // Beside the tiles kernel of the same call, which has waited for everything
  // before the call and shares nothing with this one: only the last CTA waits
  // for it, at its end, so that whoever waits for this kernel has waited for
  // both.
  if (beside)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  else
    pdl_begin();
  using C = RowCfg<D, WARPS>;
  auto leave = [&]() {
    if (beside && blockIdx.x == gridDim.x - 1)
      asm volatile("griddepcontrol.wait;" ::: "memory");
  };
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ ScanShared<WARPS * 32> scan;
  const int warp = threadIdx.x >> 5;
  OwnScan own = {};
  if (g.own_rows_kernel) own = scan_own<SliceSteps>(g, scan);
  const int64_t total = g.r_ptotal + own.total;
  int ctas = gridDim.x;
  if (beside) ctas = share_out<D>(g, own.total, ctas * WARPS / kRowWarps).workers / WARPS;
  const int64_t piece = max(quotient(total + ctas * WARPS - 1, ctas * WARPS),
                            static_cast<int64_t>(kMinSlices));
  if (blockIdx.x == 0 && g.own_rows_kernel) write_meta<SliceSteps>(g, own);
  // consecutive pieces on different SMs
  const int worker = warp * ctas + blockIdx.x;
  const int64_t lo = static_cast<int64_t>(worker) * piece, hi = min(lo + piece, total);
  if (lo >= total || static_cast<int>(blockIdx.x) >= ctas) {
    leave();
    return;
  }
  const uint32_t ring = smem_u32(smem) + warp * C::WARP_BYTES;
  const bool any_own = own.total > 0 && hi > g.r_ptotal;
  OwnWalk<SliceSteps> walk;
  if (any_own) walk.begin(g, scan, max(lo - g.r_ptotal, int64_t{0}), hi - g.r_ptotal);
  int64_t u = lo < g.r_ptotal ? quotient(lo, g.r_pcost) : 0;
  bool in_prefix = lo < g.r_ptotal;
  while (true) {
    Stretch x;
    int64_t slot, place;
    if (in_prefix) {
      if (u * g.r_pcost >= min(hi, g.r_ptotal)) {
        in_prefix = false;
        continue;
      }
      const int64_t at = u++;
      x.n = g.r_slices;
      x.s0 = step_at<SliceSteps>(lo - at * g.r_pcost, x.n, 0);
      x.s1 = step_at<SliceSteps>(hi - at * g.r_pcost, x.n, 0);
      if (x.s0 >= x.s1) continue;
      x.head = static_cast<int>(quotient(at, g.r_blocks));
      x.tok0 = static_cast<int>(at - static_cast<int64_t>(x.head) * g.r_blocks) * g.r_tok;
      x.ntok = min(g.r_tok, g.a.T - x.tok0);
      x.lim0 = x.kv_len = g.a.prefix_len;
      x.pages = g.a.prefix_pages;
      slot = (at + worker) * g.r_rows;
      place = at;
    } else {
      if (!any_own || !walk.next(g, &x)) break;
      slot = g.own.slot0 + (x.unit + worker) * g.own.rows;
      place = g.own.span0 + x.unit;
    }
    if ((threadIdx.x & 31) == 0) mark_span(g, place, x, worker);
    attend<DTYPE, D, MT, WARPS>(g, x, slot, ring);
  }
  leave();
}

template <int DTYPE, int D, int MT, int WARPS>
cudaError_t run(const AttnArgs &g, int ctas, cudaStream_t s) {
  using C = RowCfg<D, WARPS>;
  auto kernel = attention_rows_kernel<DTYPE, D, MT, WARPS>;
  const cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (err != cudaSuccess) return err;
  MOE_LAUNCH_PDL(kernel, ctas * kRowWarps / WARPS, WARPS * 32, C::SMEM_BYTES, s, g, g.share);
  return cudaGetLastError();
}

template <int DTYPE, int D>
cudaError_t run_d(const AttnArgs &g, int ctas, cudaStream_t s) {
  const bool small = g.share && g.a.B <= 128;
  if constexpr (D == 64)  // 16 rows are the most at D = 128
    if (g.r_mt == 2)
      return small ? run<DTYPE, D, 2, 2>(g, ctas, s) : run<DTYPE, D, 2, kRowWarps>(g, ctas, s);
  return small ? run<DTYPE, D, 1, 2>(g, ctas, s) : run<DTYPE, D, 1, kRowWarps>(g, ctas, s);
}

}  // namespace

cudaError_t launch_attention_rows(const AttnArgs &g, int dtype, int ctas, cudaStream_t s) {
  if (dtype == MOE_DTYPE_BF16)
    return g.a.D == 64 ? run_d<MOE_DTYPE_BF16, 64>(g, ctas, s)
                       : run_d<MOE_DTYPE_BF16, 128>(g, ctas, s);
  return g.a.D == 64 ? run_d<MOE_DTYPE_FP16, 64>(g, ctas, s)
                     : run_d<MOE_DTYPE_FP16, 128>(g, ctas, s);
}

}  // namespace moe
