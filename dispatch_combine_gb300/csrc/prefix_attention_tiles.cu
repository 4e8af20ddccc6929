// prefix_attention_tiles.cu -- shared-prefix attention for many query rows, on
// the tensor cores.
//
// The query heads of one key head and several tokens fill the 128 rows of a
// tensor-memory tile (row = token * G + head in group).  A CTA's two groups of
// 128 softmax threads each own a 128 x 128 score tile and an output
// accumulator in TMEM.  A wide unit (more than 128 rows) gives each group 128
// of its rows and both read the same K and V tiles; a narrow one gives both
// the same rows and every second tile.  The groups take turns through all
// segments: while one takes exponentials the other's products run, and while
// one ends a unit the other is at the next.
//
// The prefix's token blocks are worked on by gangs: the CTAs of a gang hold
// different blocks and walk the same stretch of the same key head's rows at
// the same time, so that one of them fetches a tile from HBM and the others
// find it in L2.  The own rows of the sequences follow, cut so that all CTAs
// end together.
//
// Bound by the tensor cores (4 D flop per score): a tile of a wide unit is 32
// products of 128 x 128 x 16 per SM at 64 cycles.  256 queries x 64 heads of
// 128 over 131072 rows (1.10 TFLOP) take 755 us, 0.75 of the measured bf16
// peak; the MMAs alone would take 570, the softmax alone 545.
#include <algorithm>
#include <cstddef>
#include <mutex>

#include "attention.cuh"

namespace moe {
namespace {

constexpr int kAttnThreads = 352;  // 8 softmax warps, the loader, two MMA issuers
constexpr int kDescs = 4;          // segments the loader may be ahead

template <int D>
struct AttnCfg {
  static constexpr int BLK = kTile * 128;           // 128 rows x 64 elements
  static constexpr int TILE_BYTES = (D / 64) * BLK;  // a K, V or Q tile
  static constexpr int STAGES = D == 128 ? 2 : 4;
  // Columns of TMEM: scores 128 a group, accumulators D a group.  At D = 128
  // that is all, and the probabilities lie over the scores; at D = 64 they have
  // columns of their own, so that the next scores are computed while the
  // exponentials of these are taken (256 queries over 131072 rows: 610 ->
  // 540 us).
  static constexpr bool APART = D == 64;
  static constexpr int T_P = APART ? 256 : 0;
  static constexpr int T_P_STEP = APART ? 64 : 128;
  static constexpr int T_O = APART ? 384 : 256;
  static constexpr int K_OFF = 2 * TILE_BYTES;
  static constexpr int V_OFF = K_OFF + STAGES * TILE_BYTES;
  static constexpr int BAR_OFF = V_OFF + STAGES * TILE_BYTES;
  static constexpr int SMEM_BYTES = BAR_OFF + 2048 + 1024;  // + barriers, + alignment
};

// One segment, written by the loader and read by every other warp.
struct Segment {
  int t0, t1;       // tiles [t0, t1); t0 == t1 ends the kernel
  int kv_len;       // rows of the unit's keys
  int wide;         // the groups take 128 rows each
  int ntok;         // tokens of the unit
  int lim0;         // token i sees keys below min(kv_len, lim0 + i)
  int rows;         // rows of a slot half
  int64_t slot;     // index of the partial result's first row, in rows
};

// ---------------------------------------------------------------------------
// PTX not in common.cuh
// ---------------------------------------------------------------------------

// Shared-memory descriptor of an N-major operand: rows of 64 elements (128
// bytes, swizzled) run along N, 8-row groups along K follow every 1024
// bytes, the next 64 elements of N `n_step` bytes further.
__device__ __forceinline__ uint64_t sw128_nmajor_desc(uint32_t smem_addr, uint32_t n_step) {
  uint64_t desc = 0;
  desc |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  desc |= static_cast<uint64_t>(n_step >> 4) << 16;
  desc |= static_cast<uint64_t>(1024u >> 4) << 32;
  desc |= static_cast<uint64_t>(1u) << 46;
  desc |= static_cast<uint64_t>(2u) << 61;
  return desc;
}

// Instruction descriptor, 16-bit operands of one type, fp32 accumulator; bit
// 16: B is N-major.
template <int DTYPE>
__host__ __device__ constexpr uint32_t attn_idesc(int M, int N, bool b_nmajor) {
  return (1u << 4) | (DTYPE == MOE_DTYPE_BF16 ? (1u << 7) | (1u << 10) : 0u) |
         (b_nmajor ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// D[tmem] (+)= A[tmem] * B[smem], one elected thread.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(void *smem_dst, const CUtensorMap *map, uint64_t *bar,
                                            int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}
// a condition whose code belongs out of the straight line (the loops below
// pass through the instruction cache once per tile)
__device__ __forceinline__ bool rare(bool x) { return __builtin_expect(x, false); }

// Barriers are addressed by their 32-bit shared-memory address.  A test of a
// complete phase takes about 45 cycles, a try_wait about 125, so waits here
// poll with tests.
__device__ __forceinline__ uint32_t bar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void bar_commit(uint32_t bar) {  // when the MMAs so far are complete
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
// What a wait needs when it becomes long.
struct WaitCtx {
  uint32_t base;  // shared address of the barriers
  uint64_t *bars;
  volatile int *abort;
  uint32_t *status;
  uint64_t limit_ns;
};
// The wait proper, out of line (a dozen places wait, and code that does not
// stay in the instruction cache costs more than the call): polls for as long
// as several tiles take, then by the clock (the global timer takes about a
// microsecond to read).
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, const WaitCtx &c) {
#pragma unroll 1
  for (int i = 0; i < 2048; ++i)
    if (__all_sync(0xffffffffu, bar_test(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait_bounded(c.bars + (bar - c.base) / 8, parity, c.abort,
                                                   c.status, c.limit_ns));
}
// Whole warp: true for all lanes when the phase completed, false for all when
// some lane gave up.
__device__ __forceinline__ bool wait_bar(const WaitCtx &c, uint32_t bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, bar_test(bar, parity))) return true;
  return wait_long(bar, parity, c);
}
// Time-bounded wait that ignores the abort flag (to drain after an abort).
__device__ __noinline__ bool wait_drain(uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 0;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 63u && globaltimer_ns() - t0 > limit_ns) return false;
  }
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------

// Barriers, all in shared memory.  A ring slot's n-th use waits with parity
// n & 1 for full and (n & 1) ^ 1 for empty.
template <int STAGES>
struct Bars {
  uint64_t k_full[STAGES], k_empty[STAGES], v_full[STAGES], v_empty[STAGES];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2];  // scores of a group are in TMEM
  uint64_t s_read[2];  // and in its threads' registers (APART)
  uint64_t p_lo[2], p_hi[2];  // its probabilities are: keys 0-63, 64-127
  uint64_t o_full[2];  // its accumulator is: at the segment's end (APART: after every step)
  uint64_t d_full[kDescs], d_empty[kDescs];
  uint64_t drain[2];
  Segment seg[kDescs];
  uint32_t tmem;
  int abort;
};

template <int DTYPE, int D>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attention_tiles_kernel(const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV,
                            const __grid_constant__ CUtensorMap tmQp,
                            const __grid_constant__ CUtensorMap tmQs, const AttnArgs g) {
  pdl_begin();
  if (!g.own_on && static_cast<int>(blockIdx.x) >= g.p_gangs * g.p_gang) return;
  using C = AttnCfg<D>;
  constexpr int kBlocks = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  using B = Bars<C::STAGES>;
  static_assert(sizeof(B) <= 2048, "barrier block");
  B &bar = *reinterpret_cast<B *>(smem + C::BAR_OFF);
  volatile int *abort_flag = &bar.abort;
  const PrefixAttnArgs &a = g.a;
  constexpr uint64_t limit = kDefaultWaitLimitNs;
  __shared__ ScanShared<kAttnThreads> scan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = smem_u32(&bar);
#define BAR(field, i) (bars + static_cast<uint32_t>(offsetof(B, field)) + 8u * (i))
  const WaitCtx wc = {bars, reinterpret_cast<uint64_t *>(&bar), abort_flag, a.status, limit};

  if (threadIdx.x == 0) {
    bar.abort = 0;
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&bar.k_full[s], 1);
      mbar_init(&bar.k_empty[s], 2);
      mbar_init(&bar.v_full[s], 1);
      mbar_init(&bar.v_empty[s], 2);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&bar.q_full[h], 1);
      mbar_init(&bar.q_empty[h], 2);
      mbar_init(&bar.s_full[h], 1);
      mbar_init(&bar.s_read[h], 4);
      mbar_init(&bar.p_lo[h], 4);
      mbar_init(&bar.p_hi[h], 4);
      mbar_init(&bar.o_full[h], 1);
    }
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(&bar.d_full[i], 1);
      mbar_init(&bar.d_empty[i], 10);
    }
    mbar_init(&bar.drain[0], 1);
    mbar_init(&bar.drain[1], 1);
    fence_mbar_init();
  }
  // ---- what this CTA does: gang member `member` of gang `gang` (in the
  // prefix), then a piece [lo, hi) of the own units' line.  The CTAs outside
  // the gangs take more of that line: all are to end at the same time.
  OwnScan own = {};
  int gangs = g.p_gangs;
  int64_t p_piece = g.p_piece;
  if (g.own_on) {
    own = scan_own<TileSteps>(g, scan);
  } else if (g.share) {
    // the rows kernel gets the SMs of the gangs that are not used
    const int64_t slices = scan_own<SliceSteps>(g, scan).total;
    gangs = share_out<D>(g, slices, gridDim.x).gangs;
    p_piece = quotient(static_cast<int64_t>(a.hkv) * g.p_groups * g.p_tiles + gangs - 1, gangs);
  }
  const int ganged = g.p_on ? gangs * g.p_gang : 0, cta = blockIdx.x;
  const int others = gridDim.x - ganged;
  const int64_t p_time = g.p_on ? p_piece * TileSteps::cost(g.p_wide) : 0;
  int64_t own_ganged = 0, own_other = 1;
  if (own.total > 0) {
    const int64_t least = TileSteps::kMostCost;
    if (own.total <= others * p_time) {
      own_other = max(quotient(own.total + others - 1, others), least);
    } else {
      own_other = max(quotient(own.total + ganged * p_time + gridDim.x - 1, gridDim.x), least);
      own_ganged = own_other > p_time ? max(own_other - p_time, least) : 0;
      if (others == 0) own_other = least;
    }
  }
  if (blockIdx.x == 0 && g.own_on) write_meta<TileSteps>(g, own);
  const int64_t lo = cta < ganged ? cta * own_ganged
                                  : ganged * own_ganged + (cta - ganged) * own_other;
  const int64_t hi = min(lo + (cta < ganged ? own_ganged : own_other), own.total);
  const bool in_gang = cta < ganged;
  if (!in_gang && lo >= own.total) return;  // uniform across the CTA
  __syncthreads();
  if (warp == 9) tmem_alloc(&bar.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = bar.tmem;

  if (warp == 8) {
    // ---------------- loader: walks the line, fetches Q, K and V ----------------
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      tma_prefetch_desc(g.p_on ? &tmQp : &tmQs);
    }
    const int ppt = max(1, kTile >> a.page_shift);  // pages per tile
    const int page_rows = min(1 << a.page_shift, kTile);
    uint32_t issued[2] = {0, 0}, nseg = 0, q_use[2] = {0, 0};  // issued: K and V tiles
    bool ok = true;
    // the gang's stretch of the prefix line (key head, group of blocks, tile):
    // this member has one block of each group
    const int gang = in_gang ? cta / g.p_gang : 0, member = cta - gang * g.p_gang;
    const int64_t p_lo = gang * p_piece;
    const int64_t p_hi = in_gang ? min(p_lo + p_piece, static_cast<int64_t>(a.hkv) *
                                                             g.p_groups * g.p_tiles)
                                 : 0;
    int64_t p_at = in_gang ? p_lo : 0;
    const bool any_own = own.total > 0 && lo < hi;
    OwnWalk<TileSteps> walk;
    if (any_own) walk.begin(g, scan, lo, hi);
    while (ok) {
      Stretch x;
      int64_t slot, place;
      const bool is_own = p_at >= p_hi;
      if (!is_own) {
        const int64_t q = quotient(p_at, g.p_tiles);  // key head and group
        x.head = static_cast<int>(quotient(q, g.p_groups));
        x.s0 = static_cast<int>(p_at - q * g.p_tiles);
        x.s1 = static_cast<int>(min(static_cast<int64_t>(g.p_tiles), x.s0 + (p_hi - p_at)));
        x.n = g.p_tiles;
        p_at += x.s1 - x.s0;
        const int block = static_cast<int>(q - static_cast<int64_t>(x.head) * g.p_groups) *
                              g.p_gang + member;
        if (block >= g.p_blocks) continue;
        x.tok0 = block * g.p_tok;
        x.ntok = min(g.p_tok, a.T - x.tok0);
        x.lim0 = x.kv_len = a.prefix_len;
        x.pages = a.prefix_pages;
        slot = ((q + gang) * g.p_gang + member) * 2 * g.p_rows;
        place = q * g.p_gang + member;
      } else {
        if (!any_own || !walk.next(g, &x)) break;
        slot = g.own.slot0 + (x.unit + cta) * 2 * g.own.rows;
        place = g.own.span0 + x.unit;
      }
      if (lane == 0) mark_span(g, place, x, is_own ? cta : gang);
      const int head = x.head, tok0 = x.tok0, kv_len = x.kv_len, t0 = x.s0, t1 = x.s1;
      const int wide = is_own ? g.s_wide : g.p_wide;
      const int32_t *pages = x.pages;
      auto page_at = [&](int t) {
        int p = -1;
        const int first = static_cast<int>((static_cast<int64_t>(t) * kTile) >> a.page_shift);
        const int last = (kv_len - 1) >> a.page_shift;
        if (t < t1 && lane < ppt && first + lane <= last) {
          p = pages[first + lane];
          if (p < 0 || p >= a.num_pages) {
            set_status(a.status, kStatusBadId);
            p = 0;
          }
        }
        return p;
      };
      int page = page_at(t0);  // on its way while the segment is published
      // publish the segment, then fetch its queries and tiles
      const uint32_t r = nseg % kDescs;
      ok = wait_bar(wc, BAR(d_empty, r), ((nseg / kDescs) & 1u) ^ 1u);
      if (!ok) break;
      const int h0 = wide ? 0 : nseg & 1;  // a narrow unit's rows alternate between the buffers
      if (lane == 0) {
        bar.seg[r] = Segment{t0, t1, kv_len, wide, x.ntok, x.lim0,
                             is_own ? g.own.rows : g.p_rows, slot};
        bar_arrive(BAR(d_full, r));
      }
      ++nseg;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h < h0 || h > h0 + wide) continue;
        ok = wait_bar(wc, BAR(q_empty, h), (q_use[h] & 1u) ^ 1u);
        if (!ok) break;
        ++q_use[h];
        if (lane == 0) {
          const int box = is_own ? g.s_box : g.p_box;
          mbar_arrive_expect_tx(&bar.q_full[h], static_cast<uint32_t>(box * g.G * 128 * kBlocks));
          for (int d = 0; d < kBlocks; ++d)
            tma_load_3d(smem + h * C::TILE_BYTES + d * C::BLK, is_own ? &tmQs : &tmQp, &bar.q_full[h],
                        d * 64, head * g.G, tok0 + (wide ? h * g.tpt : 0));
        }
      }
      if (!ok) break;
#pragma unroll 1
      for (int t = t0; t < t1; ++t) {
        const int next = page_at(t + 1);
        const int stage = issued[0] % C::STAGES;
        const uint32_t par = ((issued[0] / C::STAGES) & 1u) ^ 1u;
        const uint32_t bytes =
            static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, page >= 0)) * page_rows * 128 *
                                  kBlocks);
        const int in_page = (t * kTile) & ((1 << a.page_shift) - 1);  // pages of 256 rows
        const int row = ((page * a.hkv + head) << a.page_shift) + in_page;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          uint64_t *full = which ? &bar.v_full[stage] : &bar.k_full[stage];
          ok = wait_bar(wc, which ? BAR(v_empty, stage) : BAR(k_empty, stage), par);
          if (!ok) break;
          ++issued[which];
          if (lane == 0) mbar_arrive_expect_tx(full, bytes);
          __syncwarp();
          if (page >= 0) {
            uint8_t *dst = smem + (which ? C::V_OFF : C::K_OFF) + stage * C::TILE_BYTES +
                           lane * page_rows * 128;
#pragma unroll
            for (int d = 0; d < kBlocks; ++d)
              tma_load_2d(dst + d * C::BLK, which ? &tmV : &tmK, full, d * 64, row);
          }
        }
        if (!ok) break;
        page = next;
      }
    }
    if (ok) {  // the end
      const uint32_t r = nseg % kDescs;
      ok = wait_bar(wc, BAR(d_empty, r), ((nseg / kDescs) & 1u) ^ 1u);
      if (ok && lane == 0) {
        bar.seg[r] = Segment{0, 0, 0, 0, 0, 0, 0, 0};
        bar_arrive(BAR(d_full, r));
      }
    }
    __syncwarp();
    // every copy must have landed before the CTA exits: a stage's last use
    // is complete when its barrier has passed that use's phase
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll 1
      for (int st = 0; st < C::STAGES; ++st) {
        const uint32_t uses = issued[which] / C::STAGES +
                              (st < static_cast<int>(issued[which] % C::STAGES) ? 1u : 0u);
        if (uses) wait_drain(which ? &bar.v_full[st] : &bar.k_full[st], (uses - 1) & 1u, limit);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (q_use[h]) wait_drain(&bar.q_full[h], (q_use[h] - 1) & 1u, limit);
  } else if (warp >= 9) {
    // ---------------- MMA issuers: warp 9 + w for group w ----------------
    // A product of 128 x 128 x 16 takes 64 cycles and the queue in front of
    // the tensor cores holds four, so what an issuer does between its batches
    // (barrier tests of 50 cycles, forming operands) would show; with a warp
    // per group it is hidden behind the other group's products.  The whole
    // warp walks the steps, so that operands stay warp-uniform, and one elected
    // lane issues.  A group's scores for its next step overwrite the
    // probabilities of this one, and follow its product with V in issue order.
    constexpr uint32_t kIdescQK = attn_idesc<DTYPE>(128, kTile, false);
    constexpr uint32_t kIdescPV = attn_idesc<DTYPE>(128, D, true);
    const uint64_t desc_q = sw128_kmajor_desc(smem_u32(smem));
    const uint64_t desc_k = sw128_kmajor_desc(smem_u32(smem + C::K_OFF));
    const uint64_t desc_v = sw128_nmajor_desc(smem_u32(smem + C::V_OFF), C::BLK);
    const int w = warp - 9;
    const uint32_t t_s = tmem_base + w * 128, t_p = tmem_base + C::T_P + w * C::T_P_STEP;
    const uint32_t t_o = tmem_base + C::T_O + w * D;
    uint32_t nseg = 0, step = 0, p_use = 0, k_tile = 0, v_tile = 0;
    uint32_t q_par = 0;  // a bit per query buffer
    bool ok = true, any = false;
    auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
    // Both groups pass every tile and query buffer in order, and each arrives
    // once on its release (without an MMA where it does not use it), so a
    // buffer's phase never runs ahead of a group that has not looked at it.
    auto skip_k = [&]() {
      const uint32_t st = k_tile % C::STAGES;
      ok = ok && wait_bar(wc, BAR(k_full, st), (k_tile / C::STAGES) & 1u);
      if (ok && lane == 0) bar_arrive(BAR(k_empty, st));
      ++k_tile;
    };
    auto skip_v = [&]() {
      const uint32_t st = v_tile % C::STAGES;
      ok = ok && wait_bar(wc, BAR(v_full, st), (v_tile / C::STAGES) & 1u);
      if (ok && lane == 0) bar_arrive(BAR(v_empty, st));
      ++v_tile;
    };
    auto skip_q = [&](int h) {
      ok = ok && wait_bar(wc, BAR(q_full, h), (q_par >> h) & 1u);
      if (ok && lane == 0) bar_arrive(BAR(q_empty, h));
      q_par ^= 1u << h;
    };
    while (ok) {
      const uint32_t r = nseg % kDescs;
      ok = wait_bar(wc, BAR(d_full, r), (nseg / kDescs) & 1u);
      if (!ok) break;
      const int tiles = __reduce_max_sync(0xffffffffu, bar.seg[r].t1 - bar.seg[r].t0);
      const int wide = __reduce_max_sync(0xffffffffu, bar.seg[r].wide);
      __syncwarp();
      if (lane == 0) bar_arrive(BAR(d_empty, r));
      if (tiles == 0) break;
      const int i0 = (step + w) & 1;      // the group's first step of the segment
      const int n = wide ? tiles : (tiles + 1 - i0) / 2;
      const int h = wide ? w : nseg & 1;  // its query buffer
      const uint32_t k_end = k_tile + tiles, v_end = v_tile + tiles;
      step += tiles << wide;
      ++nseg;
      const uint64_t qd = desc_q + static_cast<uint32_t>(h * (C::TILE_BYTES / 16));
      auto scores = [&](bool last) {
        const uint32_t st = k_tile % C::STAGES;
        ok = ok && wait_bar(wc, BAR(k_full, st), (k_tile / C::STAGES) & 1u);
        if (!ok) return;
        tc_fence_after();
        const uint64_t kd = desc_k + st * (C::TILE_BYTES / 16);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t at = (k / 4) * (C::BLK / 16) + 2 * (k & 3);
            mma_bf16_ss(t_s, qd + at, kd + at, kIdescQK, k ? 1u : 0u);
          }
          bar_commit(BAR(s_full, w));
          bar_commit(BAR(k_empty, st));
          if (last) bar_commit(BAR(q_empty, h));
        }
        __syncwarp();
        any = true;
        ++k_tile;
      };
      if (n > 0) {
        if (!wide && i0) skip_k();
        ok = ok && wait_bar(wc, BAR(q_full, h), (q_par >> h) & 1u);
        q_par ^= 1u << h;
        scores(n == 1);
      } else {
        skip_q(h);
      }
#pragma unroll 1
      for (int i = 0; ok && i < n; ++i) {
        if (C::APART && i + 1 < n) {  // the next scores, once these are read
          if (!wide) skip_k();
          ok = ok && wait_bar(wc, BAR(s_read, w), p_use & 1u);
          scores(i + 2 == n);
        }
        if (!wide && (i || i0)) skip_v();
        const uint32_t st = v_tile % C::STAGES, v_par = (v_tile / C::STAGES) & 1u;
        const uint32_t p_par = p_use & 1u;
        if (!ok) break;
        if (!all(bar_test(BAR(v_full, st), v_par) & bar_test(BAR(p_lo, w), p_par))) {
          ok = wait_bar(wc, BAR(v_full, st), v_par) && wait_bar(wc, BAR(p_lo, w), p_par);
          if (!ok) break;
        }
        tc_fence_after();
        const uint64_t vd = desc_v + st * (C::TILE_BYTES / 16);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kTile / 32; ++k)
            mma_ts(t_o, t_p + k * 8, vd + k * (16 * 128 / 16), kIdescPV, (i || k) ? 1u : 0u);
        }
        __syncwarp();
        ok = wait_bar(wc, BAR(p_hi, w), p_par);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = kTile / 32; k < kTile / 16; ++k)
            mma_ts(t_o, t_p + k * 8, vd + k * (16 * 128 / 16), kIdescPV, 1u);
          bar_commit(BAR(v_empty, st));
          if (C::APART || i == n - 1) bar_commit(BAR(o_full, w));
        }
        __syncwarp();
        ++p_use;
        ++v_tile;
        if (!C::APART && i + 1 < n) {
          if (!wide) skip_k();
          scores(i + 2 == n);
        }
      }
      if (wide && ok) skip_q(1 - w);
      while (ok && k_tile != k_end) skip_k();
      while (ok && v_tile != v_end) skip_v();
    }
    if (any) {
      if (elect_one()) bar_commit(BAR(drain, w));
      __syncwarp();
      wait_drain(&bar.drain[w], 0, limit);
    }
  } else {
    // ---------------- softmax: group w = warps 4w .. 4w+3, a row per thread ----------------
    const int w = warp >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t ts = tmem_base + lane_base + w * 128;
    const uint32_t tp = tmem_base + lane_base + C::T_P + w * C::T_P_STEP;
    const uint32_t to = tmem_base + lane_base + C::T_O + w * D;
    const float sl2 = a.scale * kLog2e;
    const float lag = score_lag<DTYPE>(sl2);
    const uint64_t sl2x2 = pack_f32x2(sl2, sl2);
    // segments, uses of s_full and o_full, V tiles and steps so far
    uint32_t nseg = 0, s_use = 0, o_use = 0, vc = 0, step = 0;
    bool ok = true;
    while (ok) {
      const uint32_t r = nseg % kDescs;
      ok = wait_bar(wc, BAR(d_full, r), (nseg / kDescs) & 1u);
      if (!ok) break;
      const Segment sg = bar.seg[r];
      __syncwarp();
      if (lane == 0) bar_arrive(BAR(d_empty, r));
      ++nseg;
      const int tiles = sg.t1 - sg.t0;
      if (tiles == 0) break;
      const int first_tok = sg.wide ? w * g.tpt : 0;
      const int live_rows = min(max(sg.ntok - first_tok, 0), g.tpt) * g.G;
      const bool warp_live = quad * 32 < live_rows;
      const int lim = row < live_rows ? min(sg.kv_len, sg.lim0 + first_tok + row / g.G) : 1 << 30;
      const int i0 = (step + w) & 1;  // the group's first step of the segment
      const int steps = sg.wide ? tiles : (tiles + 1 - i0) / 2;
      float m = -INFINITY;
      uint64_t l2 = 0;
      for (int i = 0; i < steps; ++i) {
        const int ti = sg.wide ? i : 2 * i + i0;  // tile of the segment
        const int t = sg.t0 + ti;
        ok = wait_bar(wc, BAR(s_full, w), s_use & 1u);
        if (!ok) break;
        ++s_use;
        tc_fence_after();
        // rows of V past the keys' end may hold anything, and 0 * NaN is not
        // 0: they are cleared in shared memory before the product (by both
        // groups of a wide unit, whose products are not ordered)
        const int valid = sg.kv_len - t * kTile;
        if (rare(valid < kTile)) {
          const uint32_t at = vc + ti;
          ok = wait_bar(wc, BAR(v_full, at % C::STAGES), (at / C::STAGES) & 1u);
          if (!ok) break;
          const uint32_t v0 = smem_u32(smem + C::V_OFF + (at % C::STAGES) * C::TILE_BYTES);
#pragma unroll 1
          for (int c = valid * 8 + row; c < kTile * 8; c += 128)  // 16 bytes each, consecutive
#pragma unroll
            for (int d = 0; d < kBlocks; ++d) st_shared_v4(v0 + d * C::BLK + c * 16, 0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        // APART: the product of the last step must have read its probabilities
        // before these overwrite them (waited for after the first quarter's
        // exponentials: 538 -> 527 us at 256 queries over 131072 rows)
        auto last_product = [&]() {
          if (!C::APART || i == 0) return true;
          ok = wait_bar(wc, BAR(o_full, w), o_use & 1u);
          ++o_use;
          tc_fence_after();
          return ok;
        };
        if (rare(!warp_live)) {
          tc_fence_before();
          __syncwarp();
          if (C::APART && lane == 0) bar_arrive(BAR(s_read, w));
          if (!last_product()) break;
          if (lane == 0) {
            bar_arrive(BAR(p_lo, w));
            bar_arrive(BAR(p_hi, w));
          }
          continue;
        }
        uint32_t v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(ts + c * 32, v[c]);
        const int vis = lim - t * kTile;  // keys of the tile the row sees
        const bool masked = __any_sync(0xffffffffu, vis < kTile);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_regs_fence(v[c]);
        if (C::APART) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(BAR(s_read, w));
        }
        if (rare(masked)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c * 32 + j >= vis) v[c][j] = 0xff800000u;  // -inf
        }
        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // four chains
#pragma unroll
        for (int j = 0; j < 32; j += 2)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float x = __uint_as_float(v[c][j]), y = __uint_as_float(v[c][j + 1]);
            asm("max.f32 %0, %0, %1, %2;" : "+f"(tops[c]) : "f"(x), "f"(y));
          }
        const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        const bool moves = top - m > lag;
        bool waited = false;
        if (rare(__any_sync(0xffffffffu, moves))) {
          if (!last_product()) break;
          waited = true;
          const float m1 = moves ? in_range<DTYPE>(top, sl2) : m;
          const float f = moves ? rescale<DTYPE>(m, m1, sl2) : 1.0f;
          m = m1;
          const float2 lv = unpack_f32x2(l2);
          l2 = pack_f32x2(lv.x * f, lv.y * f);
          if (i > 0) {
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld_32x32b_x16(to + c * 16, o);
              tmem_ld_wait();
              tmem_regs_fence16(o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st_32x32b_x16(to + c * 16, o);
            }
          }
        }
        const float c0 = prob_offset<DTYPE>(m, sl2);
        const uint64_t c0x2 = pack_f32x2(c0, c0);
        uint64_t sums[4] = {l2, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint64_t x = fma_f32x2(
                pack_f32x2(__uint_as_float(v[c][2 * j]), __uint_as_float(v[c][2 * j + 1])), sl2x2,
                c0x2);
            float2 e = unpack_f32x2(x);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            sums[j & 3] = add_f32x2(sums[j & 3], pack_f32x2(e.x, e.y));
            p[j] = pack2<DTYPE>(e.x, e.y);
          }
          if (C::APART && c == 0 && !waited && !last_product()) break;
          tmem_st_32x32b_x16(tp + c * 16, p);
          if (c == 1 || c == 3) {  // the MMA issuer starts on the first half
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(c == 1 ? BAR(p_lo, w) : BAR(p_hi, w));
          }
        }
        if (!ok) break;
        l2 = add_f32x2(add_f32x2(sums[0], sums[1]), add_f32x2(sums[2], sums[3]));
      }
      if (!ok) break;
      vc += tiles;
      step += tiles << sg.wide;
      const int64_t at = sg.slot + static_cast<int64_t>(w) * sg.rows + row;
      const bool mine = row < live_rows;
      if (steps == 0) {  // a single tile: the other group's
        if (mine) g.part_lse[at] = -INFINITY;
        continue;
      }
      ok = wait_bar(wc, BAR(o_full, w), o_use & 1u);
      if (!ok) break;
      ++o_use;
      tc_fence_after();
      if (warp_live) {
        const float2 lv = unpack_f32x2(l2);
        const PartEnd end = end_part<DTYPE>(m, lv.x + lv.y, sl2);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(to + c * 32, o);
          tmem_ld_wait();
          tmem_regs_fence(o);
          if (mine) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t x[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                x[e] = __float_as_uint(__uint_as_float(o[8 * j + e]) * end.inv);
              st_global_v8(g.part_o + at * D + c * 32 + j * 8, x);
            }
          }
        }
        if (mine) g.part_lse[at] = end.lse;  // in powers of two
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem_base, 512);
#undef BAR
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn attn_encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 16-bit elements, box 64 x b1 (x b2), 128-byte swizzle; dims past the second
// are absent when n2 is 0
bool attn_tmap(CUtensorMap *map, int dtype, const void *base, uint64_t n0, uint64_t n1, uint64_t s1,
               uint32_t b1, uint64_t n2 = 0, uint64_t s2 = 0, uint32_t b2 = 1) {
  EncodeTiledFn fn = attn_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {n0, n1, n2 ? n2 : 1};
  const cuuint64_t strides[2] = {s1, s2};
  const cuuint32_t box[3] = {64, b1, b2};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map,
            dtype == MOE_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
            n2 ? 3 : 2, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DTYPE, int D>
cudaError_t run(const AttnArgs &g, int ctas, cudaStream_t s) {
  using C = AttnCfg<D>;
  const PrefixAttnArgs &a = g.a;
  CUtensorMap tmK, tmV, tmQp, tmQs;
  const uint64_t rows = (static_cast<uint64_t>(a.num_pages) * a.hkv) << a.page_shift;
  const uint32_t page_rows = std::min(1 << a.page_shift, kTile);
  if (!attn_tmap(&tmK, DTYPE, a.k_cache, D, rows, D * 2, page_rows) ||
      !attn_tmap(&tmV, DTYPE, a.v_cache, D, rows, D * 2, page_rows) ||
      !attn_tmap(&tmQp, DTYPE, a.q, D, a.hq, D * 2, g.G, a.T, a.q_stride * 2,
                 std::max(g.p_box, 1)) ||
      !attn_tmap(&tmQs, DTYPE, a.q, D, a.hq, D * 2, g.G, a.T, a.q_stride * 2,
                 std::max(g.s_box, 1)))
    return cudaErrorInvalidValue;
  const cudaError_t err =
      cudaFuncSetAttribute(attention_tiles_kernel<DTYPE, D>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (err != cudaSuccess) return err;
  MOE_LAUNCH_PDL(attention_tiles_kernel<DTYPE, D>, ctas, kAttnThreads, C::SMEM_BYTES, s, tmK, tmV,
                 tmQp, tmQs, g);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_tiles(const AttnArgs &g, int dtype, int ctas, cudaStream_t s) {
  if (dtype == MOE_DTYPE_BF16)
    return g.a.D == 64 ? run<MOE_DTYPE_BF16, 64>(g, ctas, s)
                       : run<MOE_DTYPE_BF16, 128>(g, ctas, s);
  return g.a.D == 64 ? run<MOE_DTYPE_FP16, 64>(g, ctas, s)
                     : run<MOE_DTYPE_FP16, 128>(g, ctas, s);
}

}  // namespace moe
