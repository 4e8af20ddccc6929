// prefix_attention.cu -- attention of a batch that shares a long prefix
// (moe_prefix_attention).
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q.k_j)
// over the prefix's rows and then the sequence's own up to the token's causal
// limit.  The sum over j splits anywhere: a part keeps its o normalised and
// lse = ln sum p, and parts join with weights exp(lse - max lse).
//
// Work.  The query heads of one key head and several tokens fill the 128 rows
// of a tensor-core tile (row = token * G + head in group), so a unit is
//   prefix: a block of tokens of the whole batch x a key head x the prefix
//           (its keys and values are read once per block, not per sequence);
//   own:    a block of one sequence's tokens x a key head x its own rows,
// cut along the keys into tiles of 128.  All tiles of all units stand in one
// line, weighted by their time, and every SM takes an equal piece of it
// (stretches of several units or a part of one), so the load is even whatever
// the lengths, which only the device knows.  A unit's stretch on an SM is a
// segment and leaves one partial result; a second kernel joins them.
//
// A CTA's two groups of 128 softmax threads each own a 128 x 128 score tile
// and an output accumulator in TMEM.  A wide unit (more than 128 rows) gives
// each group 128 of its rows and both read the same K and V tiles; a narrow
// one gives both the same rows and every second tile.  The groups take turns
// through all segments, so while one ends a short unit the other is at the
// next.
//
// Bounds: with many rows the tensor cores (4 D flop per score; the two MMAs
// of one group run while the other group takes exponentials), with few the
// cache's bytes.
#include <algorithm>
#include <cstddef>
#include <mutex>

#include "elem.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kTile = 128;         // keys per tile
constexpr int kAttnThreads = 320;  // 8 softmax warps, the loader, the MMA issuer
constexpr int kDescs = 4;          // segments the loader may be ahead
constexpr int kMaxCtas = 160;      // grid limit (slots of partial results)
// time of a tile in the line, and of starting a unit
constexpr int kWideCost = 3, kNarrowCost = 2, kUnitCost = 1;

template <int D>
struct AttnCfg {
  static constexpr int BLK = kTile * 128;           // 128 rows x 64 elements
  static constexpr int TILE_BYTES = (D / 64) * BLK;  // a K, V or Q tile
  static constexpr int STAGES = D == 128 ? 2 : 4;
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

// What the joining kernel needs of a sequence.
struct SeqMeta {
  int64_t cum;   // where its units start in the line
  int32_t unit;  // number of its first unit among the own units
  int32_t tiles;
};

struct AttnArgs {
  PrefixAttnArgs a;
  int G, tpt;                 // heads per key head, tokens per 128 rows
  int p_wide, p_tok, p_blocks, p_tiles, p_rows, p_box;
  int s_wide, s_tok, s_rows, s_box;
  int64_t p_cost, p_total;    // of a prefix unit, of all
  int64_t s_slot0;            // first row of the own units' slots
  int64_t *piece;  // the length of a piece
  SeqMeta *meta;
  float *part_o, *part_lse;
};

// ---------------------------------------------------------------------------
// the plan
// ---------------------------------------------------------------------------

struct Seq {
  int q0, nq, len, tiles, units;
  int64_t cost;  // of all its units
};

// Sequence b with every value clamped into the buffers.
__device__ __forceinline__ Seq read_seq(const AttnArgs &g, int b, bool *bad_off, bool *bad) {
  const PrefixAttnArgs &a = g.a;
  Seq s = {0, 0, 0, 0, 0, 0};
  if (b >= a.B) return s;
  s.q0 = b;
  s.nq = 1;
  if (a.q_offsets) {
    const int q0 = a.q_offsets[b], q1 = a.q_offsets[b + 1];
    if (q0 < 0 || q1 < q0 || q1 > a.T) *bad_off = true;
    s.q0 = min(max(q0, 0), a.T);
    s.nq = max(min(q1, a.T), s.q0) - s.q0;
    if (s.nq > a.max_q) *bad = true;
    s.nq = min(s.nq, a.max_q);
  }
  const int cap = a.max_pages << a.page_shift;
  const int len = a.kv_lens[b];
  if (len < 0 || len > cap) *bad = true;
  s.len = min(max(len, 0), cap);
  s.tiles = (s.len + kTile - 1) / kTile;
  s.units = (s.nq + g.s_tok - 1) / g.s_tok * a.hkv;
  s.cost = s.tiles > 0 ? static_cast<int64_t>(s.units) *
                             (s.tiles * (g.s_wide ? kWideCost : kNarrowCost) + kUnitCost)
                       : 0;
  return s;
}

// The line is cut into pieces of one length, at least the longest tile's.
// 64-bit divisions are kept out of line: they are long code.
__device__ __noinline__ int64_t div64(int64_t n, int64_t d) { return n / d; }
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d) {
  if (n < (int64_t{1} << 31) && d < (int64_t{1} << 31))
    return static_cast<uint32_t>(n) / static_cast<uint32_t>(d);
  return div64(n, d);
}
__device__ __forceinline__ int64_t piece_length(int64_t total, int ctas) {
  return max(quotient(total + ctas - 1, ctas), static_cast<int64_t>(kWideCost));
}

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
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
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
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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
// The bounded wait, out of line: its code is long, and it reads the global
// timer, which takes about a microsecond.
__device__ __noinline__ bool wait_long(uint64_t *bar, uint32_t parity, volatile int *abort,
                                       uint32_t *status, uint64_t limit_ns) {
  return mbar_wait_bounded(bar, parity, abort, status, limit_ns);
}
// What a wait needs when it becomes long.
struct WaitCtx {
  uint32_t base;  // shared address of the barriers
  uint64_t *bars;
  volatile int *abort;
  uint32_t *status;
  uint64_t limit_ns;
};
// Whole warp: true for all lanes when the phase completed, false for all when
// some lane gave up.
__device__ __forceinline__ bool wait_bar(const WaitCtx &c, uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < 2048; ++i)
    if (__all_sync(0xffffffffu, bar_test(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_long(c.bars + (bar - c.base) / 8, parity, c.abort, c.status,
                                           c.limit_ns));
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
  uint64_t p_lo[2], p_hi[2];  // its probabilities are: keys 0-63, 64-127
  uint64_t o_full[2];  // its segment's accumulator is complete
  uint64_t d_full[kDescs], d_empty[kDescs];
  uint64_t drain[1];
  Segment seg[kDescs];
  int64_t start_cum;
  int start_seq, start_unit;
  int64_t warp_cost[kAttnThreads / 32];
  int warp_units[kAttnThreads / 32];
  uint32_t tmem;
  int abort;
};

template <int DTYPE, int D>
__global__ void __launch_bounds__(kAttnThreads, 1)
    prefix_attention_kernel(const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV,
                            const __grid_constant__ CUtensorMap tmQp,
                            const __grid_constant__ CUtensorMap tmQs, const AttnArgs g) {
  pdl_begin();
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
  const uint64_t limit = a.wait_limit_ns;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = smem_u32(&bar);
#define BAR(field, i) (bars + static_cast<uint32_t>(offsetof(B, field)) + 8u * (i))
  const WaitCtx wc = {bars, reinterpret_cast<uint64_t *>(&bar), abort_flag, a.status, limit};

  // ---- where this CTA's piece of the line lies (every CTA by itself) ----
  const int per = (a.B + kAttnThreads - 1) / kAttnThreads;
  const int b_lo = threadIdx.x * per, b_hi = min(b_lo + per, a.B);
  int64_t my_cost = 0;
  int my_units = 0;
  bool bad_off = false, bad = false;
  for (int b = b_lo; b < b_hi; ++b) {
    const Seq s = read_seq(g, b, &bad_off, &bad);
    my_cost += s.cost;
    my_units += s.units;
  }
  int64_t cost = my_cost;
  int units = my_units;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t c = __shfl_up_sync(0xffffffffu, cost, off);
    const int u = __shfl_up_sync(0xffffffffu, units, off);
    if (lane >= off) {
      cost += c;
      units += u;
    }
  }
  if (lane == 31) {
    bar.warp_cost[warp] = cost;
    bar.warp_units[warp] = units;
  }
  if (threadIdx.x == 0) {
    bar.abort = 0;
    bar.start_seq = a.B;
    bar.start_unit = 0;
    bar.start_cum = 0;
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&bar.k_full[s], 1);
      mbar_init(&bar.k_empty[s], 1);
      mbar_init(&bar.v_full[s], 1);
      mbar_init(&bar.v_empty[s], 1);
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&bar.q_full[h], 1);
      mbar_init(&bar.q_empty[h], 1);
      mbar_init(&bar.s_full[h], 1);
      mbar_init(&bar.p_lo[h], 4);
      mbar_init(&bar.p_hi[h], 4);
      mbar_init(&bar.o_full[h], 1);
    }
    for (int i = 0; i < kDescs; ++i) {
      mbar_init(&bar.d_full[i], 1);
      mbar_init(&bar.d_empty[i], 9);
    }
    mbar_init(&bar.drain[0], 1);
    fence_mbar_init();
  }
  // offsets that are no partition of the tokens: the own rows are left out
  const bool drop = __syncthreads_or(bad_off);
  int64_t before = 0, own_total = 0;
  int units_before = 0;
  for (int w = 0; w < kAttnThreads / 32; ++w) {
    if (w < warp) {
      before += bar.warp_cost[w];
      units_before += bar.warp_units[w];
    }
    own_total += bar.warp_cost[w];
  }
  before += cost - my_cost;
  units_before += units - my_units;
  if (drop) own_total = 0;
  const int64_t total = g.p_total + own_total;
  const int64_t piece = piece_length(total, gridDim.x);
  const int64_t lo = blockIdx.x * piece, hi = min(lo + piece, total);
  const bool idle = lo >= total;
  if (blockIdx.x == 0 || !idle) {
    const int64_t from = max(lo - g.p_total, int64_t{0});
    int64_t cum = before;
    int unit = units_before;
    for (int b = b_lo; b < b_hi; ++b) {
      const Seq s = read_seq(g, b, &bad_off, &bad);
      if (blockIdx.x == 0) g.meta[b] = SeqMeta{cum, unit, drop ? 0 : s.tiles};
      if (!drop && cum <= from && from < cum + s.cost) {
        bar.start_seq = b;
        bar.start_cum = cum;
        bar.start_unit = unit;
      }
      cum += s.cost;
      unit += s.units;
    }
    if (blockIdx.x == 0) {
      if (bad || bad_off) set_status(a.status, kStatusBadId);
      if (threadIdx.x == 0) *g.piece = piece;
    }
  }
  if (idle) return;  // uniform across the CTA
  if (warp == 9) tmem_alloc(&bar.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = bar.tmem;

  if (warp == 8) {
    // ---------------- loader: walks the line, fetches Q, K and V ----------------
    const int ppt = max(1, kTile >> a.page_shift);  // pages per tile
    const int page_rows = min(1 << a.page_shift, kTile);
    uint32_t issued[2] = {0, 0}, nseg = 0, q_use[2] = {0, 0};  // issued: K and V tiles
    bool ok = true;
    // tiles [t0, t1) of a unit that starts at `start` in the line with n tiles
    // of the given width; false: none of them here
    int t0, t1;
    auto tile_at = [&](int64_t ahead, int n, int wide) {  // first tile at or past `ahead`
      if (ahead <= 0) return 0;
      if (ahead >= static_cast<int64_t>(n) * (wide ? kWideCost : kNarrowCost)) return n;
      const int x = static_cast<int>(ahead);
      return wide ? (x + kWideCost - 1) / kWideCost : (x + kNarrowCost - 1) / kNarrowCost;
    };
    auto cut = [&](int64_t start, int n, int wide) {
      t0 = tile_at(lo - start, n, wide);
      t1 = tile_at(hi - start, n, wide);
      return t0 < t1;
    };
    // the prefix units of this piece, then its sequences, 32 at a time (one
    // per lane; `todo`: those with work here), each with its units
    int64_t u = lo < g.p_total ? quotient(lo, g.p_cost) : 0;
    bool own = lo >= g.p_total;
    int base = bar.start_seq - 32, seq = 0;
    int64_t cum0 = g.p_total + bar.start_cum, cum = 0, start = 0, unit_cost = 1;
    int unit0 = bar.start_unit, un = 0, batch_units = 0;
    int64_t batch = 0;
    unsigned todo = 0;
    Seq s = {0, 0, 0, 0, 0, 0};
    int j = 0, n_units = 0, q0 = 0, nq = 0, len = 0, tiles = 0, unit = 0;
    while (ok) {
      int head, tok0, ntok, lim0, kv_len, wide;
      int64_t slot;
      const int32_t *pages;
      if (!own) {
        if (u * g.p_cost >= min(hi, g.p_total)) {
          own = true;
          continue;
        }
        const int64_t at = u++;
        if (!cut(at * g.p_cost, g.p_tiles, g.p_wide)) continue;
        head = static_cast<int>(quotient(at, g.p_blocks));
        tok0 = static_cast<int>(at - static_cast<int64_t>(head) * g.p_blocks) * g.p_tok;
        ntok = min(g.p_tok, a.T - tok0);
        lim0 = kv_len = a.prefix_len;
        wide = g.p_wide;
        slot = (at + blockIdx.x) * 2 * g.p_rows;
        pages = a.prefix_pages;
      } else if (j < n_units && start + j * unit_cost < hi) {
        const int at = j++;
        if (!cut(start + at * unit_cost, tiles, g.s_wide)) continue;
        const int block = at / a.hkv;
        head = at - block * a.hkv;
        const int i0 = block * g.s_tok;
        tok0 = q0 + i0;
        ntok = min(g.s_tok, nq - i0);
        lim0 = len - nq + i0 + 1;
        kv_len = len;
        wide = g.s_wide;
        slot = g.s_slot0 + (static_cast<int64_t>(unit + at) + blockIdx.x) * 2 * g.s_rows;
        pages = a.page_table + static_cast<int64_t>(seq) * a.max_pages;
      } else if (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        seq = base + src;
        q0 = __shfl_sync(0xffffffffu, s.q0, src);
        nq = __shfl_sync(0xffffffffu, s.nq, src);
        len = __shfl_sync(0xffffffffu, s.len, src);
        tiles = __shfl_sync(0xffffffffu, s.tiles, src);
        n_units = __shfl_sync(0xffffffffu, s.units, src);
        start = __shfl_sync(0xffffffffu, cum, src);
        unit = __shfl_sync(0xffffffffu, un, src);
        unit_cost = static_cast<int64_t>(tiles) * (g.s_wide ? kWideCost : kNarrowCost) + kUnitCost;
        j = lo <= start ? 0 : static_cast<int>(quotient(lo - start, unit_cost));
        continue;
      } else {
        base += 32;
        cum0 += batch;
        unit0 += batch_units;
        if (base >= a.B || cum0 >= hi) break;
        s = read_seq(g, base + lane, &bad_off, &bad);
        cum = s.cost;
        un = s.units;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int64_t c = __shfl_up_sync(0xffffffffu, cum, off);
          const int v = __shfl_up_sync(0xffffffffu, un, off);
          if (lane >= off) {
            cum += c;
            un += v;
          }
        }
        batch = __shfl_sync(0xffffffffu, cum, 31);
        batch_units = __shfl_sync(0xffffffffu, un, 31);
        cum += cum0 - s.cost;
        un += unit0 - s.units;
        todo = __ballot_sync(0xffffffffu, s.cost > 0 && cum < hi && cum + s.cost > lo);
        continue;
      }
      // publish the segment, then fetch its queries and tiles
      const uint32_t r = nseg % kDescs;
      ok = wait_bar(wc, BAR(d_empty, r), ((nseg / kDescs) & 1u) ^ 1u);
      if (!ok) break;
      const int h0 = wide ? 0 : nseg & 1;  // a narrow unit's rows alternate between the buffers
      if (lane == 0) {
        bar.seg[r] = Segment{t0, t1, kv_len, wide, ntok, lim0, own ? g.s_rows : g.p_rows, slot};
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
          const int box = own ? g.s_box : g.p_box;
          mbar_arrive_expect_tx(&bar.q_full[h], static_cast<uint32_t>(box * g.G * 128 * kBlocks));
          for (int d = 0; d < kBlocks; ++d)
            tma_load_3d(smem + h * C::TILE_BYTES + d * C::BLK, own ? &tmQs : &tmQp, &bar.q_full[h],
                        d * 64, head * g.G, tok0 + (wide ? h * g.tpt : 0));
        }
      }
      if (!ok) break;
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
      int page = page_at(t0);
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
  } else if (warp == 9) {
    // ---------------- MMA issuer ----------------
    // Steps are numbered through all segments; step n belongs to group n & 1.
    // Scores run up to two steps ahead of products with V: scores(n + 2)
    // overwrite the probabilities of step n, so they follow product(n) (MMAs
    // complete in issue order).  Issuing takes as long as computing (64 cycles
    // for 128 x 128 x 16) except for the last four, the depth of the queue in
    // front of the tensor cores, so what lies between two batches must stay
    // below 256 cycles.  The whole warp walks the steps, so that operands stay
    // warp-uniform, and one elected lane issues.
    constexpr uint32_t kIdescQK = attn_idesc<DTYPE>(128, kTile, false);
    constexpr uint32_t kIdescPV = attn_idesc<DTYPE>(128, D, true);
    const uint64_t desc_q = sw128_kmajor_desc(smem_u32(smem));
    const uint64_t desc_k = sw128_kmajor_desc(smem_u32(smem + C::K_OFF));
    const uint64_t desc_v = sw128_nmajor_desc(smem_u32(smem + C::V_OFF), C::BLK);
    // cursors of the scores and of the products: steps done, segments opened,
    // tiles done, steps left in the segment, step in the segment, its width
    uint32_t s_n = 0, s_seg = 0, s_tile = 0, o_n = 0, o_seg = 0, o_tile = 0;
    int s_left = 0, s_i = 0, s_wide = 0, o_left = 0, o_i = 0, o_wide = 0;
    uint32_t q_par = 0, p_par = 0;  // a bit per buffer / group
    bool end = false;
    auto all = [](bool x) { return __all_sync(0xffffffffu, x) != 0; };
    while (true) {
      // ---- the next scores, if everything is there (or nothing else can be done)
      if (s_n < o_n + 2 && !end) {
        const bool alone = s_n == o_n;
        bool have = s_left > 0;
        if (rare(!have)) {
          const uint32_t r = s_seg % kDescs, par = (s_seg / kDescs) & 1u;
          have = all(bar_test(BAR(d_full, r), par));
          if (rare(!have && alone)) {
            have = wait_bar(wc, BAR(d_full, r), par);
            if (!have) break;
          }
          if (have) {
            const int tiles = __reduce_max_sync(0xffffffffu, bar.seg[r].t1 - bar.seg[r].t0);
            s_wide = __reduce_max_sync(0xffffffffu, bar.seg[r].wide);
            s_left = tiles << s_wide;
            s_i = 0;
            ++s_seg;
            end = tiles == 0;
            if (end) continue;
          }
        }
        if (have) {
          const int w = s_n & 1, h = s_wide ? w : (s_seg - 1) & 1;
          const bool first_q = s_i <= s_wide;
          const uint32_t stage = s_tile % C::STAGES, k_par = (s_tile / C::STAGES) & 1u;
          bool there = all(bar_test(BAR(k_full, stage), k_par) &
                           bar_test(BAR(q_full, h), first_q ? (q_par >> h) & 1u : ~(q_par >> h) & 1u));
          if (rare(!there && alone)) {
            there = wait_bar(wc, BAR(k_full, stage), k_par) &&
                    (!first_q ||
                     wait_bar(wc, BAR(q_full, h), (q_par >> h) & 1u));
            if (!there) break;
          }
          if (there) {
            tc_fence_after();
            const uint64_t qd = desc_q + static_cast<uint32_t>(h * (C::TILE_BYTES / 16));
            const uint64_t kd = desc_k + stage * (C::TILE_BYTES / 16);
            const bool last_k = !s_wide || (s_i & 1);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint32_t at = (k / 4) * (C::BLK / 16) + 2 * (k & 3);
                mma_bf16_ss(tmem_base + w * 128, qd + at, kd + at, kIdescQK, k ? 1u : 0u);
              }
              bar_commit(BAR(s_full, w));
              if (last_k) bar_commit(BAR(k_empty, stage));
              if (s_left <= 1 + s_wide) bar_commit(BAR(q_empty, h));
            }
            __syncwarp();
            if (first_q) q_par ^= 1u << h;
            s_tile += last_k;
            ++s_i;
            --s_left;
            ++s_n;
            continue;
          }
        }
      }
      if (rare(s_n == o_n)) break;  // the end
      // ---- the next product; its first half of keys may be ready early
      if (rare(o_left == 0)) {  // its segment was opened by the scores
        const uint32_t r = o_seg % kDescs;
        const int tiles = __reduce_max_sync(0xffffffffu, bar.seg[r].t1 - bar.seg[r].t0);
        o_wide = __reduce_max_sync(0xffffffffu, bar.seg[r].wide);
        __syncwarp();
        if (lane == 0) bar_arrive(BAR(d_empty, r));
        o_left = tiles << o_wide;
        o_i = 0;
        ++o_seg;
      }
      const int w = o_n & 1;
      const uint32_t stage = o_tile % C::STAGES, v_par = (o_tile / C::STAGES) & 1u;
      const uint32_t par = (p_par >> w) & 1u;
      const uint64_t vd = desc_v + stage * (C::TILE_BYTES / 16);
      const uint32_t t_p = tmem_base + w * 128, t_o = tmem_base + 256 + w * 128;
      if (rare(!all(bar_test(BAR(v_full, stage), v_par) & bar_test(BAR(p_lo, w), par)))) {
        if (!wait_bar(wc, BAR(v_full, stage), v_par) ||
            !wait_bar(wc, BAR(p_lo, w), par))
          break;
      }
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kTile / 32; ++k)
          mma_ts(t_o, t_p + k * 8, vd + k * (16 * 128 / 16), kIdescPV, (o_i >= 2 || k) ? 1u : 0u);
      }
      __syncwarp();
      if (!wait_bar(wc, BAR(p_hi, w), par)) break;
      tc_fence_after();
      const bool last_v = !o_wide || (o_i & 1);
      if (elect_one()) {
#pragma unroll
        for (int k = kTile / 32; k < kTile / 16; ++k)
          mma_ts(t_o, t_p + k * 8, vd + k * (16 * 128 / 16), kIdescPV, 1u);
        if (last_v) bar_commit(BAR(v_empty, stage));
        if (o_left <= 2) bar_commit(BAR(o_full, w));
      }
      __syncwarp();
      p_par ^= 1u << w;
      o_tile += last_v;
      ++o_i;
      --o_left;
      ++o_n;
    }
    if (s_n > 0) {
      if (elect_one()) bar_commit(BAR(drain, 0));
      __syncwarp();
      wait_drain(&bar.drain[0], 0, limit);
    }
  } else {
    // ---------------- softmax: group w = warps 4w .. 4w+3, a row per thread ----------------
    const int w = warp >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t ts = tmem_base + lane_base + w * 128, to = tmem_base + lane_base + 256 + w * 128;
    // p = 2^(s * sl2 - m * sl2 + off): fp16 probabilities are kept 2^10 up,
    // away from its subnormals; the running maximum may lag by kLag powers
    // of two before the accumulator is rescaled, so p stays below 2^15 (fp16
    // holds 65504) or 2^8 (bf16).
    constexpr float kOff = DTYPE == MOE_DTYPE_FP16 ? 10.0f : 0.0f;
    constexpr float kLag = DTYPE == MOE_DTYPE_FP16 ? 5.0f : 8.0f;
    const float sl2 = a.scale * 1.4426950408889634f;
    const float lag = kLag / sl2;
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
        // 0: they are cleared in shared memory before the product (in a wide
        // unit by the group whose product comes first)
        const int valid = sg.kv_len - t * kTile;
        if (rare(valid < kTile && (!sg.wide || i0 == 0))) {
          const uint32_t at = vc + ti;
          ok = wait_bar(wc, BAR(v_full, at % C::STAGES), (at / C::STAGES) & 1u);
          if (!ok) break;
          if (row >= valid) {
#pragma unroll 1
            for (int q = 0; q < 8 * kBlocks; ++q)
              st_shared_v4(smem_u32(smem + C::V_OFF + (at % C::STAGES) * C::TILE_BYTES +
                                    (q >> 3) * C::BLK + row * 128 + (q & 7) * 16),
                           0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (rare(!warp_live)) {
          tc_fence_before();
          __syncwarp();
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
        const bool moves = top > m + lag;
        if (rare(__any_sync(0xffffffffu, moves))) {
          const float m1 = moves ? top : m;
          // 0 where the row has seen nothing yet
          const float f = moves ? ex2((m - m1) * sl2) : 1.0f;
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
        const float c0 = m == -INFINITY ? kOff : kOff - m * sl2;
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
          tmem_st_32x32b_x16(ts + c * 16, p);
          if (c == 1 || c == 3) {  // the MMA issuer starts on the first half
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(c == 1 ? BAR(p_lo, w) : BAR(p_hi, w));
          }
        }
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
        const float l = lv.x + lv.y;
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
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
                x[e] = __float_as_uint(__uint_as_float(o[8 * j + e]) * inv);
              st_global_v8(g.part_o + at * D + c * 32 + j * 8, x);
            }
          }
        }
        // in powers of two
        if (mine) g.part_lse[at] = l > 0.0f ? m * sl2 - kOff + log2f(l) : -INFINITY;
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
// joining the parts: a warp per token and query head
// ---------------------------------------------------------------------------

template <int DTYPE, int D>
__global__ void __launch_bounds__(256) prefix_attention_join_kernel(const AttnArgs g, int planned) {
  pdl_begin();
  constexpr int E = D / 32;
  const PrefixAttnArgs &a = g.a;
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  const int64_t piece = planned ? *g.piece : 1;
  // the token's sequence: how many end at or before it
  int b = t;
  if (a.q_offsets) {
    __shared__ int s_ends[8];
    int n = 0;
    for (int i = threadIdx.x; i < a.B; i += blockDim.x) n += a.q_offsets[i + 1] <= t;
#pragma unroll
    for (int off = 16; off; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
    if (lane == 0) s_ends[threadIdx.x >> 5] = n;
    __syncthreads();
    b = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) b += s_ends[w];
  }
  int tiles = 0, place = 0, unit = 0;
  int64_t cum = 0;
  if (b < a.B && planned) {
    const SeqMeta m = g.meta[b];
    const int q0 = a.q_offsets ? a.q_offsets[b] : b;
    place = t - q0;
    if (place >= 0 && place < a.max_q) tiles = m.tiles;
    cum = m.cum;
    unit = m.unit;
  }
  const int h = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (h < a.hq) {
    const int kvh = h / g.G, hg = h - kvh * g.G;
    // parts: `n` of them `step` rows apart from row `first`, of two kinds
    int64_t first[2] = {0, 0};
    int n[2] = {0, 0}, step[2] = {1, 1};
    if (g.p_tiles > 0) {
      const int block = t / g.p_tok, in = t - block * g.p_tok;
      const int64_t u = static_cast<int64_t>(kvh) * g.p_blocks + block;
      const int64_t start = u * g.p_cost;
      const int c0 = static_cast<int>(quotient(start, piece));
      const int c1 = static_cast<int>(
          quotient(start + static_cast<int64_t>(g.p_tiles - 1) *
                               (g.p_wide ? kWideCost : kNarrowCost),
                   piece));
      first[0] = (u + c0) * 2 * g.p_rows + (g.p_wide ? in / g.tpt * g.p_rows : 0) +
                 in % g.tpt * g.G + hg;
      n[0] = g.p_wide ? c1 - c0 + 1 : 2 * (c1 - c0 + 1);
      step[0] = g.p_wide ? 2 * g.p_rows : g.p_rows;
    }
    if (tiles > 0) {
      const int w = g.s_wide ? kWideCost : kNarrowCost;
      const int block = place / g.s_tok, in = place - block * g.s_tok;
      const int j = block * a.hkv + kvh;
      const int64_t start =
          g.p_total + cum + j * (static_cast<int64_t>(tiles) * w + kUnitCost);
      const int c0 = static_cast<int>(quotient(start, piece));
      const int c1 =
          static_cast<int>(quotient(start + static_cast<int64_t>(tiles - 1) * w, piece));
      first[1] = g.s_slot0 + (static_cast<int64_t>(unit + j) + c0) * 2 * g.s_rows +
                 (g.s_wide ? in / g.tpt * g.s_rows : 0) + in % g.tpt * g.G + hg;
      n[1] = g.s_wide ? c1 - c0 + 1 : 2 * (c1 - c0 + 1);
      step[1] = g.s_wide ? 2 * g.s_rows : g.s_rows;
    }
    const int parts = n[0] + n[1];
    auto row_of = [&](int i) {
      return i < n[0] ? first[0] + static_cast<int64_t>(i) * step[0]
                      : first[1] + static_cast<int64_t>(i - n[0]) * step[1];
    };
    float top = -INFINITY;
    for (int i = lane; i < parts; i += 32) top = fmaxf(top, g.part_lse[row_of(i)]);
#pragma unroll
    for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float ref = top == -INFINITY ? 0.0f : top;
    float o[E], l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
    for (int base = 0; base < parts; base += 32) {
      const int i = base + lane;
      const float wgt = i < parts ? ex2(g.part_lse[row_of(i)] - ref) : 0.0f;
      const int m = min(32, parts - base);
#pragma unroll 4
      for (int k = 0; k < m; ++k) {
        const float wk = __shfl_sync(0xffffffffu, wgt, k);
        l += wk;
        if (wk == 0.0f) continue;  // an empty part has no row
        const float *src = g.part_o + row_of(base + k) * D + lane * E;
        if (E == 4) {
          const float4 x = *reinterpret_cast<const float4 *>(src);
          o[0] = fmaf(wk, x.x, o[0]);
          o[1] = fmaf(wk, x.y, o[1]);
          o[E - 2] = fmaf(wk, x.z, o[E - 2]);
          o[E - 1] = fmaf(wk, x.w, o[E - 1]);
        } else {
          const float2 x = *reinterpret_cast<const float2 *>(src);
          o[0] = fmaf(wk, x.x, o[0]);
          o[1] = fmaf(wk, x.y, o[1]);
        }
      }
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.o) + t * a.o_stride +
                                                 h * D) +
                    lane * (E / 2);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = pack2<DTYPE>(o[e] * inv, o[e + 1] * inv);
    if (a.lse && lane == 0)
      a.lse[static_cast<int64_t>(t) * a.hq + h] =
          l > 0.0f ? (ref + log2f(l)) * 0.6931471805599453f : -INFINITY;
  }
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

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

struct Scratch {
  size_t head, meta, lse, o, bytes;
};

// The shape half of the plan (everything the host knows) and the scratch it
// needs.  Slots: a segment's number is its unit's number + its CTA's, which
// grows along the line, so `units + kMaxCtas` numbers are enough.
Scratch plan(AttnArgs &g, int T, int B, int max_q, int hq, int hkv, int D, int prefix_len) {
  g.G = hq / hkv;
  g.tpt = kTile / g.G;
  g.p_wide = T > g.tpt;
  g.p_tok = g.p_wide ? 2 * g.tpt : g.tpt;
  g.p_blocks = (T + g.p_tok - 1) / g.p_tok;
  g.p_tiles = static_cast<int>((static_cast<int64_t>(prefix_len) + kTile - 1) / kTile);
  g.p_box = std::min(g.tpt, std::max(T, 1));
  g.p_rows = g.p_box * g.G;
  g.s_wide = max_q > g.tpt;
  g.s_tok = g.s_wide ? 2 * g.tpt : g.tpt;
  g.s_box = std::min(std::min(g.tpt, max_q), std::max(T, 1));
  g.s_rows = g.s_box * g.G;
  g.p_cost = static_cast<int64_t>(g.p_tiles) * (g.p_wide ? kWideCost : kNarrowCost) + kUnitCost;
  const int64_t p_units = g.p_tiles ? static_cast<int64_t>(hkv) * g.p_blocks : 0;
  g.p_total = p_units * g.p_cost;
  const int64_t s_units = static_cast<int64_t>(hkv) * (B + T / g.s_tok);
  const int64_t p_slots = p_units ? p_units + kMaxCtas : 0;
  g.s_slot0 = p_slots * 2 * g.p_rows;
  const int64_t rows = g.s_slot0 + (s_units + kMaxCtas) * 2 * g.s_rows;
  Scratch s;
  s.head = 0;
  s.meta = 256;
  s.lse = up256(s.meta + sizeof(SeqMeta) * static_cast<size_t>(B));
  s.o = up256(s.lse + 4 * static_cast<size_t>(rows));
  s.bytes = up256(s.o + 4 * static_cast<size_t>(rows) * D);
  return s;
}

template <int DTYPE, int D>
cudaError_t run(const PrefixAttnArgs &a, cudaStream_t s) {
  using C = AttnCfg<D>;
  AttnArgs g = {};
  g.a = a;
  if (!g.a.wait_limit_ns) g.a.wait_limit_ns = kDefaultWaitLimitNs;
  const Scratch sc = plan(g, a.T, a.B, a.max_q, a.hq, a.hkv, D, a.prefix_len);
  g.piece = reinterpret_cast<int64_t *>(a.scratch + sc.head);
  g.meta = reinterpret_cast<SeqMeta *>(a.scratch + sc.meta);
  g.part_lse = reinterpret_cast<float *>(a.scratch + sc.lse);
  g.part_o = reinterpret_cast<float *>(a.scratch + sc.o);
  // no pages at all: nothing is seen
  const int planned = a.prefix_len > 0 || (a.B > 0 && a.max_pages > 0);
  if (planned) {
    CUtensorMap tmK, tmV, tmQp, tmQs;
    const uint64_t rows = (static_cast<uint64_t>(a.num_pages) * a.hkv) << a.page_shift;
    const uint32_t page_rows = std::min(1 << a.page_shift, kTile);
    if (!attn_tmap(&tmK, DTYPE, a.k_cache, D, rows, D * 2, page_rows) ||
        !attn_tmap(&tmV, DTYPE, a.v_cache, D, rows, D * 2, page_rows) ||
        !attn_tmap(&tmQp, DTYPE, a.q, D, a.hq, D * 2, g.G, a.T, a.q_stride * 2, g.p_box) ||
        !attn_tmap(&tmQs, DTYPE, a.q, D, a.hq, D * 2, g.G, a.T, a.q_stride * 2, g.s_box))
      return cudaErrorInvalidValue;
    const cudaError_t err = cudaFuncSetAttribute(
        prefix_attention_kernel<DTYPE, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
        C::SMEM_BYTES);
    if (err != cudaSuccess) return err;
    MOE_LAUNCH_PDL(prefix_attention_kernel<DTYPE, D>, std::min(num_sms(), kMaxCtas), kAttnThreads,
                   C::SMEM_BYTES, s, tmK, tmV, tmQp, tmQs, g);
  }
  const int warps = std::min(8, a.hq);
  MOE_LAUNCH_PDL(prefix_attention_join_kernel<DTYPE, D>,
                 dim3(static_cast<unsigned>(a.T), (a.hq + warps - 1) / warps), warps * 32, 0, s, g,
                 planned);
  return cudaGetLastError();
}

}  // namespace

size_t prefix_attention_scratch_bytes(int T, int B, int max_q, int hq, int hkv, int D,
                                      int prefix_len) {
  AttnArgs g = {};
  return plan(g, T, B, max_q, hq, hkv, D, prefix_len).bytes;
}

cudaError_t launch_prefix_attention(const PrefixAttnArgs &a, int dtype, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  if (dtype == MOE_DTYPE_BF16)
    return a.D == 64 ? run<MOE_DTYPE_BF16, 64>(a, s) : run<MOE_DTYPE_BF16, 128>(a, s);
  return a.D == 64 ? run<MOE_DTYPE_FP16, 64>(a, s) : run<MOE_DTYPE_FP16, 128>(a, s);
}

}  // namespace moe
