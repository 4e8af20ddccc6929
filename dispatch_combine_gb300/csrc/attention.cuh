// attention.cuh -- what the kernels of the shared-prefix attention have in
// common: the plan of the work, and the walk over it.
//
// Work is cut into units: a block of tokens x a key head x the rows those
// tokens see in one place (the shared prefix, or their sequence's own rows),
// each a run of steps along the keys.  The units of one kind stand in a line,
// weighted by their time, and the line is cut into pieces of one length, one
// per worker, so the load is even whatever the lengths, which only the device
// knows.  A unit's stretch on a worker is a segment and leaves one partial
// result (o normalised, and its log-sum-exp); a last kernel joins them.
// A segment's slot among the partial results is its unit's number + its
// worker's, which grows along the line, so `units + workers` slots are enough.
#pragma once

#include "elem.cuh"
#include "kernels.h"

namespace moe {

// What the joining kernel needs of a sequence.
struct SeqMeta {
  int32_t unit;   // number of its first unit
  int32_t steps;  // per unit
};

// How the own rows of the sequences are cut (by either kernel).
struct OwnPlan {
  int tok;        // tokens of a unit
  int rows;       // rows of a slot (or of its half)
  int64_t slot0;  // first row of its slots
  int span0;      // its first unit's place in AttnArgs::span
};
// What a step of a unit costs there: constants of the kernel.
constexpr int kMaxCtas = 160;   // grid limit of both (slots of partial results)
constexpr int kRowWarps = 8;    // warps per CTA of the rows kernel

struct SliceSteps {  // rows kernel
  static constexpr int kKeys = 16, kUnitCost = 2;
  static __device__ __forceinline__ int cost(int) { return 1; }
  static __device__ __forceinline__ int steps_up(int x, int) { return x; }  // ceil(x / cost)
};
struct TileSteps {  // tiles kernel: a narrow tile 2, a wide one 3
  static constexpr int kKeys = 128, kUnitCost = 1, kMostCost = 3;
  static __device__ __forceinline__ int cost(int wide) { return 2 + wide; }
  static __device__ __forceinline__ int steps_up(int x, int wide) {
    return wide ? (x + 2) / 3 : (x + 1) / 2;
  }
};

struct AttnArgs {
  PrefixAttnArgs a;
  int G;  // query heads per key head
  // rows kernel: units of up to 16 * r_mt rows, a step is a slice of 16 keys
  int r_on, r_mt, r_tok, r_rows;
  int r_prefix, r_blocks, r_slices;  // the prefix's units are its: token blocks, slices
  int64_t r_pcost, r_ptotal;         // of a prefix unit, of all
  // tiles kernel: units of up to 128 (narrow) or 256 (wide) rows, a step is a
  // tile of 128 keys
  int t_on, tpt;                     // tokens per 128 rows
  int p_on, p_wide, p_tok, p_blocks, p_tiles, p_rows, p_box;
  int p_gang, p_groups, p_gangs;     // CTAs of a gang, token blocks / gang, gangs
  int64_t p_piece;                   // tiles of a gang's piece
  int share;                         // the rows kernel does the own rows beside it: the tiles
                                     // kernel works out how many of its gangs to use
  int own_on, s_wide, s_box;
  OwnPlan own;
  int own_rows_kernel;               // the own rows are the rows kernel's
  SeqMeta *meta;
  // device: the first and the last worker of every unit (prefix units, then
  // own units), written by those two
  int2 *span;
  float *part_o, *part_lse;
};

struct Seq {
  int q0, nq, len, steps, units;
  int64_t cost;  // of all its units
};

// Sequence b with every value clamped into the buffers.
template <class K>
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
  s.steps = (s.len + K::kKeys - 1) / K::kKeys;
  const int blocks = s.nq <= g.own.tok ? s.nq > 0 : (s.nq + g.own.tok - 1) / g.own.tok;
  s.units = blocks * a.hkv;
  s.cost = s.steps > 0 ? s.units * (static_cast<int64_t>(s.steps) * K::cost(g.s_wide) + K::kUnitCost)
                       : 0;
  return s;
}

// 64-bit divisions are kept out of line: they are long code.
__device__ __noinline__ inline int64_t div64(int64_t n, int64_t d) { return n / d; }
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d) {
  if (n < (int64_t{1} << 31) && d < (int64_t{1} << 31))
    return static_cast<uint32_t>(n) / static_cast<uint32_t>(d);
  return div64(n, d);
}

// Costs and unit counts of all sequences, scanned by the whole CTA (THREADS
// threads, any number of sequences).  `before` of a thread's first sequence.
struct OwnScan {
  int b_lo, b_hi;
  int64_t before, total;
  int units_before;
  bool drop, bad;  // offsets that are no partition of the tokens: nothing is attended
};
template <int THREADS>
struct ScanShared {
  int64_t warp_cost[THREADS / 32], before[THREADS];
  int warp_units[THREADS / 32], units[THREADS];
};
template <class K, int THREADS>
__device__ __forceinline__ OwnScan scan_own(const AttnArgs &g, ScanShared<THREADS> &sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (g.a.B + THREADS - 1) / THREADS;
  OwnScan r;
  r.b_lo = threadIdx.x * per;
  r.b_hi = min(r.b_lo + per, g.a.B);
  int64_t my_cost = 0;
  int my_units = 0;
  bool bad_off = false, bad = false;
#pragma unroll 1
  for (int b = r.b_lo; b < r.b_hi; ++b) {
    const Seq s = read_seq<K>(g, b, &bad_off, &bad);
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
    sh.warp_cost[warp] = cost;
    sh.warp_units[warp] = units;
  }
  r.drop = __syncthreads_or(bad_off);
  r.bad = bad || bad_off;
  r.before = cost - my_cost;
  r.units_before = units - my_units;
  r.total = 0;
#pragma unroll 1
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) {
      r.before += sh.warp_cost[w];
      r.units_before += sh.warp_units[w];
    }
    r.total += sh.warp_cost[w];
  }
  if (r.drop) r.total = 0;
  sh.before[threadIdx.x] = r.before;
  sh.units[threadIdx.x] = r.units_before;
  __syncthreads();
  return r;
}

// What each kernel gets when the rows kernel has `slices` slices of own rows to
// read beside the prefix's tiles; a whole warp.  Both ends are estimated for
// every number of gangs (the warp tries 32 at a time) from measured rates, and
// the first is taken: a gang's tiles cost a fixed time each, the rows run at
// sm_rate per SM left to them up to the HBM's rate, and either stay on those
// SMs or, cut into pieces for all SMs, go on everywhere once the tiles are done
// (at the price of one more start and a part of a piece: 64 sequences with one
// own row each over a prefix of 1024 took 26.2 us without it, 22.8 with it).
//   sm_rate 60, 70, 80 GB/s at D = 128: 64 sequences, prefix 8192, own rows up
// to 1024: 53.8, 51.7, 49.7 us; 64, 2048 and 4096: 115.7, 115.6, 120.2; 128,
// 8192 and 512: 67.8, 65.8, 65.3.  45 and 55 at D = 64 (4 key heads of 7): 64 of
// up to 4 tokens, 4099 and 777: 29.1, 34.6; 100, 4099 and 2000: 36.9, 34.6.
// Without rows_us0, D = 64: the former 34.7, 32 of up to 2 tokens (8 heads of 8),
// 1000 and 300: 26.9 instead of 20.6; D = 128: 64, 8192 and 1024: 49.3, 52.9 with.
struct ShareOut {
  int gangs, workers;
};
template <int D>
__device__ __forceinline__ ShareOut share_out(const AttnArgs &g, int64_t slices, int ctas) {
  const float tile_us = (D == 128 ? 1.75f : 1.25f) * (g.p_wide ? 1.0f : 0.6f), tiles_us0 = 9.0f;
  const float sm_rate = D == 128 ? 70e3f : 45e3f, hbm_rate = 6.4e6f, rows_us0 = 5.0f;  // per us
  const float bytes = static_cast<float>(slices) * (64.0f * D);
  const float tiles = static_cast<float>(g.a.hkv) * g.p_groups * g.p_tiles;
  const float tail = 3.5f + 0.25f * bytes / (ctas * sm_rate);
  struct Ends {
    float tiles, rows, rows_all;
  };
  auto ends = [&](int k) {
    const float t = tiles_us0 + ceilf(tiles / k) * tile_us;
    const float rate = fminf((ctas - k * g.p_gang) * sm_rate, hbm_rate);
    return Ends{t, rate > 0.0f ? rows_us0 + bytes / rate : INFINITY,
                t + fmaxf(bytes - (t - rows_us0) * rate, 0.0f) / hbm_rate + tail};
  };
  float best = INFINITY;
  int use = 1;
  for (int k = 1 + (threadIdx.x & 31); k <= g.p_gangs; k += 32) {
    const Ends e = ends(k);
    // where the rows take longest any way, the fewer tiles in a row the better
    const float cost = fmaxf(e.tiles, fminf(e.rows, e.rows_all)) + e.tiles * (1.0f / 16);
    if (cost < best) {
      best = cost;
      use = k;
    }
  }
  const unsigned first = __reduce_min_sync(0xffffffffu, __float_as_uint(best));  // best > 0
  use = __reduce_min_sync(0xffffffffu, __float_as_uint(best) == first ? use : g.p_gangs);
  const Ends e = ends(use);
  const int left = e.rows <= e.rows_all ? ctas - use * g.p_gang : ctas;
  return {use, left * kRowWarps};
}

// The scan's values of each sequence for the joining kernel (one CTA).
template <class K>
__device__ __forceinline__ void write_meta(const AttnArgs &g, const OwnScan &r) {
  bool x = false, y = false;
  int unit = r.units_before;
#pragma unroll 1
  for (int b = r.b_lo; b < r.b_hi; ++b) {
    const Seq s = read_seq<K>(g, b, &x, &y);
    g.meta[b] = SeqMeta{unit, r.drop ? 0 : s.steps};
    unit += s.units;
  }
  if (r.bad) set_status(g.a.status, kStatusBadId);
}

// A unit's stretch on one worker.
struct Stretch {
  int head, tok0, ntok;  // key head, first token, tokens
  int lim0, kv_len;      // token i sees keys below min(kv_len, lim0 + i)
  int s0, s1, n;         // steps [s0, s1) of n
  int64_t unit;          // its number among the units of its kind
  const int32_t *pages;
};

// The unit's partial results: from which worker to which.
__device__ __forceinline__ void mark_span(const AttnArgs &g, int64_t place, const Stretch &x,
                                          int worker) {
  if (x.s0 == 0) g.span[place].x = worker;
  if (x.s1 == x.n) g.span[place].y = worker;
}

// the first of a unit's n steps at or past `ahead` of its start
template <class K>
__device__ __forceinline__ int step_at(int64_t ahead, int n, int wide) {
  if (ahead <= 0) return 0;
  if (ahead >= static_cast<int64_t>(n) * K::cost(wide)) return n;
  return K::steps_up(static_cast<int>(ahead), wide);
}

// Walks the own units in [lo, hi) of their line; a whole warp.  next() gives
// one stretch at a time.
template <class K>
struct OwnWalk {
  int64_t lo, hi, cum0, batch, cum, start, unit_cost;
  int unit0, batch_units, base, un;
  unsigned todo;
  Seq s;
  int seq, j, n_units, q0, nq, len, steps, unit;

  template <int THREADS>
  __device__ __forceinline__ void begin(const AttnArgs &g, const ScanShared<THREADS> &sh,
                                        int64_t lo_, int64_t hi_) {
    lo = lo_;
    hi = hi_;
    // the last thread of the scan whose sequences start at or before lo
    int i = 0;
    for (int k = threadIdx.x & 31; k < THREADS; k += 32)
      if (sh.before[k] <= lo) i = k;
    i = __reduce_max_sync(0xffffffffu, i);
    base = i * ((g.a.B + THREADS - 1) / THREADS) - 32;
    cum0 = sh.before[i];
    unit0 = sh.units[i];
    batch = 0;
    batch_units = 0;
    todo = 0;
    j = n_units = 0;
    start = 0;
    unit_cost = 1;
  }
  __device__ __forceinline__ bool next(const AttnArgs &g, Stretch *out) {
    const int lane = threadIdx.x & 31;
    while (true) {
      if (j < n_units && start + j * unit_cost < hi) {
        const int at = j++;
        const int64_t from = start + at * unit_cost;
        out->s0 = step_at<K>(lo - from, steps, g.s_wide);
        out->s1 = step_at<K>(hi - from, steps, g.s_wide);
        out->n = steps;
        if (out->s0 >= out->s1) continue;
        const int block = at / g.a.hkv;
        out->head = at - block * g.a.hkv;
        const int i0 = block * g.own.tok;
        out->tok0 = q0 + i0;
        out->ntok = min(g.own.tok, nq - i0);
        out->lim0 = len - nq + i0 + 1;
        out->kv_len = len;
        out->unit = unit + at;
        out->pages = g.a.page_table + static_cast<int64_t>(seq) * g.a.max_pages;
        return true;
      }
      if (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        seq = base + src;
        q0 = __shfl_sync(0xffffffffu, s.q0, src);
        nq = __shfl_sync(0xffffffffu, s.nq, src);
        len = __shfl_sync(0xffffffffu, s.len, src);
        steps = __shfl_sync(0xffffffffu, s.steps, src);
        n_units = __shfl_sync(0xffffffffu, s.units, src);
        start = __shfl_sync(0xffffffffu, cum, src);
        unit = __shfl_sync(0xffffffffu, un, src);
        unit_cost = static_cast<int64_t>(steps) * K::cost(g.s_wide) + K::kUnitCost;
        j = lo <= start ? 0 : static_cast<int>(quotient(lo - start, unit_cost));
        continue;
      }
      base += 32;
      cum0 += batch;
      unit0 += batch_units;
      if (base >= g.a.B || cum0 >= hi) return false;
      bool x = false, y = false;
      s = read_seq<K>(g, base + lane, &x, &y);
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
    }
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The probabilities of both kernels are 2^(s * sl2 + c0), c0 = off - m * sl2:
// fp16 ones are kept 2^10 up, away from its subnormals; the running maximum m
// may lag by `lag` powers of two behind the true one before sums and
// accumulators are rescaled, so they stay below 2^15 (fp16 holds 65504) or 2^8
// (bf16).  c0 is one fp32 number, the same for all keys that it serves, so its
// rounding cancels as long as the sums are rescaled by, and the log-sum-exp taken
// from, this number.  It must not carry a probability past its type: up to
// kMost it rounds by at most 1/2 (2^15.5) or 32 (2^40).  Past it a row's result
// is NaN.  (Taking the maximum off the scores first has no such end, but as one
// more addition per score, or a branch around the exponentials for such rows
// alone, 256 queries over 32768 rows took 231 to 255 us at head size 128
// instead of 212.)
// They are rounded to the cache's type for the product with V, the one rounding
// to 16 bits before the output's: the tensor cores take both operands in one
// type, and in two parts (high and low) the products would double.  It makes the
// output's error against 64 bits 1.2 to 1.4 times that of the output's own
// rounding (bf16 0.0020 to 0.0023 relative, 0.0017 without; fp16 0.00027 and
// 0.00021).  The sum is taken of the unrounded ones.
template <int DTYPE>
struct Prob {
  static constexpr float kOff = DTYPE == MOE_DTYPE_FP16 ? 10.0f : 0.0f;
  static constexpr float kLag = DTYPE == MOE_DTYPE_FP16 ? 5.0f : 8.0f;
  static constexpr float kMost = DTYPE == MOE_DTYPE_FP16 ? 16777216.0f : 1073741824.0f;
};
template <int DTYPE>
__device__ __forceinline__ float prob_offset(float m, float sl2) {
  return m == -INFINITY ? Prob<DTYPE>::kOff : fmaf(-m, sl2, Prob<DTYPE>::kOff);
}
// What sums taken with maximum m become with m1 > m.
template <int DTYPE>
__device__ __forceinline__ float rescale(float m, float m1, float sl2) {
  return m == -INFINITY ? 0.0f : ex2(prob_offset<DTYPE>(m1, sl2) - prob_offset<DTYPE>(m, sl2));
}
// The maximum to take for scores up to `top`: none below the range, so that
// scores down there have probabilities of 0 and not of their type's infinity.
template <int DTYPE>
__device__ __forceinline__ float in_range(float top, float sl2) {
  return fmaxf(top, -Prob<DTYPE>::kMost / sl2);
}
// A part's scale and log2-sum-exp from its sum l: 0 and -infinity where it saw
// nothing, or only scores below the range; a NaN (a query that is not finite,
// scores above the range) stays one.
struct PartEnd {
  float inv, lse;
};
template <int DTYPE>
__device__ __forceinline__ PartEnd end_part(float m, float l, float sl2) {
  const float c0 = prob_offset<DTYPE>(m, sl2);
  if (c0 < -Prob<DTYPE>::kMost) l = NAN;
  if (l == 0.0f) return {0.0f, -INFINITY};
  return {1.0f / l, log2f(l) - c0};
}
constexpr float kLog2e = 1.4426950408889634f;
// The lag in units of a score; finite for the smallest scales too, whose
// reciprocal is not: -infinity + lag is the first maximum's bar.
template <int DTYPE>
__device__ __forceinline__ float score_lag(float sl2) {
  return fminf(Prob<DTYPE>::kLag / sl2, 3.4028234663852886e38f);
}

constexpr int kTile = TileSteps::kKeys;    // keys per tile
constexpr int kSlice = SliceSteps::kKeys;  // keys per slice
constexpr int kMinSlices = 2;   // shortest piece of the rows kernel's line

// prefix_attention_rows.cu, prefix_attention_tiles.cu
cudaError_t launch_attention_rows(const AttnArgs &g, int dtype, int ctas, cudaStream_t s);
cudaError_t launch_attention_tiles(const AttnArgs &g, int dtype, int ctas, cudaStream_t s);

}  // namespace moe
