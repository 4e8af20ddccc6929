// prefix_attention.cu -- attention of a batch that shares a long prefix
// (moe_prefix_attention): the plan, and the join of the partial results.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q.k_j)
// over the prefix's rows and then the sequence's own up to the token's causal
// limit.  The sum over j splits anywhere: a part keeps its o normalised and
// lse = log sum p, and parts join with weights exp(lse - max lse).
//
// The prefix is read once for the whole batch (a block of tokens of all
// sequences is one set of query rows), each sequence's own rows once for each
// block of its tokens (up to 256 rows).  Few rows per key head (the common
// decode step) go to the rows kernel, which is made to stream the cache; many
// go to the tiles kernel, which is made to feed the tensor cores.  A call that needs both runs them
// side by side: the tiles kernel uses as many SMs as lets both end together
// (it reads the lengths on the device), and the rows kernel, launched behind it
// without waiting for it, starts on the others (64 sequences, prefix 8192, own
// rows up to 1024: 63.5 us one after the other, 51.5 so; 256, 32768 and 512: 247
// and 228).
#include <algorithm>

#include "attention.cuh"

namespace moe {
namespace {

// Parts of one kind for one row: n slots `step` rows apart, each of one or
// two rows (the halves of a narrow tile unit).
struct Parts {
  int64_t first, step;
  int n, halves, half_step;
  __device__ __forceinline__ int count() const { return n * halves; }
  __device__ __forceinline__ int64_t row(int i) const {
    return halves == 2 ? first + (i >> 1) * step + (i & 1) * half_step : first + i * step;
  }
};

// the row of a tile unit's token: in the half of a wide unit that holds it
__device__ __forceinline__ int half_row(const AttnArgs &g, int in, int rows) {
  return in < g.tpt ? in * g.G : rows + (in - g.tpt) * g.G;
}

// The workers of a unit, inside the slots whatever stands there (a tiles
// kernel whose wait ran out leaves spans unwritten).
__device__ __forceinline__ int2 span_of(const AttnArgs &g, int64_t place, bool rows_kernel) {
  const int most = rows_kernel ? kMaxCtas * kRowWarps : kMaxCtas;
  int2 w = g.span[place];
  w.x = min(max(w.x, 0), most - 1);
  w.y = min(max(w.y, w.x), most - 1);
  return w;
}

// A whole CTA, where there are no pages of own rows: what the scan of the lengths
// would have found wrong with them and the offsets.
__device__ __forceinline__ void report_bad(const PrefixAttnArgs &a) {
  bool bad = false;
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    bad |= a.kv_lens[b] != 0;
    if (a.q_offsets) {
      const int64_t q0 = a.q_offsets[b], q1 = a.q_offsets[b + 1];
      bad |= q0 < 0 || q1 < q0 || q1 > a.T || q1 - q0 > a.max_q;
    }
  }
  if (bad) set_status(a.status, kStatusBadId);
}

// W warps per token and query head, each with every W-th batch of its parts
// (one token has as many parts as its rows have workers, and little else to
// fill the GPU).
template <int DTYPE, int D, int W>
__global__ void __launch_bounds__(256) attention_join_kernel(const AttnArgs g) {
  // A kernel of the same call that ran before has waited for everything before
  // the call, so the call's inputs can be read ahead of this one's own wait.
  const bool alone = !g.r_on && !g.t_on;
  if (alone) pdl_begin();
  if (!g.own_rows_kernel && !g.own_on && blockIdx.x == 0 && blockIdx.y == 0) report_bad(g.a);
  constexpr int E = D / 32;
  constexpr int kBatch = W > 1 ? 8 : 4;  // with many rows the other warps hide a row's way
  const PrefixAttnArgs &a = g.a;
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  // the token's sequence: how many end at or before it, by a search 32 ways at a
  // time (4096 sequences of up to 512 rows over 1024, 16 + 2 heads: 257 us a call,
  // 285 when every CTA counts them all; up to 64 sequences: the same)
  int b = t;
  if (a.q_offsets) {
    b = 0;
#pragma unroll 1
    for (int n = a.B; n > 0;) {  // the answer is in [b, b + n]
      const int part = (n + 31) >> 5;
      const int probe = b + min((lane + 1) * part, n);
      const int k = __popc(__ballot_sync(0xffffffffu, a.q_offsets[probe] <= t));
      b += min(k * part, n);
      n = max(min(part, n - k * part) - 1, 0);
    }
  }
  if (!alone) pdl_begin();
  const int h0 = (blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5)) / W;
  const int wi = (threadIdx.x >> 5) % W;
  if (W == 1 && h0 >= a.hq) return;
  const int h = min(h0, a.hq - 1);  // W > 1: all warps meet at a barrier
  const int kvh = h / g.G, hg = h - kvh * g.G;
  Parts pre = {0, 0, 0, 1, 0}, own = {0, 0, 0, 1, 0};
  const bool has_own = (g.own_rows_kernel || g.own_on) && b < a.B;
  SeqMeta m = {0, 0};
  int q0 = b;
  if (has_own) {  // on their way while the prefix's place is worked out
    m = g.meta[b];
    if (a.q_offsets) q0 = a.q_offsets[b];
  }
  if (g.r_prefix) {
    const int block = t / g.r_tok, u = kvh * g.r_blocks + block;
    const int2 w = span_of(g, u, true);
    pre.step = g.r_rows;
    pre.first = static_cast<int64_t>(u + w.x) * g.r_rows + (t - block * g.r_tok) * g.G + hg;
    pre.n = w.y - w.x + 1;
  } else if (g.p_on) {
    const int block = t / g.p_tok, in = t - block * g.p_tok;
    const int group = block / g.p_gang, member = block - group * g.p_gang;
    const int64_t q = static_cast<int64_t>(kvh) * g.p_groups + group;
    const int2 w = span_of(g, q * g.p_gang + member, false);
    pre.step = static_cast<int64_t>(g.p_gang) * 2 * g.p_rows;
    pre.halves = g.p_wide ? 1 : 2;
    pre.half_step = g.p_rows;
    pre.first = (q + w.x) * pre.step + member * 2 * g.p_rows + half_row(g, in, g.p_rows) + hg;
    pre.n = w.y - w.x + 1;
  }
  if (has_own) {
    const int place = t - q0;
    if (place >= 0 && place < a.max_q && m.steps > 0) {
      const int block = place / g.own.tok, in = place - block * g.own.tok;
      const int u = m.unit + block * a.hkv + kvh;
      const int2 w = span_of(g, g.own.span0 + u, g.own_rows_kernel);
      own.halves = g.own_rows_kernel || g.s_wide ? 1 : 2;
      own.half_step = g.own.rows;
      own.step = g.own_rows_kernel ? g.own.rows : 2 * g.own.rows;
      own.first = g.own.slot0 + static_cast<int64_t>(u + w.x) * own.step +
                  (g.own_rows_kernel ? in * g.G : half_row(g, in, g.own.rows)) + hg;
      own.n = w.y - w.x + 1;
    }
  }
  const int np = pre.count(), parts = np + own.count();
  auto row_of = [&](int i) { return i < np ? pre.row(i) : own.row(i - np); };
  // kBatch rows on their way at a time, the first of them before the maximum is
  // known; a part with weight 0 may have no row, and whatever lies there does
  // not count
  float x[kBatch][E];
  int here = min(32, parts);
  int64_t mine = row_of(min(lane, max(parts, 1) - 1));
  auto fetch = [&](int k) {
#pragma unroll
    for (int c = 0; c < kBatch; ++c) {
      const float *src = g.part_o + __shfl_sync(0xffffffffu, mine, k + c) * D + lane * E;
      if (k + c < here) {
        if (E == 4)
          *reinterpret_cast<float4 *>(x[c]) = *reinterpret_cast<const float4 *>(src);
        else
          *reinterpret_cast<float2 *>(x[c]) = *reinterpret_cast<const float2 *>(src);
      }
    }
  };
  float lse = lane < parts ? g.part_lse[mine] : -INFINITY;
  if (kBatch * wi < here) fetch(kBatch * wi);
  float top = lse;
#pragma unroll 2
  for (int i = lane + 32; i < parts; i += 32) top = fmaxf(top, g.part_lse[row_of(i)]);
#pragma unroll
  for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  const float ref = top == -INFINITY ? 0.0f : top;
  float o[E], l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
#pragma unroll 1
  for (int base = 0; base < parts;) {
    const float wgt = ex2(lse - ref);  // 0 past the end
#pragma unroll 1
    for (int k = kBatch * wi; k < here;) {
#pragma unroll
      for (int c = 0; c < kBatch; ++c) {
        const float wk = __shfl_sync(0xffffffffu, wgt, k + c);
        l += wk;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = wk == 0.0f ? o[e] : fmaf(wk, x[c][e], o[e]);
      }
      k += kBatch * W;
      if (k < here) fetch(k);
    }
    base += 32;
    if (base >= parts) break;
    here = min(32, parts - base);
    mine = row_of(min(base + lane, parts - 1));
    lse = base + lane < parts ? g.part_lse[mine] : -INFINITY;
    if (kBatch * wi < here) fetch(kBatch * wi);
  }
  if (W > 1) {
    __shared__ float s_o[8][E + 1][32];
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][e][lane] = o[e];
    s_o[warp][E][lane] = l;
    __syncthreads();
    if (wi != 0 || h0 >= a.hq) return;
#pragma unroll
    for (int w = 1; w < W; ++w) {  // in order: the sum does not depend on timing
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += s_o[warp + w][e][lane];
      l += s_o[warp + w][E][lane];
    }
  }
  // A sum of zero: no key is visible, or every score is -infinity (an infinite
  // element in the query, or a product past fp32), where the quotient is 0 / 0.
  // A query with a NaN has left one in l.
  float inv = 1.0f / l;
  if (l == 0.0f) {
    bool seen = a.prefix_len > 0;
    if (m.steps > 0) {
      const int nq = a.q_offsets ? a.q_offsets[b + 1] - q0 : 1;
      seen |= a.kv_lens[b] - nq + (t - q0) + 1 > 0;
    }
    if (seen) l = NAN;
    inv = l;
  }
  uint32_t *dst =
      reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.o) + t * a.o_stride + h * D) +
      lane * (E / 2);
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = pack2<DTYPE>(o[e] * inv, o[e + 1] * inv);
  if (a.lse && lane == 0)
    a.lse[static_cast<int64_t>(t) * a.hq + h] =
        l == 0.0f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
}

// ---------------------------------------------------------------------------
// the plan: everything the host knows, and the scratch it needs
// ---------------------------------------------------------------------------

// Rows (tokens x query heads of a key head) that the rows kernel takes, as one
// unit: of one sequence's own, or of the whole batch over the prefix.  Both
// kernels on the same work (us, rows kernel and tiles kernel):
//   own, 64 sequences x 4096, 8 key heads of 128: 16 rows 172 and 181, 20 rows
// 205 and 183, 32 rows 214 and 188 (two 16-row blocks of accumulators of 128 do
// not fit a warp's registers); key heads of 64, lengths up to 4096: 32 rows 62
// and 72, 48 rows (two units, so keys and values read twice) 77 and 74;
//   prefix of 1000, heads of 128: 16 rows 7.9 and 10.3, 20 rows 11.7 and 10.3;
// heads of 64, 28 rows, beside own rows of up to 300 (which the rows kernel then
// takes along): prefix 1000 12.1 and 15.2, 4000 16.2 and 20.8; without own rows:
// 1000 8.1 and 9.1, 4000 12.7 and 11.5, 8192 20.8 and 12.2.
constexpr int most_rows(int D) { return D == 64 ? 32 : 16; }
constexpr int kRows = 16, kPrefixOf32 = 4096;  // any prefix; up to which 32 rows are taken
bool own_by_rows(int D, int64_t rows) { return rows <= most_rows(D); }
bool prefix_by_rows(int D, int64_t rows, int prefix_len) {
  return rows <= (prefix_len <= kPrefixOf32 ? most_rows(D) : kRows);
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Units of one kind, and rows of partial results for them.
struct Slots {
  int64_t units, rows;
};
struct Scratch {
  size_t span, lse, o, bytes;
};
Scratch layout(int B, const Slots &prefix, const Slots &own, int D) {
  const size_t units = static_cast<size_t>(prefix.units + own.units);
  const size_t rows = static_cast<size_t>(prefix.rows + own.rows);
  Scratch s;
  s.span = up256(sizeof(SeqMeta) * static_cast<size_t>(B));
  s.lse = up256(s.span + sizeof(int2) * units);
  s.o = up256(s.lse + 4 * rows);
  s.bytes = up256(s.o + 4 * rows * D);
  return s;
}
struct Need {
  Slots prefix, own;
};

// own_rows: whether sequences can have rows of their own
Need plan(AttnArgs &g, int T, int B, int max_q, int hq, int hkv, int D, int prefix_len,
             bool own_rows, int ctas) {
  const int G = hq / hkv, nq = std::max(1, std::min(max_q, T));
  g.G = G;
  g.tpt = kTile / G;
  const bool own = own_rows && B > 0;
  const bool small_prefix = prefix_by_rows(D, static_cast<int64_t>(T) * G, prefix_len);
  g.r_prefix = prefix_len > 0 && small_prefix;
  g.p_on = prefix_len > 0 && !small_prefix;
  g.own_rows_kernel = own && own_by_rows(D, static_cast<int64_t>(nq) * G);
  g.own_on = own && !g.own_rows_kernel;
  g.r_on = g.r_prefix || g.own_rows_kernel;
  g.t_on = g.p_on || g.own_on;
  g.share = g.p_on && g.own_rows_kernel;
  // rows kernel: one 16-row block if all units fit, else 32-row units
  const int most = std::max(g.r_prefix ? T * G : 0, g.own_rows_kernel ? nq * G : 0);
  g.r_mt = most <= 16 ? 1 : 2;
  g.r_tok = std::max(1, std::min(16 * g.r_mt / G, std::max(T, 1)));
  g.r_rows = g.r_tok * G;
  g.r_blocks = (T + g.r_tok - 1) / g.r_tok;
  g.r_slices = g.r_prefix ? (prefix_len + kSlice - 1) / kSlice : 0;
  g.r_pcost = g.r_slices + SliceSteps::kUnitCost;
  g.r_ptotal = g.r_prefix ? static_cast<int64_t>(hkv) * g.r_blocks * g.r_pcost : 0;
  // tiles kernel
  g.p_wide = T > g.tpt;
  g.p_tok = g.p_wide ? 2 * g.tpt : g.tpt;
  g.p_blocks = (T + g.p_tok - 1) / g.p_tok;
  g.p_tiles = static_cast<int>((static_cast<int64_t>(prefix_len) + kTile - 1) / kTile);
  g.p_box = std::min(g.tpt, std::max(T, 1));
  g.p_rows = g.p_box * G;
  if (g.p_on) {
    // the gang size that takes the least time; 4 blocks sharing a tile are
    // enough to keep HBM out of the way, 16 the most that is tried
    int64_t best = -1;
    for (int gs = std::min({g.p_blocks, 4, ctas}); gs <= std::min({g.p_blocks, 16, ctas}); ++gs) {
      const int groups = (g.p_blocks + gs - 1) / gs, gangs = ctas / gs;
      const int64_t piece =
          (static_cast<int64_t>(hkv) * groups * g.p_tiles + gangs - 1) / gangs;
      if (best < 0 || piece <= best) {
        best = piece;
        g.p_gang = gs;
        g.p_groups = groups;
        g.p_gangs = gangs;
        g.p_piece = piece;
      }
    }
  }
  g.s_wide = nq > g.tpt;
  g.s_box = std::min(g.tpt, nq);
  if (g.own_rows_kernel) {
    g.own.tok = std::min(g.r_tok, nq);
    g.own.rows = g.own.tok * G;
  } else {
    g.own.tok = g.s_wide ? 2 * g.tpt : g.tpt;
    g.own.rows = g.s_box * G;
  }
  Need n = {};
  if (g.r_prefix) {
    n.prefix.units = static_cast<int64_t>(hkv) * g.r_blocks;
    n.prefix.rows = (n.prefix.units + kMaxCtas * kRowWarps) * g.r_rows;
  } else if (g.p_on) {  // (hkv * groups + gangs) * gang slots, whatever the grid
    n.prefix.units = static_cast<int64_t>(hkv) * (g.p_blocks + 16);
    n.prefix.rows = (n.prefix.units + kMaxCtas) * 2 * g.p_rows;
  }
  g.own.slot0 = n.prefix.rows;
  g.own.span0 = static_cast<int>(n.prefix.units);
  if (own) {
    // blocks of all sequences: the tokens may lie in any of them, max_q in each
    const int64_t blocks = std::min<int64_t>(
        B + T / g.own.tok, static_cast<int64_t>(B) * ((nq + g.own.tok - 1) / g.own.tok));
    n.own.units = blocks * hkv;
    n.own.rows = g.own_rows_kernel ? (n.own.units + kMaxCtas * kRowWarps) * g.own.rows
                                   : (n.own.units + kMaxCtas) * 2 * g.own.rows;
  }
  return n;
}

template <int DTYPE, int D>
cudaError_t join(const AttnArgs &g, int ctas, cudaStream_t s) {
  // four warps per row where that still leaves every warp slot of the GPU at
  // most one row (one token, 64 heads, 17 parts: 14.5 -> 11.3 us a call)
  constexpr int kWarps = 8, kWide = 4;
  const int64_t rows = static_cast<int64_t>(g.a.T) * g.a.hq;
  if (rows * kWide <= static_cast<int64_t>(ctas) * 64) {
    MOE_LAUNCH_PDL(attention_join_kernel<DTYPE, D, kWide>,
                   dim3(static_cast<unsigned>(g.a.T), (g.a.hq * kWide + kWarps - 1) / kWarps),
                   kWarps * 32, 0, s, g);
    return cudaGetLastError();
  }
  const int warps = std::min(kWarps, g.a.hq);
  MOE_LAUNCH_PDL(attention_join_kernel<DTYPE, D, 1>,
                 dim3(static_cast<unsigned>(g.a.T), (g.a.hq + warps - 1) / warps), warps * 32, 0, s,
                 g);
  return cudaGetLastError();
}

}  // namespace

size_t prefix_attention_scratch_bytes(int T, int B, int max_q, int hq, int hkv, int D,
                                      int prefix_len) {
  // What no smaller call passes.  Either kernel's need grows with every argument,
  // but the rows kernel has eight workers per CTA where the tiles kernel has one,
  // so its largest call can need more than the tiles kernel's smallest: the larger
  // of the two counts.
  AttnArgs g = {};
  Need n = plan(g, T, B, max_q, hq, hkv, D, prefix_len, true, kMaxCtas);
  const int tokens = most_rows(D) / (hq / hkv);
  if (tokens > 0) {
    const Slots p = plan(g = {}, std::min(T, tokens), B, max_q, hq, hkv, D,
                         std::min(prefix_len, kPrefixOf32), true, kMaxCtas).prefix;
    const Slots o = plan(g = {}, T, B, std::min(max_q, tokens), hq, hkv, D, prefix_len, true,
                         kMaxCtas).own;
    n.prefix = {std::max(n.prefix.units, p.units), std::max(n.prefix.rows, p.rows)};
    n.own = {std::max(n.own.units, o.units), std::max(n.own.rows, o.rows)};
  }
  return layout(B, n.prefix, n.own, D).bytes;
}

cudaError_t launch_prefix_attention(const PrefixAttnArgs &a, int dtype, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  AttnArgs g = {};
  g.a = a;
  const int ctas = std::min(num_sms(), kMaxCtas);
  const Need n = plan(g, a.T, a.B, a.max_q, a.hq, a.hkv, a.D, a.prefix_len, a.max_pages > 0, ctas);
  const Scratch sc = layout(a.B, n.prefix, n.own, a.D);
  g.meta = reinterpret_cast<SeqMeta *>(a.scratch);
  g.span = reinterpret_cast<int2 *>(a.scratch + sc.span);
  g.part_lse = reinterpret_cast<float *>(a.scratch + sc.lse);
  g.part_o = reinterpret_cast<float *>(a.scratch + sc.o);
  if (g.t_on) {
    const cudaError_t err = launch_attention_tiles(g, dtype, ctas, s);
    if (err != cudaSuccess) return err;
  }
  if (g.r_on) {
    const cudaError_t err = launch_attention_rows(g, dtype, ctas, s);
    if (err != cudaSuccess) return err;
  }
  if (dtype == MOE_DTYPE_BF16)
    return a.D == 64 ? join<MOE_DTYPE_BF16, 64>(g, ctas, s) : join<MOE_DTYPE_BF16, 128>(g, ctas, s);
  return a.D == 64 ? join<MOE_DTYPE_FP16, 64>(g, ctas, s) : join<MOE_DTYPE_FP16, 128>(g, ctas, s);
}

}  // namespace moe
