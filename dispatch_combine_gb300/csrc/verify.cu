// verify.cu -- drafted tokens against the target's probabilities, from given
// uniform numbers (moe_verify_drafts).
//
//   draft x of row i stands iff u_i q_i(x) < p_i(x) and all before it stand;
//   the first that falls leaves the token to max(p_i - q_i, 0), none to p_n:
//   token = min { v : sum_{w <= v} r_w > u sum r }.
// One row of p and one of q are read for each sequence, by a cluster of CTAs: 64
// sequences of 7 drafts over 131072 tokens in fp32 (67 MB) take 15.7 us, 0.63 of the
// measured copy bandwidth; one sequence over 32000 4.9.  What bounds it is the chain
// of dependent reads: offsets, drafts, their probabilities, the row, the sums of the
// cluster's CTAs, and the border's piece once more (from L2).  Rows of p and q that do not
// start alike modulo 16 bytes are read element by element: those 64 sequences 32 us, 37
// over 50021 tokens with the target's rows padded to 50048 11.2 (8.1 where both are dense).
//
// The sums are whole numbers: a weight in [0, 1] counts in units of 2^-60, so
// they are exact in any order (to 2^-60 a weight), and which token is the first
// past the border does not depend on how the row was cut.
#include "elem.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSlots = 2;  // of a lane on their way while as many are summed (23.1 us; 1: 23.5, 3: 26.4)

template <int DTYPE>
__device__ __forceinline__ float prob_at(const void *p, int64_t i) {
  if (DTYPE == MOE_DTYPE_FP32) return static_cast<const float *>(p)[i];
  return load1<DTYPE>(p, i);
}
// a weight in [0, 1] in units of 2^-60, cut off
__device__ __forceinline__ uint64_t units_of(float w) {
  const uint32_t b = __float_as_uint(w);
  const uint32_t high = b << 8 | 0x80000000u;  // the significand at the top of 64 bits
  const int down = 130 - static_cast<int>(b >> 23);  // 3 and more; 130 for zero
  const uint32_t low = __funnelshift_rc(0u, high, down);  // as far as 32
  uint32_t hi, lo;
  asm("shr.u32 %0, %1, %2;" : "=r"(hi) : "r"(high), "r"(down));  // 0 from 32 on
  asm("shr.u32 %0, %1, %2;" : "=r"(lo) : "r"(low), "r"(max(down - 32, 0)));
  return static_cast<uint64_t>(hi) << 32 | lo;
}
// floor(u * total) for u in [0, 1), total - 1 past it
__device__ __forceinline__ uint64_t part_of(float u, uint64_t total) {
  if (!(u > 0.0f) || total == 0) return 0;
  if (u >= 1.0f) return total - 1;
  const uint32_t b = __float_as_uint(u);
  const uint32_t m = b < 0x800000u ? b : (b & 0x7FFFFFu) | 0x800000u;
  const int down = 150 - max(static_cast<int>(b >> 23), 1);  // u = m 2^-down
  const uint64_t lo = total * m, hi = __umul64hi(total, m);
  if (down >= 128) return 0;
  if (down >= 64) return hi >> (down - 64);
  return hi << (64 - down) | lo >> down;
}

// A row's weights, 16 bytes of them at a time: slot j holds elements [VEC j - m, VEC
// (j + 1) - m), m what the row's start lies past a 16-byte boundary, so that all
// slots but the first and the last are one aligned load.
struct Row {
  const uint8_t *p, *q;  // of the row, back to the boundary; q nullptr: p alone
  int without;           // token whose weight is 0 (-1: none)
  int vocab, m;
  int full0, full1;      // slots that are one load of each row
};
template <int DTYPE>
constexpr int kVec = DTYPE == MOE_DTYPE_FP32 ? 4 : 8;
template <int DTYPE>
__device__ __forceinline__ void probs(const uint4 &v, float (&f)[kVec<DTYPE>]) {
  if constexpr (DTYPE == MOE_DTYPE_FP32) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  } else {
    unpack8<DTYPE>(v, f);
  }
}
// One slot as it lies in memory; zeros where there is nothing, and from `end` on
template <int DTYPE>
struct Slot {
  uint4 p, q;
  static __device__ __forceinline__ uint32_t word(const uint8_t *row, const Row &r, int64_t at) {
    constexpr int E = DTYPE == MOE_DTYPE_FP32 ? 1 : 2;  // elements of a word
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int64_t i = at + e;
      if (i < r.m || i - r.m >= r.vocab) continue;
      if (E == 1)
        w = reinterpret_cast<const uint32_t *>(row)[i];
      else
        w |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(row)[i]) << (16 * e);
    }
    return w;
  }
  static __device__ __noinline__ uint4 edge(const uint8_t *row, const Row &r, int j) {
    constexpr int V = kVec<DTYPE>;
    const int64_t at = static_cast<int64_t>(j) * V;
    return make_uint4(word(row, r, at), word(row, r, at + V / 4), word(row, r, at + V / 2),
                      word(row, r, at + 3 * (V / 4)));
  }
  __device__ __forceinline__ void load(const Row &r, int j, int end) {
    p = q = make_uint4(0, 0, 0, 0);
    if (j >= end) return;
    if (j >= r.full0 && j < r.full1) {
      p = *reinterpret_cast<const uint4 *>(r.p + static_cast<int64_t>(j) * 16);
      if (r.q) q = *reinterpret_cast<const uint4 *>(r.q + static_cast<int64_t>(j) * 16);
    } else {
      p = edge(r.p, r, j);
      if (r.q) q = edge(r.q, r, j);
    }
  }
  __device__ __forceinline__ void weights(const Row &r, int j, uint64_t (&w)[kVec<DTYPE>]) const {
    constexpr int V = kVec<DTYPE>;
    float x[V], y[V];
    probs<DTYPE>(p, x);
    probs<DTYPE>(q, y);
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = units_of(__saturatef(x[e] - y[e]));
    if (r.without >= 0 && (r.without + r.m) / V == j)
#pragma unroll
      for (int e = 0; e < V; ++e)
        if ((r.without + r.m) % V == e) w[e] = 0;
  }
};
__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

template <int DTYPE>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const VerifyArgs a, const int ctas) {
  pdl_begin();
  __shared__ uint64_t s_sums[kWarps];
  struct Found {
    uint64_t total, border, before;
    int owner;
  };
  __shared__ Found s_found;
  const int b = blockIdx.x / ctas, rank = blockIdx.x - b * ctas;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q0 = a.offsets[b], q1 = a.offsets[b + 1];
  const bool broken = q0 < 0 || q1 < q0 || q1 > a.T;
  const bool writer = rank == 0 && threadIdx.x == 0;
  if (broken || q1 == q0) {  // the whole cluster
    if (writer) {
      if (broken) set_status(a.status, kStatusBadId);
      a.accepted[b] = 0;
    }
    return;
  }
  const int n = q1 - q0 - 1;
  const float last = a.uniforms[q1 - 1];  // asked for now, needed late (one sequence 5.2 -> 4.9 us)
  const int size = DTYPE == MOE_DTYPE_FP32 ? 4 : 2;
  // ---- the drafts before the first that falls; every warp for itself
  int accepted = n, fallen = -1;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    bool falls = false;
    int x = 0;
    if (i < n) {
      x = a.tokens[q0 + i + 1];
      const int64_t row = q0 + i;
      if (x < 0 || x >= a.vocab) {
        falls = true;  // and is reported below, with those that are not looked at here
      } else {
        const double p = prob_at<DTYPE>(a.target, row * a.target_stride + x);
        const double q = a.draft ? prob_at<DTYPE>(a.draft, row * a.draft_stride + x) : 1.0f;
        falls = !(static_cast<double>(a.uniforms[row]) * q < p);
      }
    }
    const unsigned f = __ballot_sync(0xffffffffu, falls);
    if (f) {
      accepted = i0 + __ffs(f) - 1;
      fallen = __shfl_sync(0xffffffffu, x, __ffs(f) - 1);
      break;
    }
  }
  constexpr int V = kVec<DTYPE>;
  const int64_t row = q0 + accepted;
  Row r = {static_cast<const uint8_t *>(a.target) + row * a.target_stride * size, nullptr, -1,
           a.vocab, 0, 0, 0};
  bool alike = true;
  if (accepted < n) {
    if (a.draft) {
      r.q = static_cast<const uint8_t *>(a.draft) + row * a.draft_stride * size;
      alike = ((reinterpret_cast<uintptr_t>(r.p) ^ reinterpret_cast<uintptr_t>(r.q)) & 15) == 0;
    } else if (fallen >= 0 && fallen < a.vocab) {
      r.without = fallen;
    }
  }
  r.m = alike ? static_cast<int>(reinterpret_cast<uintptr_t>(r.p) & 15) / size : 0;
  r.p -= r.m * size;
  if (r.q) r.q -= r.m * size;
  r.full0 = r.m > 0;
  r.full1 = alike ? (a.vocab + r.m) / V : 0;
  // ---- sums of the warps' parts of the row; a part is 8 pieces
  const int slots = (a.vocab + r.m + V - 1) / V;
  const int parts = ctas * kWarps, mine = rank * kWarps + warp;
  const int piece = (slots + parts * kWarps - 1) / (parts * kWarps);
  const int64_t part_slots = static_cast<int64_t>(piece) * kWarps;
  const int lo = static_cast<int>(min(mine * part_slots, static_cast<int64_t>(slots)));
  const int hi = static_cast<int>(min((mine + 1) * part_slots, static_cast<int64_t>(slots)));
  uint64_t total = 0, border = 0;
  int owner = -1;       // the part that holds the border
  uint64_t before = 0;  // it
#pragma unroll 1
  for (int again = 0; again < 2; ++again) {
    constexpr int N = kSlots;
    uint64_t own = 0;
    Slot<DTYPE> now[N], next[N];
#pragma unroll
    for (int k = 0; k < N; ++k) now[k].load(r, lo + 32 * k + lane, hi);
#pragma unroll 1
    for (int j0 = lo; j0 < hi; j0 += 32 * N) {
#pragma unroll
      for (int k = 0; k < N; ++k) next[k].load(r, j0 + 32 * (N + k) + lane, hi);
#pragma unroll
      for (int k = 0; k < N; ++k) {
        uint64_t w[V];
        now[k].weights(r, j0 + 32 * k + lane, w);
#pragma unroll
        for (int e = 0; e < V; ++e) own += w[e];
        now[k] = next[k];
      }
    }
    __syncwarp();
    own = warp_sum(own);
    if (lane == 0) s_sums[warp] = own;
    cluster_sync_all();
    // The first warp looks for the border's part for all of them (each for itself takes
    // issue slots from the other CTAs: 37 sequences over 50021 tokens 7.4 us, so 7.1):
    // lane k has parts k and k + 32.
    if (warp == 0) {
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = lane + 32 * i;
        if (k < parts) {
          const uint32_t at = mapa_shared(&s_sums[k % kWarps], k / kWarps);
          asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(sum[i]) : "r"(at) : "memory");
        }
      }
      uint64_t cum[2] = {sum[0], sum[1]};
#pragma unroll
      for (int off = 1; off < 32; off <<= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint64_t up = __shfl_up_sync(0xffffffffu, cum[i], off);
          if (lane >= off) cum[i] += up;
        }
      const uint64_t first = __shfl_sync(0xffffffffu, cum[0], 31);
      total = first + __shfl_sync(0xffffffffu, cum[1], 31);
      border = part_of(last, total);
      const unsigned past = __ballot_sync(0xffffffffu, cum[0] > border);
      const unsigned late = __ballot_sync(0xffffffffu, cum[1] + first > border);
      owner = past ? __ffs(past) - 1 : 31 + __ffs(late);  // total 0: it is not looked at
      const uint64_t upto = past ? cum[0] - sum[0] : cum[1] - sum[1] + first;
      before = __shfl_sync(0xffffffffu, upto, owner & 31);
      if (lane == 0) s_found = {total, border, before, total > 0 ? owner : -1};
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // the sums have been read
    __syncthreads();
    total = s_found.total;
    border = s_found.border;
    before = s_found.before;
    owner = s_found.owner;
    if (total > 0) break;
    if (again) break;
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    r.q = nullptr;  // nothing is left of the difference: the target's own row
    r.without = -1;
  }
  // ---- the token: the warps of the owner's CTA take a piece of its part each
  if (owner >= 0 && owner / kWarps == rank) {
    const int end = static_cast<int>(min((owner + 1) * part_slots, static_cast<int64_t>(slots)));
    const int64_t from64 = owner * part_slots + static_cast<int64_t>(warp) * piece;
    const int from = static_cast<int>(min(from64, static_cast<int64_t>(end)));
    const int to = min(from + piece, end);
    // the first slots of a lane are kept for the search (all of them up to 64 a piece:
    // vocabularies of 130000 in fp32, 260000 in 16 bits)
    constexpr int K = 2;
    uint64_t w[K][V], sums[K], own = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      Slot<DTYPE> x;
      x.load(r, from + 32 * k + lane, to);
      x.weights(r, from + 32 * k + lane, w[k]);
      sums[k] = 0;
#pragma unroll
      for (int e = 0; e < V; ++e) sums[k] += w[k][e];
      own += sums[k];
    }
#pragma unroll 1
    for (int j = from + 32 * K + lane; j < to; j += 32) {
      Slot<DTYPE> x;
      uint64_t more[V];
      x.load(r, j, to);
      x.weights(r, j, more);
#pragma unroll
      for (int e = 0; e < V; ++e) own += more[e];
    }
    __syncwarp();
    own = warp_sum(own);
    __shared__ uint64_t s_piece[kWarps];
    if (lane == 0) s_piece[warp] = own;
    __syncthreads();
    for (int k = 0; k < warp; ++k) before += s_piece[k];
    if (before <= border && border < before + own) {
      // whether the border lies in the 32 slots from j on
      auto search = [&](int j, const uint64_t (&x)[V], uint64_t sum) {
        uint64_t cum = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const uint64_t up = __shfl_up_sync(0xffffffffu, cum, off);
          if (lane >= off) cum += up;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + cum > border);
        if (past && lane == __ffs(past) - 1) {
          uint64_t upto = before + cum - sum;
          int e = 0;
#pragma unroll
          for (int k = 0; k < V; ++k) {
            upto += x[k];
            e += upto <= border;
          }
          a.out_tokens[row] = static_cast<int>(static_cast<int64_t>(j + lane) * V - r.m + e);
        }
        before += __shfl_sync(0xffffffffu, cum, 31);
        return past != 0;
      };
      bool found = false;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (!found) found = search(from + 32 * k, w[k], sums[k]);
#pragma unroll 1
      for (int j = from + 32 * K; j < to && !found; j += 32) {
        Slot<DTYPE> x;
        uint64_t more[V], sum = 0;
        x.load(r, j + lane, to);
        x.weights(r, j + lane, more);
#pragma unroll
        for (int e = 0; e < V; ++e) sum += more[e];
        __syncwarp();
        found = search(j, more, sum);
      }
    }
  }
  if (rank == 0) {
    for (int i = threadIdx.x; i <= n; i += kThreads) {
      if (i < n) {
        const int x = a.tokens[q0 + i + 1];
        if (x < 0 || x >= a.vocab) set_status(a.status, kStatusBadId);
        if (i < accepted) a.out_tokens[q0 + i] = x;
      }
      if (i > accepted) a.out_tokens[q0 + i] = -1;
    }
    if (threadIdx.x == 0) {
      a.accepted[b] = accepted;
      if (total == 0) a.out_tokens[row] = 0;
    }
  }
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // for the arrival above
}

template <int DTYPE>
cudaError_t run(const VerifyArgs &a, int ctas, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, verify_kernel<DTYPE>, a, ctas);
  return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs &a, int dtype, cudaStream_t s) {
  if (a.B == 0) return cudaSuccess;
  // CTAs of a sequence, 8 at most (a warp looks at 64 parts): fewer where there are
  // more sequences than one wave has room for, or not a slot for every thread.  us with
  // 8, 4, 2, 1 of them, fp32: 64 sequences of 131072 tokens 16.0, 20.1, 32.6, 58.6; 512
  // of 32000 50.6, 35.4, 29.4, 28.2; 1024 of 8192 81, 43, 29, 21; 64 of 1000 7.2,
  // 5.6, 4.9, 4.9; one of 32000 5.1, 5.7, 7.1, 10.7.
  const int slots = a.vocab / (dtype == MOE_DTYPE_FP32 ? 4 : 8);
  int ctas = 8;
  while (ctas > 1 && (static_cast<int64_t>(a.B) * ctas > 4 * num_sms() || ctas * kThreads > slots))
    ctas /= 2;
  if (dtype == MOE_DTYPE_FP32) return run<MOE_DTYPE_FP32>(a, ctas, s);
  if (dtype == MOE_DTYPE_BF16) return run<MOE_DTYPE_BF16>(a, ctas, s);
  return run<MOE_DTYPE_FP16>(a, ctas, s);
}

}  // namespace moe
