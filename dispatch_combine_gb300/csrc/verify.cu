// verify.cu -- drafted tokens against the target's probabilities, from given
// uniform numbers (moe_verify_drafts).
//
//   draft x of row i stands iff u_i q_i(x) < p_i(x) and all before it stand;
//   the first that falls leaves the token to max(p_i - q_i, 0), none to p_n:
//   token = min { v : sum_{w <= v} r_w > u sum r }.
// One row of p and one of q are read for each sequence, by a cluster of CTAs.
//
// The sums are whole numbers: a weight in [0, 1] counts in units of 2^-60, so
// they are exact in any order (to 2^-60 a weight), and which token is the first
// past the border does not depend on how the row was cut.
#include "elem.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

template <int DTYPE>
__device__ __forceinline__ float prob_at(const void *p, int64_t i) {
  if (DTYPE == MOE_DTYPE_FP32) return static_cast<const float *>(p)[i];
  return load1<DTYPE>(p, i);
}
// a weight in [0, 1] in units of 2^-60 (NaN: 0)
__device__ __forceinline__ uint64_t units_of(float w) {
  w = fminf(fmaxf(w, 0.0f), 1.0f);
  const uint32_t b = __float_as_uint(w);
  const uint64_t m = (b & 0x7FFFFFu) | 0x800000u;
  const int up = static_cast<int>(b >> 23) - (127 + 23 - 60);
  if (up >= 0) return m << up;
  return up > -24 ? m >> -up : 0;
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
  const uint8_t *p, *q;  // of the row; q nullptr: p alone
  int without;           // token whose weight is 0 (-1: none)
  int vocab, m;
  bool vectors;          // both rows start alike
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
// The slots lane, lane + 32, ... (N of them from j0 on): their weights
template <int DTYPE, int N>
__device__ __forceinline__ void weights(const Row &r, int j0, int end, int lane,
                                        uint64_t (&w)[N][kVec<DTYPE>]) {
  constexpr int V = kVec<DTYPE>, SIZE = 16 / V;
  float p[N][V], q[N][V];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int j = j0 + k * 32 + lane;
    const int64_t v0 = static_cast<int64_t>(j) * V - r.m;
    if (r.vectors && j < end && v0 >= 0 && v0 + V <= r.vocab) {
      probs<DTYPE>(*reinterpret_cast<const uint4 *>(r.p + v0 * SIZE), p[k]);
      if (r.q) probs<DTYPE>(*reinterpret_cast<const uint4 *>(r.q + v0 * SIZE), q[k]);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int64_t v = v0 + e;
        const bool in = j < end && v >= 0 && v < r.vocab;
        p[k][e] = in ? prob_at<DTYPE>(r.p, v) : 0.0f;
        q[k][e] = in && r.q ? prob_at<DTYPE>(r.q, v) : 0.0f;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int64_t v = static_cast<int64_t>(j0 + k * 32 + lane) * V - r.m + e;
      w[k][e] = v == r.without ? 0 : units_of(r.q ? p[k][e] - q[k][e] : p[k][e]);
    }
}
__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

template <int DTYPE>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const VerifyArgs a, const int ctas) {
  pdl_begin();
  __shared__ uint64_t s_sums[kWarps];
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
        if (writer) set_status(a.status, kStatusBadId);
        falls = true;
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
           a.vocab, 0, true};
  r.m = static_cast<int>(reinterpret_cast<uintptr_t>(r.p) & 15) / size;
  if (accepted < n) {
    if (a.draft) {
      r.q = static_cast<const uint8_t *>(a.draft) + row * a.draft_stride * size;
      r.vectors = ((reinterpret_cast<uintptr_t>(r.p) ^ reinterpret_cast<uintptr_t>(r.q)) & 15) == 0;
    } else {
      r.without = fallen;
    }
  }
  // ---- sums of the warps' parts of the row; a part is 8 pieces of whole warps
  const int slots = (a.vocab + r.m + V - 1) / V;
  const int parts = ctas * kWarps, mine = rank * kWarps + warp;
  const int piece = ((slots + parts * kWarps - 1) / (parts * kWarps) + 31) / 32 * 32;
  const int64_t part_slots = static_cast<int64_t>(piece) * kWarps;
  const int lo = static_cast<int>(min(mine * part_slots, static_cast<int64_t>(slots)));
  const int hi = static_cast<int>(min((mine + 1) * part_slots, static_cast<int64_t>(slots)));
  uint64_t total = 0, border = 0;
  int owner = -1;       // the part that holds the border
  uint64_t before = 0;  // it
#pragma unroll 1
  for (int again = 0; again < 2; ++again) {
    constexpr int N = 16 / V;  // as many elements in flight with either size
    uint64_t own = 0;
#pragma unroll 1
    for (int j0 = lo; j0 < hi; j0 += 32 * N) {
      uint64_t w[N][V];
      weights<DTYPE, N>(r, j0, hi, lane, w);
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) own += w[k][e];
    }
    __syncwarp();
    own = warp_sum(own);
    if (lane == 0) s_sums[warp] = own;
    cluster_sync_all();
    // every warp: lane k has parts k and k + 32
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = lane + 32 * i;
      if (k < parts) {
        const uint32_t at = mapa_shared(&s_sums[k % kWarps], k / kWarps);
        asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(sum[i]) : "r"(at) : "memory");
      }
    }
    __syncwarp();
    cluster_sync_all();  // the sums have been read
    const uint64_t first = warp_sum(sum[0]);
    total = first + warp_sum(sum[1]);
    if (total > 0) {
      border = part_of(a.uniforms[q1 - 1], total);
      uint64_t cum[2] = {sum[0], sum[1]};
#pragma unroll
      for (int off = 1; off < 32; off <<= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint64_t up = __shfl_up_sync(0xffffffffu, cum[i], off);
          if (lane >= off) cum[i] += up;
        }
      const unsigned past = __ballot_sync(0xffffffffu, cum[0] > border);
      const unsigned late = __ballot_sync(0xffffffffu, cum[1] + first > border);
      owner = past ? __ffs(past) - 1 : 31 + __ffs(late);
      const uint64_t upto = past ? cum[0] - sum[0] : cum[1] - sum[1] + first;
      before = __shfl_sync(0xffffffffu, upto, owner & 31);
      break;
    }
    r.q = nullptr;  // nothing is left of the difference: the target's own row
    r.without = -1;
    r.vectors = true;
  }
  // ---- the token: the warps of the owner's CTA take a piece of its part each
  if (owner >= 0 && owner / kWarps == rank) {
    const int end = static_cast<int>(min((owner + 1) * part_slots, static_cast<int64_t>(slots)));
    const int64_t from64 = owner * part_slots + static_cast<int64_t>(warp) * piece;
    const int from = static_cast<int>(min(from64, static_cast<int64_t>(end)));
    const int to = min(from + piece, end);
    uint64_t own = 0;
#pragma unroll 4
    for (int j0 = from; j0 < to; j0 += 32) {
      uint64_t w[1][V];
      weights<DTYPE, 1>(r, j0, to, lane, w);
#pragma unroll
      for (int e = 0; e < V; ++e) own += w[0][e];
    }
    __syncwarp();
    own = warp_sum(own);
    __shared__ uint64_t s_piece[kWarps];
    if (lane == 0) s_piece[warp] = own;
    __syncthreads();
    for (int k = 0; k < warp; ++k) before += s_piece[k];
    if (before <= border && border < before + own) {
#pragma unroll 1
      for (int j0 = from; j0 < to; j0 += 32) {
        uint64_t w[1][V];
        weights<DTYPE, 1>(r, j0, to, lane, w);
        __syncwarp();
        uint64_t mine4 = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) mine4 += w[0][e];
        uint64_t cum = mine4;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const uint64_t up = __shfl_up_sync(0xffffffffu, cum, off);
          if (lane >= off) cum += up;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + cum > border);
        if (past) {
          if (lane == __ffs(past) - 1) {
            uint64_t sum = before + cum - mine4;
            int e = 0;
#pragma unroll
            for (int k = 0; k < V; ++k) {
              sum += w[0][k];
              e += sum <= border;
            }
            a.out_tokens[row] = static_cast<int>(static_cast<int64_t>(j0 + lane) * V - r.m + e);
          }
          break;
        }
        before += __shfl_sync(0xffffffffu, cum, 31);
      }
    }
  }
  if (rank == 0) {
    for (int i = threadIdx.x; i <= n; i += kThreads) {
      if (i < accepted) a.out_tokens[q0 + i] = a.tokens[q0 + i + 1];
      if (i > accepted) a.out_tokens[q0 + i] = -1;
    }
    if (threadIdx.x == 0) {
      a.accepted[b] = accepted;
      if (total == 0) a.out_tokens[row] = 0;
    }
  }
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
  const int ctas = 8;  // a warp looks at 64 parts
  if (dtype == MOE_DTYPE_FP32) return run<MOE_DTYPE_FP32>(a, ctas, s);
  if (dtype == MOE_DTYPE_BF16) return run<MOE_DTYPE_BF16>(a, ctas, s);
  return run<MOE_DTYPE_FP16>(a, ctas, s);
}

}  // namespace moe
