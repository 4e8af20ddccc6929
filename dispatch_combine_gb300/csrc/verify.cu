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

struct Row {
  const void *p, *q;  // of the row; q nullptr: p alone
  int without;        // token whose weight is 0 (-1: none)
};
template <int DTYPE>
__device__ __forceinline__ uint64_t weight(const Row &r, int v) {
  float w = prob_at<DTYPE>(r.p, v);
  if (r.q) w -= prob_at<DTYPE>(r.q, v);
  if (v == r.without) w = 0.0f;
  return units_of(w);
}

template <int DTYPE>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a, const int ctas) {
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
  const int64_t row = q0 + accepted;
  Row r = {static_cast<const uint8_t *>(a.target) + row * a.target_stride * size, nullptr, -1};
  if (accepted < n) {
    if (a.draft)
      r.q = static_cast<const uint8_t *>(a.draft) + row * a.draft_stride * size;
    else
      r.without = fallen;
  }
  // ---- sums of the warps' parts of the row
  const int parts = ctas * kWarps, mine = rank * kWarps + warp;
  const int length = ((a.vocab + parts - 1) / parts + 31) / 32 * 32;
  const int64_t from = static_cast<int64_t>(mine) * length;
  const int lo = static_cast<int>(min(from, static_cast<int64_t>(a.vocab)));
  const int hi = static_cast<int>(min(from + length, static_cast<int64_t>(a.vocab)));
  uint64_t total = 0, before = 0, own = 0;
#pragma unroll 1
  for (int again = 0; again < 2; ++again) {
    own = 0;
#pragma unroll 8
    for (int v = lo + lane; v < hi; v += 32) own += weight<DTYPE>(r, v);
#pragma unroll
    for (int off = 16; off; off >>= 1) own += __shfl_xor_sync(0xffffffffu, own, off);
    if (lane == 0) s_sums[warp] = own;
    cluster_sync_all();
    total = before = 0;
    for (int k = lane; k < parts; k += 32) {
      const uint32_t at = mapa_shared(&s_sums[k % kWarps], k / kWarps);
      uint64_t sum;
      asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(sum) : "r"(at) : "memory");
      total += sum;
      if (k < mine) before += sum;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, off);
      before += __shfl_xor_sync(0xffffffffu, before, off);
    }
    cluster_sync_all();  // the sums have been read
    if (total > 0) break;
    r.q = nullptr;  // nothing is left of the difference: the target's own row
    r.without = -1;
  }
  const uint64_t border = part_of(a.uniforms[q1 - 1], total);
  // ---- the token: in the part whose sums pass the border
  if (before <= border && border < before + own) {
    uint64_t sum = before;
    for (int v0 = lo; v0 < hi; v0 += 32) {
      const int v = v0 + lane;
      uint64_t cum = v < hi ? weight<DTYPE>(r, v) : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint64_t up = __shfl_up_sync(0xffffffffu, cum, off);
        if (lane >= off) cum += up;
      }
      const unsigned past = __ballot_sync(0xffffffffu, sum + cum > border);
      if (past) {
        if (lane == 0) a.out_tokens[row] = v0 + __ffs(past) - 1;
        break;
      }
      sum += __shfl_sync(0xffffffffu, cum, 31);
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
  const int ctas = 8;
  if (dtype == MOE_DTYPE_FP32) return run<MOE_DTYPE_FP32>(a, ctas, s);
  if (dtype == MOE_DTYPE_BF16) return run<MOE_DTYPE_BF16>(a, ctas, s);
  return run<MOE_DTYPE_FP16>(a, ctas, s);
}

}  // namespace moe
