// prefix_attention.cu -- attention of a batch that shares a long prefix
// (moe_prefix_attention).
#include "elem.cuh"
#include "kernels.h"

namespace moe {
namespace {

// One warp per (token, query head): the keys of the prefix, then the
// sequence's own up to the token's causal limit, with a running maximum and
// sum (all fp32).
template <int DTYPE, int D>
__global__ void __launch_bounds__(128) attention_simple_kernel(const PrefixAttnArgs a) {
  pdl_begin();
  constexpr int E = D / 32;  // elements per lane
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int t = static_cast<int>(item / a.hq), h = static_cast<int>(item % a.hq);
  if (t >= a.T) return;
  const int kvh = h / (a.hq / a.hkv);
  const int page_size = 1 << a.page_shift;
  // the token's sequence and the rows of its own that it sees
  int b = t, limit = 0;
  if (a.q_offsets) {
    int lo = 0, hi = a.B;  // last b with q_offsets[b] <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.q_offsets[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    b = lo;
  }
  if (b < a.B) {
    const int q0 = a.q_offsets ? a.q_offsets[b] : b;
    const int q1 = a.q_offsets ? a.q_offsets[b + 1] : b + 1;
    const int len = a.kv_lens[b], cap = a.max_pages << a.page_shift;
    if (len < 0 || len > cap || q1 - q0 > a.max_q || q1 > a.T)
      set_status(a.status, kStatusBadId);
    limit = t >= q0 && t < q1 ? min(max(len, 0), cap) - (q1 - q0) + (t - q0) + 1 : 0;
    limit = max(limit, 0);
  }
  float q[E], o[E], m = -INFINITY, l = 0.0f;
  const uint16_t *qr = static_cast<const uint16_t *>(a.q) + t * a.q_stride + h * D;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = load1<DTYPE>(qr, lane * E + e) * a.scale;
    o[e] = 0.0f;
  }
  for (int part = 0; part < 2; ++part) {
    const int n = part == 0 ? a.prefix_len : limit;
    const int32_t *pages =
        part == 0 ? a.prefix_pages : a.page_table + static_cast<int64_t>(b) * a.max_pages;
    for (int j = 0; j < n; ++j) {
      int page = pages[j >> a.page_shift];
      if (page < 0 || page >= a.num_pages) {
        set_status(a.status, kStatusBadId);
        page = 0;
      }
      const int64_t row =
          (((static_cast<int64_t>(page) * a.hkv + kvh) << a.page_shift) + (j & (page_size - 1))) * D;
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(q[e], load1<DTYPE>(a.k_cache, row + lane * E + e), s);
#pragma unroll
      for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      const float m1 = fmaxf(m, s), c = expf(m - m1), p = expf(s - m1);
      m = m1;
      l = fmaf(l, c, p);
#pragma unroll
      for (int e = 0; e < E; ++e)
        o[e] = fmaf(o[e], c, p * load1<DTYPE>(a.v_cache, row + lane * E + e));
    }
  }
  uint16_t *orow = static_cast<uint16_t *>(a.o) + t * a.o_stride + h * D;
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    reinterpret_cast<uint32_t *>(orow)[(lane * E + e) / 2] =
        pack2<DTYPE>(o[e] * inv, o[e + 1] * inv);
  if (a.lse && lane == 0) a.lse[static_cast<int64_t>(t) * a.hq + h] = l > 0.0f ? m + logf(l) : -INFINITY;
}

template <int DTYPE>
cudaError_t run(const PrefixAttnArgs &a, cudaStream_t s) {
  const int64_t items = static_cast<int64_t>(a.T) * a.hq;
  const unsigned ctas = static_cast<unsigned>((items + 3) / 4);
  if (a.D == 64)
    MOE_LAUNCH_PDL(attention_simple_kernel<DTYPE, 64>, ctas, 128, 0, s, a);
  else
    MOE_LAUNCH_PDL(attention_simple_kernel<DTYPE, 128>, ctas, 128, 0, s, a);
  return cudaGetLastError();
}

}  // namespace

size_t prefix_attention_scratch_bytes(int, int, int, int, int, int, int) { return 0; }

cudaError_t launch_prefix_attention(const PrefixAttnArgs &a, int dtype, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  return dtype == MOE_DTYPE_BF16 ? run<MOE_DTYPE_BF16>(a, s) : run<MOE_DTYPE_FP16>(a, s);
}

}  // namespace moe
