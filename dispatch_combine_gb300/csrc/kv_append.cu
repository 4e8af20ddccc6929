// kv_append.cu -- append of new keys and values to the paged cache, with the
// position rotation of queries and keys on the way (moe_kv_append).
//
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = position * inv_freq
// Each element is read and written once, so the kernel is bound by HBM.  A
// token's angles are computed once and shared by its heads.
#include "elem.cuh"
#include "kernels.h"

namespace moe {
namespace {

// units per thread whose loads are in flight together: a prefill step of 16384
// tokens (64 + 8 heads of 128) takes 144 us with one, 124 with two, 109 with
// four (671 MB: 6.1 TB/s, 0.91 of the measured copy bandwidth)
constexpr int kAppendUnroll = 4;

// One CTA per token.  Its work is cut into units of 16 elements (two 16-byte
// vectors): for the half style, vector c of the first half of the rotated
// part with vector c of its second half; otherwise, and in the part that is
// not rotated, two neighbouring vectors.  Units are numbered through the
// token's query heads, key heads, value heads.
template <int DTYPE>
__global__ void __launch_bounds__(512, 2) kv_append_kernel(const KvAppendArgs a) {
  pdl_begin();
  __shared__ float s_cos[64], s_sin[64];
  const int t = blockIdx.x;
  const int upr = a.D / 16;  // units per head row
  const int nq = a.q ? a.hq : 0;
  const int units = (nq + 2 * a.hkv) * upr;
  const int32_t slot = a.slots[t];
  const bool bad = slot < -1 || static_cast<int64_t>(slot) >= a.num_slots;
  const bool skip = slot < 0 || bad;
  if (bad && threadIdx.x == 0) set_status(a.status, kStatusBadId);
  const int half = a.rot / 2;
  const int64_t page = slot >> a.page_shift, in_page = slot & ((1 << a.page_shift) - 1);
  bool first = true;
  // (every thread passes the loop once, for the barrier inside)
  for (int base = threadIdx.x; first || base < units; base += blockDim.x * kAppendUnroll) {
    uint4 lo[kAppendUnroll], hi[kAppendUnroll];
    int head[kAppendUnroll], e0[kAppendUnroll], e1[kAppendUnroll];
#pragma unroll
    for (int j = 0; j < kAppendUnroll; ++j) {
      const int u = base + j * blockDim.x;
      lo[j] = hi[j] = make_uint4(0, 0, 0, 0);
      head[j] = u / upr;
      const int c = u - head[j] * upr;
      const bool rot_half = a.style == MOE_ROPE_HALF && 16 * c < a.rot && head[j] < nq + a.hkv;
      e0[j] = rot_half ? 8 * c : 16 * c;
      e1[j] = e0[j] + (rot_half ? half : 8);
      if (u >= units || (skip && head[j] >= nq)) continue;
      const uint16_t *row;
      if (head[j] < nq)
        row = static_cast<const uint16_t *>(a.q) + t * a.q_stride + head[j] * a.D;
      else if (head[j] < nq + a.hkv)
        row = static_cast<const uint16_t *>(a.k) + t * a.k_stride + (head[j] - nq) * a.D;
      else
        row = static_cast<const uint16_t *>(a.v) + t * a.v_stride + (head[j] - nq - a.hkv) * a.D;
      lo[j] = *reinterpret_cast<const uint4 *>(row + e0[j]);
      hi[j] = *reinterpret_cast<const uint4 *>(row + e1[j]);
    }
    if (first) {  // with the first units on their way
      first = false;
      for (int i = threadIdx.x; i < half; i += blockDim.x) {
        // turns = position * inv_freq / 2 pi, its fraction in fp64: two products
        // and the constant round at 2^-53 each, so up to 2^31 positions (3.4e8
        // turns at a frequency of 1) it is good to 1.2e-7 of a turn, 23 bits, and
        // up to 10^6 to 6e-11
        const double turns = static_cast<double>(a.positions[t]) * static_cast<double>(a.inv_freq[i]) *
                             0.15915494309189535;
        const float frac = static_cast<float>(turns - rint(turns));
        sincospif(2.0f * frac, &s_sin[i], &s_cos[i]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kAppendUnroll; ++j) {
      const int u = base + j * blockDim.x;
      if (u >= units || (skip && head[j] >= nq)) continue;
      const bool rotated = head[j] < nq + a.hkv && 16 * (u - head[j] * upr) < a.rot;
      if (rotated) {
        float x[8], y[8];
        unpack8<DTYPE>(lo[j], x);
        unpack8<DTYPE>(hi[j], y);
        if (a.style == MOE_ROPE_HALF) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float c = s_cos[e0[j] + e], s = s_sin[e0[j] + e];
            const float p = x[e] * c - y[e] * s, q = y[e] * c + x[e] * s;
            x[e] = p;
            y[e] = q;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const int i = (e0[j] + e) / 2;
            const float c0 = s_cos[i], s0 = s_sin[i], c1 = s_cos[i + 4], s1 = s_sin[i + 4];
            const float p0 = x[e] * c0 - x[e + 1] * s0, q0 = x[e + 1] * c0 + x[e] * s0;
            const float p1 = y[e] * c1 - y[e + 1] * s1, q1 = y[e + 1] * c1 + y[e] * s1;
            x[e] = p0;
            x[e + 1] = q0;
            y[e] = p1;
            y[e + 1] = q1;
          }
        }
        lo[j] = pack8<DTYPE>(x);
        hi[j] = pack8<DTYPE>(y);
      }
      uint16_t *row;
      if (head[j] < nq) {
        row = static_cast<uint16_t *>(a.q_out) + t * a.q_out_stride + head[j] * a.D;
      } else {
        const bool is_k = head[j] < nq + a.hkv;
        const int64_t h = head[j] - nq - (is_k ? 0 : a.hkv);
        row = static_cast<uint16_t *>(is_k ? a.k_cache : a.v_cache) +
              (((page * a.hkv + h) << a.page_shift) + in_page) * a.D;
      }
      *reinterpret_cast<uint4 *>(row + e0[j]) = lo[j];
      *reinterpret_cast<uint4 *>(row + e1[j]) = hi[j];
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs &a, int dtype, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  const int units = ((a.q ? a.hq : 0) + 2 * a.hkv) * (a.D / 16);
  int threads = (units + kAppendUnroll * 32 - 1) / (kAppendUnroll * 32) * 32;
  if (threads > 512) threads = 512;
  if (dtype == MOE_DTYPE_BF16)
    MOE_LAUNCH_PDL(kv_append_kernel<MOE_DTYPE_BF16>, static_cast<unsigned>(a.T), threads, 0, s, a);
  else
    MOE_LAUNCH_PDL(kv_append_kernel<MOE_DTYPE_FP16>, static_cast<unsigned>(a.T), threads, 0, s, a);
  return cudaGetLastError();
}

}  // namespace moe
