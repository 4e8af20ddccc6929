// norm.cu -- the norms before and after a block (moe_norm_in, moe_norm_out).
//
//   v     = post ? N(f) * (pw + off) + pb : f
//   r     = residual_scale * x + gate * v          (moe_norm_in: r = its input)
//   x_out = rn(r)
//   n_out = N(r) * (nw + off) + nb
// with N(v) = v / sqrt(mean(v^2) + eps) or its centred form.  A row is read
// once and stays in registers through both statistics, so the kernel moves
// each input and output row exactly once; everything is fp32 until the one
// rounding of each output.
#include "elem.cuh"
#include "kernels.h"

namespace moe {
namespace {

// Sum over the threads that hold one row: a warp, or the whole CTA (red: one
// float per warp; two arrays are used alternately, so that one barrier per
// sum is enough).
template <bool WARP_ROW>
__device__ __forceinline__ float row_sum(float v, float *red) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (WARP_ROW) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int nw = blockDim.x >> 5;
  float t = (threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int off = 16; off; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
  return t;
}

// N(v) * (w + off) + b on the row's registers.  Elements past d are zero in v
// and stay out of the sums.
template <int DTYPE, int VPT, bool WARP_ROW>
__device__ __forceinline__ void normalise(float (&v)[VPT][8], const void *w, const void *b,
                                          const NormArgs &a, int vec0, int step, int nvec,
                                          float *red0, float *red1) {
  const float inv_d = 1.0f / static_cast<float>(a.d);
  float mean = 0.0f;
  if (a.kind == MOE_NORM_LAYER) {
    float s = 0.0f;
#pragma unroll
    for (int u = 0; u < VPT; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[u][e];
    mean = row_sum<WARP_ROW>(s, red0) * inv_d;
  }
  float ss = 0.0f;
#pragma unroll
  for (int u = 0; u < VPT; ++u)
    if (vec0 + u * step < nvec) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[u][e] -= mean;
        ss = fmaf(v[u][e], v[u][e], ss);
      }
    }
  const float rs = rsqrtf(row_sum<WARP_ROW>(ss, red1) * inv_d + a.eps);
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int i = vec0 + u * step;
    if (i >= nvec) continue;
    float wf[8], bf[8];
    if (w) unpack8<DTYPE>(__ldg(static_cast<const uint4 *>(w) + i), wf);
    if (b) unpack8<DTYPE>(__ldg(static_cast<const uint4 *>(b) + i), bf);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[u][e] = fmaf(v[u][e] * rs, w ? wf[e] + a.w_off : 1.0f, b ? bf[e] : 0.0f);
  }
}

// VPT 16-byte vectors per thread; a row per warp (d small) or per CTA.
template <int DTYPE, int VPT, bool WARP_ROW>
__global__ void norm_kernel(const NormArgs a) {
  pdl_begin();
  __shared__ float red[4][32];
  const int row = WARP_ROW ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= a.T) return;  // WARP_ROW: no barrier follows
  const int vec0 = WARP_ROW ? threadIdx.x & 31 : threadIdx.x;
  const int step = WARP_ROW ? 32 : blockDim.x;
  const int nvec = a.d / 8;
  const uint16_t *f = static_cast<const uint16_t *>(a.f) + row * a.f_stride;
  const uint16_t *x = static_cast<const uint16_t *>(a.x) + row * a.x_stride;
  uint4 fr[VPT], xr[VPT];
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int i = vec0 + u * step;
    fr[u] = xr[u] = make_uint4(0, 0, 0, 0);
    if (i < nvec) {
      fr[u] = reinterpret_cast<const uint4 *>(f)[i];
      if (a.x) xr[u] = reinterpret_cast<const uint4 *>(x)[i];
    }
  }
  float v[VPT][8];
#pragma unroll
  for (int u = 0; u < VPT; ++u) unpack8<DTYPE>(fr[u], v[u]);
  if (a.x) {
    if (a.post)
      normalise<DTYPE, VPT, WARP_ROW>(v, a.pw, a.pb, a, vec0, step, nvec, red[0], red[1]);
    const float tg = a.gate_kind == MOE_GATE_TOKEN ? load1<DTYPE>(a.gate, row) : 1.0f;
    const uint16_t *g = static_cast<const uint16_t *>(a.gate) +
                        (a.gate_kind == MOE_GATE_FULL ? row * a.gate_stride : 0);
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int i = vec0 + u * step;
      if (i >= nvec) continue;
      float xf[8], gf[8];
      unpack8<DTYPE>(xr[u], xf);
#pragma unroll
      for (int e = 0; e < 8; ++e) gf[e] = tg;
      if (a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_FULL)
        unpack8<DTYPE>(reinterpret_cast<const uint4 *>(g)[i], gf);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[u][e] = fmaf(gf[e], v[u][e], a.residual_scale * xf[e]);
      reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.x_out) + row * a.x_out_stride)[i] =
          pack8<DTYPE>(v[u]);
    }
  }
  if (!a.n_out) return;
  normalise<DTYPE, VPT, WARP_ROW>(v, a.nw, a.nb, a, vec0, step, nvec, red[2], red[3]);
  uint4 *out = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.n_out) + row * a.n_out_stride);
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int i = vec0 + u * step;
    if (i < nvec) out[i] = pack8<DTYPE>(v[u]);
  }
}

template <int DTYPE>
cudaError_t run(const NormArgs &a, cudaStream_t s) {
  const int nvec = a.d / 8;
  if (nvec <= 64) {  // a row per warp, 8 rows per CTA
    const unsigned ctas = static_cast<unsigned>((a.T + 7) / 8);
    if (nvec <= 32)
      MOE_LAUNCH_PDL(norm_kernel<DTYPE, 1, true>, ctas, 256, 0, s, a);
    else
      MOE_LAUNCH_PDL(norm_kernel<DTYPE, 2, true>, ctas, 256, 0, s, a);
    return cudaGetLastError();
  }
  const int threads = (nvec + 4 * 32 - 1) / (4 * 32) * 32;  // <= 512
  MOE_LAUNCH_PDL(norm_kernel<DTYPE, 4, false>, static_cast<unsigned>(a.T), threads, 0, s, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, int dtype, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  return dtype == MOE_DTYPE_BF16 ? run<MOE_DTYPE_BF16>(a, s) : run<MOE_DTYPE_FP16>(a, s);
}

}  // namespace moe
