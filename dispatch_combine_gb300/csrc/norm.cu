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
//
// Bound by HBM where there are many rows: 16384 x 7168 bf16 moves 470 MB in
// 73 us (6.4 TB/s, 0.94 of the measured copy bandwidth) for one input and one
// output, 940 MB in 180 us (5.2 TB/s) for two and two, where the arithmetic of
// two norms comes near the issue rate.  A row per CTA, so that rows in flight,
// not barriers, set the rate; with few rows the launch is the time (3 us).
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

// Vectors of a weight as they lie in memory (zeros past d and where there is
// none), fetched before the sums that precede their use (a gate of each element
// of 16384 x 7168: 239 us where it is used, 189 so).  Biases are read where they
// are used: their registers cost more than the wait (norm_in of 16384 x 4096
// with a bias: 44 us, 63 with it fetched ahead).
template <int VPT>
__device__ __forceinline__ void fetch_vec(uint4 (&r)[VPT], const void *p, int vec0, int step,
                                          int nvec) {
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int i = vec0 + u * step;
    r[u] = p && i < nvec ? __ldg(static_cast<const uint4 *>(p) + i) : make_uint4(0, 0, 0, 0);
  }
}

// v <- N(v) * (w + off) + b on the row's registers (four pairs a vector).
// Elements past d are zero in v and stay out of the sums.  Two elements per
// instruction: moe_norm_out has some 20 instructions a pair, near the rate at
// which an SM issues them while HBM delivers the pair.
template <int DTYPE, int VPT, bool WARP_ROW>
__device__ __forceinline__ void normalise(uint64_t (&v)[VPT][4], const uint4 (&w)[VPT], bool has_w,
                                          const void *b, const NormArgs &a, int vec0, int step,
                                          int nvec, float *red0, float *red1) {
  const float inv_d = 1.0f / static_cast<float>(a.d);
  if (a.kind == MOE_NORM_LAYER) {
    uint64_t s[2] = {0, 0};
#pragma unroll
    for (int u = 0; u < VPT; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e & 1] = add_f32x2(s[e & 1], v[u][e]);
    const float2 t = unpack_f32x2(add_f32x2(s[0], s[1]));
    const float mean = row_sum<WARP_ROW>(t.x + t.y, red0) * inv_d;
    const uint64_t minus = pack_f32x2(-mean, -mean);
#pragma unroll
    for (int u = 0; u < VPT; ++u)
      if (vec0 + u * step < nvec) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[u][e] = add_f32x2(v[u][e], minus);
      }
  }
  uint64_t s[2] = {0, 0};
#pragma unroll
  for (int u = 0; u < VPT; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e & 1] = fma_f32x2(v[u][e], v[u][e], s[e & 1]);
  const float2 t = unpack_f32x2(add_f32x2(s[0], s[1]));
  const float rs = rsqrtf(row_sum<WARP_ROW>(t.x + t.y, red1) * inv_d + a.eps);
  const uint64_t rs2 = pack_f32x2(rs, rs), off2 = pack_f32x2(a.w_off, a.w_off);
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[u][e] = mul_f32x2(v[u][e], rs2);
    if (has_w) {
      uint64_t wf[4];
      unpack8x2<DTYPE>(w[u], wf);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[u][e] = mul_f32x2(v[u][e], add_f32x2(wf[e], off2));
    }
    const int i = vec0 + u * step;
    if (b && i < nvec) {
      uint64_t bf[4];
      unpack8x2<DTYPE>(__ldg(static_cast<const uint4 *>(b) + i), bf);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[u][e] = add_f32x2(v[u][e], bf[e]);
    }
  }
}

// The weights of a row pass: of the post norm, the gate (of the channels, or the
// row's own), the next norm.
template <int DTYPE, int VPT>
struct Weights {
  uint4 pw[VPT], cg[VPT], nw[VPT];
  __device__ __forceinline__ void fetch(const NormArgs &a, int64_t row, int vec0, int step,
                                        int nvec) {
    fetch_vec<VPT>(pw, a.x ? a.pw : nullptr, vec0, step, nvec);
    const bool full = a.gate_kind == MOE_GATE_FULL;
    const void *g = a.x && (full || a.gate_kind == MOE_GATE_CHANNEL)
                        ? static_cast<const uint16_t *>(a.gate) + (full ? row * a.gate_stride : 0)
                        : nullptr;
    fetch_vec<VPT>(cg, g, vec0, step, nvec);
    fetch_vec<VPT>(nw, a.nw, vec0, step, nvec);
  }
};

// The row in registers (fr: f's, or the input's; xr: x's) to its outputs.
template <int DTYPE, int VPT, bool WARP_ROW, bool TWO>
__device__ __forceinline__ void finish_row(const NormArgs &a, int64_t row, const uint4 (&fr)[VPT],
                                           const uint4 (&xr)[VPT], const Weights<DTYPE, VPT> &w, int vec0,
                                           int step, int nvec, float (*red)[32]) {
  uint64_t v[VPT][4];
#pragma unroll
  for (int u = 0; u < VPT; ++u) unpack8x2<DTYPE>(fr[u], v[u]);
  if (TWO) {
    if (a.post)
      normalise<DTYPE, VPT, WARP_ROW>(v, w.pw, a.pw != nullptr, a.pb, a, vec0, step, nvec, red[0],
                                      red[1]);
    const float tg = a.gate_kind == MOE_GATE_TOKEN ? load1<DTYPE>(a.gate, row) : 1.0f;
    const uint64_t tg2 = pack_f32x2(tg, tg), sc2 = pack_f32x2(a.residual_scale, a.residual_scale);
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int i = vec0 + u * step;
      if (i >= nvec) continue;
      uint64_t xf[4], gf[4] = {tg2, tg2, tg2, tg2};
      unpack8x2<DTYPE>(xr[u], xf);
      if (a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_FULL)
        unpack8x2<DTYPE>(w.cg[u], gf);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[u][e] = fma_f32x2(gf[e], v[u][e], mul_f32x2(sc2, xf[e]));
      reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.x_out) + row * a.x_out_stride)[i] =
          pack8x2<DTYPE>(v[u]);
    }
  }
  if (!a.n_out) return;
  normalise<DTYPE, VPT, WARP_ROW>(v, w.nw, a.nw != nullptr, a.nb, a, vec0, step, nvec, red[2],
                                  red[3]);
  uint4 *out = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.n_out) + row * a.n_out_stride);
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int i = vec0 + u * step;
    if (i < nvec) out[i] = pack8x2<DTYPE>(v[u]);
  }
}

// VPT 16-byte vectors per thread; a row per warp (d small) or per CTA.
template <int DTYPE, int VPT, bool WARP_ROW, bool TWO>
__global__ void __launch_bounds__(1024, 1) norm_kernel(const NormArgs a) {
  pdl_begin();
  __shared__ float red[4][32];
  const int64_t row =
      WARP_ROW ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= a.T) return;  // WARP_ROW: no barrier follows
  const int vec0 = WARP_ROW ? threadIdx.x & 31 : threadIdx.x;
  const int step = WARP_ROW ? 32 : blockDim.x;
  const int nvec = a.d / 8;
  const uint4 *f = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.f) +
                                                   row * a.f_stride);
  const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) +
                                                   row * a.x_stride);
  uint4 fr[VPT], xr[VPT];
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int i = vec0 + u * step;
    fr[u] = xr[u] = make_uint4(0, 0, 0, 0);
    if (i < nvec) {
      fr[u] = f[i];
      if (TWO) xr[u] = x[i];
    }
  }
  Weights<DTYPE, VPT> w;
  w.fetch(a, row, vec0, step, nvec);
  finish_row<DTYPE, VPT, WARP_ROW, TWO>(a, row, fr, xr, w, vec0, step, nvec, red);
}

template <int DTYPE, bool TWO>
cudaError_t run(const NormArgs &a, cudaStream_t s) {
  const int nvec = a.d / 8;
  if (nvec <= 64) {  // a row per warp, 8 rows per CTA
    const unsigned ctas = (static_cast<unsigned>(a.T) + 7u) / 8u;
    if (nvec <= 32)
      MOE_LAUNCH_PDL(norm_kernel<DTYPE, 1, true, TWO>, ctas, 256, 0, s, a);
    else
      MOE_LAUNCH_PDL(norm_kernel<DTYPE, 2, true, TWO>, ctas, 256, 0, s, a);
    return cudaGetLastError();
  }
  // vectors per thread: 16384 x 7168 bf16 takes 73 us with 4 and 84 with 2 for
  // one input, 207 and 180 for two (whose registers then leave fewer rows per SM)
  constexpr int kVpt = TWO ? 2 : 4;
  const int threads = (nvec + kVpt * 32 - 1) / (kVpt * 32) * 32;  // <= 1024
  MOE_LAUNCH_PDL(norm_kernel<DTYPE, kVpt, false, TWO>, static_cast<unsigned>(a.T), threads, 0, s, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, int dtype, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  if (dtype == MOE_DTYPE_BF16)
    return a.x ? run<MOE_DTYPE_BF16, true>(a, s) : run<MOE_DTYPE_BF16, false>(a, s);
  return a.x ? run<MOE_DTYPE_FP16, true>(a, s) : run<MOE_DTYPE_FP16, false>(a, s);
}

}  // namespace moe
