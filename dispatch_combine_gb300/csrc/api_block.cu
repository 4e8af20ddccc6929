// api_block.cu -- the C ABI of the operators around the layer (norms, cache
// append, shared-prefix attention, the 4-bit cache, drafts): argument validation
// and launches.
#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool aligned16(const void *p) { return aligned(p, 16); }

moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

bool known_dtype(int32_t t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_FP16; }

// a row tensor: present, 16-byte aligned, rows of d values that do not overlap
bool good_rows(const void *p, int64_t stride, int64_t d) {
  return p && aligned16(p) && stride >= d && stride % 8 == 0;
}

moe_status_t check_norm(const moe_norm_t *n) {
  if (!n || n->T < 0 || n->d < 8 || n->d > 16384 || n->d % 8 != 0) return MOE_ERR_INVALID_ARG;
  if (n->kind != MOE_NORM_RMS && n->kind != MOE_NORM_LAYER) return MOE_ERR_INVALID_ARG;
  if (!known_dtype(n->dtype)) return MOE_ERR_INVALID_ARG;
  if (!(n->eps >= 0.0f) || !std::isfinite(n->eps) || !std::isfinite(n->weight_offset))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe::NormArgs norm_args(const moe_norm_t &n) {
  moe::NormArgs a = {};
  a.T = n.T;
  a.d = n.d;
  a.kind = n.kind;
  a.eps = n.eps;
  a.w_off = n.weight_offset;
  return a;
}

int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

moe_status_t check_kv(const moe_kv_t *kv) {
  if (!kv || kv->num_q_heads <= 0 || kv->num_kv_heads <= 0 || kv->num_pages < 0 ||
      !known_dtype(kv->dtype) || kv->num_q_heads % kv->num_kv_heads != 0)
    return MOE_ERR_INVALID_ARG;
  if (kv->num_q_heads / kv->num_kv_heads > 128 || kv->num_q_heads > 16384 ||
      (kv->head_dim != 64 && kv->head_dim != 128) || kv->page_size < 16 || kv->page_size > 256 ||
      (kv->page_size & (kv->page_size - 1)) != 0)
    return MOE_ERR_UNSUPPORTED;
  const int64_t rows = static_cast<int64_t>(kv->num_pages) * kv->page_size;
  if (rows >= (int64_t{1} << 31) || rows * kv->num_kv_heads >= (int64_t{1} << 31))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

#define MOE_TRY(expr)                    \
  do {                                   \
    moe_status_t _st = (expr);           \
    if (_st != MOE_OK) return _st;       \
  } while (0)

// the workspace's first 256 bytes hold the status word; scratch follows
constexpr size_t kStatusBytes = 256;

moe_status_t check_ws(const void *ws, size_t ws_bytes, size_t need) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < need)
    return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

// Key numbers are int, and reach past a length by a tile and a block of tokens.
constexpr int64_t kMostKeys = (int64_t{1} << 31) - 1024;

moe_status_t check_attention(const moe_kv_t *kv, int32_t T, int32_t num_seqs, int32_t max_q,
                             int32_t prefix_len) {
  MOE_TRY(check_kv(kv));
  if (T < 0 || num_seqs < 0 || max_q < 1 || prefix_len < 0 || prefix_len > kMostKeys)
    return MOE_ERR_INVALID_ARG;
  if (num_seqs > 4096) return MOE_ERR_UNSUPPORTED;
  // units (blocks of tokens x key heads, at most T x heads of them) are counted in int
  if (static_cast<int64_t>(T) * kv->num_q_heads >= (int64_t{1} << 30)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// What both appends check, and their arguments for the kernel.
moe_status_t append_args(const moe_kv_t *kv, int32_t T, const void *q, int64_t q_stride,
                         const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                         const int32_t *positions, const int32_t *slots, const float *inv_freq,
                         int32_t rot_dim, int32_t style, void *k_cache, void *v_cache,
                         void *q_out, int64_t q_out_stride, void *ws, size_t ws_bytes,
                         moe::KvAppendArgs *out) {
  MOE_TRY(check_kv(kv));
  if (T < 0 || rot_dim < 0 || rot_dim > kv->head_dim || rot_dim % 16 != 0)
    return MOE_ERR_INVALID_ARG;
  if (style != MOE_ROPE_HALF && style != MOE_ROPE_PAIRS) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const int64_t wq = static_cast<int64_t>(kv->num_q_heads) * kv->head_dim;
  const int64_t wk = static_cast<int64_t>(kv->num_kv_heads) * kv->head_dim;
  if (!good_rows(k, k_stride, wk) || !good_rows(v, v_stride, wk) || !slots || !k_cache ||
      !v_cache || !aligned16(k_cache) || !aligned16(v_cache) || k_cache == v_cache)
    return MOE_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr)) return MOE_ERR_INVALID_ARG;
  if (q && (!good_rows(q, q_stride, wq) || !good_rows(q_out, q_out_stride, wq) ||
            (q == q_out && q_stride != q_out_stride)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(slots, 4)) return MOE_ERR_INVALID_ARG;
  if (rot_dim > 0 && (!positions || !inv_freq || !aligned(positions, 4) || !aligned(inv_freq, 4)))
    return MOE_ERR_INVALID_ARG;
  if (ws) MOE_TRY(check_ws(ws, ws_bytes, kStatusBytes));
  moe::KvAppendArgs &a = *out;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.positions = positions;
  a.slots = slots;
  a.inv_freq = inv_freq;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.q_out = q_out;
  a.q_out_stride = q_out_stride;
  a.status = static_cast<uint32_t *>(ws);
  a.T = T;
  a.hq = kv->num_q_heads;
  a.hkv = kv->num_kv_heads;
  a.D = kv->head_dim;
  a.page_shift = log2_of(kv->page_size);
  a.rot = rot_dim;
  a.style = style;
  a.num_slots = static_cast<int64_t>(kv->num_pages) * kv->page_size;
  return MOE_OK;
}

// What both attentions check, and their arguments for the kernels but the
// workspace.
moe_status_t attention_args(const moe_kv_t *kv, int32_t T, int32_t num_seqs, int32_t max_q,
                            const void *q, int64_t q_stride, const int32_t *q_offsets,
                            const void *k_cache, const void *v_cache, const int32_t *prefix_pages,
                            int32_t prefix_len, const int32_t *page_table, int32_t max_pages,
                            const int32_t *kv_lens, float scale, void *o, int64_t o_stride,
                            float *lse, moe::PrefixAttnArgs *out) {
  MOE_TRY(check_attention(kv, T, num_seqs, max_q, prefix_len));
  if (max_pages < 0 || !(scale > 0.0f) || !std::isfinite(scale))
    return MOE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_pages) * kv->page_size > kMostKeys)
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!q_offsets && T != num_seqs) return MOE_ERR_INVALID_ARG;
  const int64_t wq = static_cast<int64_t>(kv->num_q_heads) * kv->head_dim;
  if (!good_rows(q, q_stride, wq) || !good_rows(o, o_stride, wq) || o == q)
    return MOE_ERR_INVALID_ARG;
  if (num_seqs > 0 && (!kv_lens || (max_pages > 0 && !page_table))) return MOE_ERR_INVALID_ARG;
  if (prefix_len > 0 && !prefix_pages) return MOE_ERR_INVALID_ARG;
  if (!aligned(q_offsets, 4) || !aligned(kv_lens, 4) || !aligned(lse, 4) ||
      (max_pages > 0 && !aligned(page_table, 4)) || (prefix_len > 0 && !aligned(prefix_pages, 4)))
    return MOE_ERR_INVALID_ARG;
  if ((prefix_len > 0 || max_pages > 0) &&
      (kv->num_pages == 0 || !k_cache || !v_cache || !aligned16(k_cache) || !aligned16(v_cache)))
    return MOE_ERR_INVALID_ARG;
  moe::PrefixAttnArgs &a = *out;
  a.q = q;
  a.q_stride = q_stride;
  a.q_offsets = q_offsets;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.prefix_pages = prefix_pages;
  a.prefix_len = prefix_len;
  a.page_table = page_table;
  a.max_pages = max_pages;
  a.kv_lens = kv_lens;
  a.scale = scale;
  a.o = o;
  a.o_stride = o_stride;
  a.lse = lse;
  a.T = T;
  a.B = num_seqs;
  a.max_q = max_q;
  a.hq = kv->num_q_heads;
  a.hkv = kv->num_kv_heads;
  a.D = kv->head_dim;
  a.page_shift = log2_of(kv->page_size);
  a.num_pages = kv->num_pages;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_norm_in(const moe_norm_t *norm, const void *x, int64_t x_stride,
                         const void *weight, const void *bias, void *out, int64_t out_stride,
                         moe_stream_t stream) {
  MOE_TRY(check_norm(norm));
  if (norm->T == 0) return MOE_OK;
  if (!good_rows(x, x_stride, norm->d) || !good_rows(out, out_stride, norm->d) ||
      !aligned16(weight) || !aligned16(bias))
    return MOE_ERR_INVALID_ARG;
  if (out == x && out_stride != x_stride) return MOE_ERR_INVALID_ARG;
  moe::NormArgs a = norm_args(*norm);
  a.f = x;
  a.f_stride = x_stride;
  a.nw = weight;
  a.nb = bias;
  a.n_out = out;
  a.n_out_stride = out_stride;
  return cuda_status(moe::launch_norm(a, norm->dtype, stream));
}

moe_status_t moe_norm_out(const moe_norm_t *norm, const void *f, int64_t f_stride, const void *x,
                          int64_t x_stride, int32_t post_norm, const void *post_weight,
                          const void *post_bias, int32_t gate_kind, const void *gate,
                          int64_t gate_stride, float residual_scale, const void *next_weight,
                          const void *next_bias, void *x_out, int64_t x_out_stride,
                          void *next_out, int64_t next_out_stride, moe_stream_t stream) {
  MOE_TRY(check_norm(norm));
  if (gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_FULL || !std::isfinite(residual_scale))
    return MOE_ERR_INVALID_ARG;
  if (norm->T == 0) return MOE_OK;
  const int64_t d = norm->d;
  if (!good_rows(f, f_stride, d) || !good_rows(x, x_stride, d) ||
      !good_rows(x_out, x_out_stride, d) || (next_out && !good_rows(next_out, next_out_stride, d)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(post_weight) || !aligned16(post_bias) || !aligned16(next_weight) ||
      !aligned16(next_bias))
    return MOE_ERR_INVALID_ARG;
  if (!post_norm && (post_weight || post_bias)) return MOE_ERR_INVALID_ARG;
  if (!next_out && (next_weight || next_bias)) return MOE_ERR_INVALID_ARG;
  if ((gate_kind == MOE_GATE_NONE) != (gate == nullptr)) return MOE_ERR_INVALID_ARG;
  if (gate_kind == MOE_GATE_FULL && !good_rows(gate, gate_stride, d)) return MOE_ERR_INVALID_ARG;
  if (gate_kind == MOE_GATE_CHANNEL && !aligned16(gate)) return MOE_ERR_INVALID_ARG;
  if (gate_kind == MOE_GATE_TOKEN && !aligned(gate, 2)) return MOE_ERR_INVALID_ARG;
  // in place only row for row
  if ((x_out == x && x_out_stride != x_stride) || x_out == f || x_out == next_out ||
      (next_out == f && next_out_stride != f_stride) || next_out == x)
    return MOE_ERR_INVALID_ARG;
  moe::NormArgs a = norm_args(*norm);
  a.f = f;
  a.f_stride = f_stride;
  a.x = x;
  a.x_stride = x_stride;
  a.post = post_norm != 0;
  a.pw = post_weight;
  a.pb = post_bias;
  a.gate_kind = gate_kind;
  a.gate = gate;
  a.gate_stride = gate_stride;
  a.residual_scale = residual_scale;
  a.nw = next_weight;
  a.nb = next_bias;
  a.x_out = x_out;
  a.x_out_stride = x_out_stride;
  a.n_out = next_out;
  a.n_out_stride = next_out_stride;
  return cuda_status(moe::launch_norm(a, norm->dtype, stream));
}

moe_status_t moe_kv_append(const moe_kv_t *kv, int32_t T, const void *q, int64_t q_stride,
                           const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                           const int32_t *positions, const int32_t *slots, const float *inv_freq,
                           int32_t rot_dim, int32_t style, void *k_cache, void *v_cache,
                           void *q_out, int64_t q_out_stride, void *ws, size_t ws_bytes,
                           moe_stream_t stream) {
  moe::KvAppendArgs a = {};
  MOE_TRY(append_args(kv, T, q, q_stride, k, k_stride, v, v_stride, positions, slots, inv_freq,
                      rot_dim, style, k_cache, v_cache, q_out, q_out_stride, ws, ws_bytes, &a));
  return cuda_status(moe::launch_kv_append(a, kv->dtype, stream));
}

moe_status_t moe_prefix_attention_workspace_size(const moe_kv_t *kv, int32_t T, int32_t num_seqs,
                                                 int32_t max_q, int32_t prefix_len,
                                                 size_t *bytes) {
  MOE_TRY(check_attention(kv, T, num_seqs, max_q, prefix_len));
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = kStatusBytes + moe::prefix_attention_scratch_bytes(T, num_seqs, max_q, kv->num_q_heads,
                                                              kv->num_kv_heads, kv->head_dim,
                                                              prefix_len);
  return MOE_OK;
}

moe_status_t moe_prefix_attention(const moe_kv_t *kv, int32_t T, int32_t num_seqs, int32_t max_q,
                                  const void *q, int64_t q_stride, const int32_t *q_offsets,
                                  const void *k_cache, const void *v_cache,
                                  const int32_t *prefix_pages, int32_t prefix_len,
                                  const int32_t *page_table, int32_t max_pages,
                                  const int32_t *kv_lens, float scale, void *o, int64_t o_stride,
                                  float *lse, void *ws, size_t ws_bytes, moe_stream_t stream) {
  moe::PrefixAttnArgs a = {};
  MOE_TRY(attention_args(kv, T, num_seqs, max_q, q, q_stride, q_offsets, k_cache, v_cache,
                         prefix_pages, prefix_len, page_table, max_pages, kv_lens, scale, o,
                         o_stride, lse, &a));
  if (T == 0) return MOE_OK;
  size_t need = 0;
  MOE_TRY(moe_prefix_attention_workspace_size(kv, T, num_seqs, max_q, prefix_len, &need));
  MOE_TRY(check_ws(ws, ws_bytes, need));
  a.status = static_cast<uint32_t *>(ws);
  a.scratch = static_cast<uint8_t *>(ws) + kStatusBytes;
  return cuda_status(moe::launch_prefix_attention(a, kv->dtype, stream));
}

size_t moe_kv4_page_bytes(const moe_kv_t *kv) {
  if (check_kv(kv) != MOE_OK) return 0;
  return static_cast<size_t>(kv->page_size) * (kv->head_dim / 2 + kv->head_dim / 16);
}

moe_status_t moe_kv4_append(const moe_kv_t *kv, int32_t T, const void *q, int64_t q_stride,
                            const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                            const int32_t *positions, const int32_t *slots,
                            const float *inv_freq, int32_t rot_dim, int32_t style,
                            void *k_cache, void *v_cache, void *q_out, int64_t q_out_stride,
                            void *ws, size_t ws_bytes, moe_stream_t stream) {
  moe::KvAppendArgs a = {};
  MOE_TRY(append_args(kv, T, q, q_stride, k, k_stride, v, v_stride, positions, slots, inv_freq,
                      rot_dim, style, k_cache, v_cache, q_out, q_out_stride, ws, ws_bytes, &a));
  return cuda_status(moe::launch_kv4_append(a, kv->dtype, stream));
}

moe_status_t moe_kv4_read(const moe_kv_t *kv, int32_t n, const int32_t *slots,
                          const void *k_cache, const void *v_cache, const int32_t *dst_slots,
                          int32_t dst_pages, void *k_out, int64_t k_out_stride, void *v_out,
                          int64_t v_out_stride, void *ws, size_t ws_bytes, moe_stream_t stream) {
  MOE_TRY(check_kv(kv));
  if (n < 0) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (!slots || !aligned(slots, 4) || !aligned(dst_slots, 4) || !k_cache || !v_cache ||
      !aligned16(k_cache) || !aligned16(v_cache) || k_out == v_out)
    return MOE_ERR_INVALID_ARG;
  const int64_t width = static_cast<int64_t>(kv->num_kv_heads) * kv->head_dim;
  if (dst_slots) {
    moe_kv_t dst = *kv;
    dst.num_pages = dst_pages;
    MOE_TRY(check_kv(&dst));
    if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)) return MOE_ERR_INVALID_ARG;
  } else if (!good_rows(k_out, k_out_stride, width) || !good_rows(v_out, v_out_stride, width)) {
    return MOE_ERR_INVALID_ARG;
  }
  if (ws) MOE_TRY(check_ws(ws, ws_bytes, kStatusBytes));
  moe::Kv4ReadArgs a = {};
  a.k_cache = static_cast<const uint8_t *>(k_cache);
  a.v_cache = static_cast<const uint8_t *>(v_cache);
  a.slots = slots;
  a.dst_slots = dst_slots;
  a.k_out = k_out;
  a.v_out = v_out;
  a.status = static_cast<uint32_t *>(ws);
  a.k_stride = k_out_stride;
  a.v_stride = v_out_stride;
  a.n = n;
  a.hkv = kv->num_kv_heads;
  a.D = kv->head_dim;
  a.page_shift = log2_of(kv->page_size);
  a.num_slots = static_cast<int64_t>(kv->num_pages) * kv->page_size;
  a.dst_num_slots = dst_slots ? static_cast<int64_t>(dst_pages) * kv->page_size : 0;
  return cuda_status(moe::launch_kv4_read(a, kv->dtype, stream));
}

moe_status_t moe_kv4_attention_workspace_size(const moe_kv_t *kv, int32_t T, int32_t num_seqs,
                                              int32_t max_q, size_t *bytes) {
  MOE_TRY(check_attention(kv, T, num_seqs, max_q, 0));
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = kStatusBytes + moe::kv4_attention_scratch_bytes(T, max_q, kv->num_q_heads,
                                                           kv->num_kv_heads, kv->head_dim);
  return MOE_OK;
}

moe_status_t moe_kv4_attention(const moe_kv_t *kv, int32_t T, int32_t num_seqs, int32_t max_q,
                               const void *q, int64_t q_stride, const int32_t *q_offsets,
                               const void *k_cache, const void *v_cache,
                               const int32_t *page_table, int32_t max_pages,
                               const int32_t *kv_lens, float scale, void *o, int64_t o_stride,
                               float *lse, void *ws, size_t ws_bytes, moe_stream_t stream) {
  moe::PrefixAttnArgs a = {};
  MOE_TRY(attention_args(kv, T, num_seqs, max_q, q, q_stride, q_offsets, k_cache, v_cache,
                         nullptr, 0, page_table, max_pages, kv_lens, scale, o, o_stride, lse, &a));
  if (T == 0) return MOE_OK;
  size_t need = 0;
  MOE_TRY(moe_kv4_attention_workspace_size(kv, T, num_seqs, max_q, &need));
  MOE_TRY(check_ws(ws, ws_bytes, need));
  a.status = static_cast<uint32_t *>(ws);
  a.scratch = static_cast<uint8_t *>(ws) + kStatusBytes;
  return cuda_status(moe::launch_kv4_attention(a, kv->dtype, stream));
}

moe_status_t moe_verify_drafts(int32_t T, int32_t num_seqs, int32_t vocab, int32_t dtype,
                               const void *target, int64_t target_stride, const void *draft,
                               int64_t draft_stride, const int32_t *tokens,
                               const float *uniforms, const int32_t *offsets, int32_t *accepted,
                               int32_t *out_tokens, void *ws, size_t ws_bytes,
                               moe_stream_t stream) {
  if (T < 0 || num_seqs < 0 || vocab < 1 || vocab > (1 << 30) ||
      (dtype != MOE_DTYPE_FP32 && !known_dtype(dtype)))
    return MOE_ERR_INVALID_ARG;
  if (num_seqs > (1 << 27)) return MOE_ERR_UNSUPPORTED;
  if (num_seqs == 0) return MOE_OK;
  const uintptr_t size = dtype == MOE_DTYPE_FP32 ? 4 : 2;
  if (!offsets || !accepted || !aligned(offsets, 4) || !aligned(accepted, 4))
    return MOE_ERR_INVALID_ARG;
  if (T > 0) {
    if (!target || !aligned(target, size) || target_stride < vocab || !tokens || !uniforms ||
        !out_tokens || !aligned(tokens, 4) || !aligned(uniforms, 4) || !aligned(out_tokens, 4) ||
        out_tokens == tokens || accepted == out_tokens || accepted == tokens)
      return MOE_ERR_INVALID_ARG;
    if (draft && (!aligned(draft, size) || draft_stride < vocab)) return MOE_ERR_INVALID_ARG;
  }
  if (ws) MOE_TRY(check_ws(ws, ws_bytes, kStatusBytes));
  moe::VerifyArgs a = {};
  a.target = target;
  a.draft = draft;
  a.tokens = tokens;
  a.offsets = offsets;
  a.uniforms = uniforms;
  a.accepted = accepted;
  a.out_tokens = out_tokens;
  a.status = static_cast<uint32_t *>(ws);
  a.target_stride = target_stride;
  a.draft_stride = draft_stride;
  a.T = T;
  a.B = num_seqs;
  a.vocab = vocab;
  return cuda_status(moe::launch_verify(a, dtype, stream));
}

}  // extern "C"
