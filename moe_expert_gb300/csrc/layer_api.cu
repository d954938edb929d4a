// C entry points of the operators around a layer's products (norm, expert
// routing, cache write, paged attention): argument validation on the host,
// then launches on the caller's stream.
#include <cuda_runtime.h>

#include <cmath>

#include "attn_launch.h"
#include "common.cuh"
#include "internal.h"

using namespace moex;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool known_type(int t) { return t == MOEX_F32 || t == MOEX_BF16 || t == MOEX_F16; }
// Rows are read four elements at a time: 16 bytes of FP32, 8 bytes of a 16-bit type.
uintptr_t row_align(int type) { return type == MOEX_F32 ? 16 : 8; }

moex_status check_kv(const moex_paged_kv* kv) {
  if (!kv || !kv->k || !kv->v) return MOEX_EINVAL;
  if (kv->type != MOEX_BF16 && kv->type != MOEX_F16) return MOEX_EUNSUPPORTED;
  if (kv->n_kv_heads < 1 || kv->n_kv_heads > 1024 || kv->n_pages < 1 || kv->n_pages > INT32_MAX) return MOEX_EINVAL;
  if (kv->head_dim < 1 || kv->page_stride < 0 || kv->head_stride < 0 || kv->row_stride < 0) return MOEX_EINVAL;
  if (kv->page_size < 8 || kv->page_size > 1024 || (kv->page_size & (kv->page_size - 1)) != 0)
    return MOEX_EUNSUPPORTED;
  if (kv->page_stride % 8 != 0 || kv->head_stride % 8 != 0 || kv->row_stride % 8 != 0) return MOEX_EALIGN;
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return MOEX_EALIGN;
  return MOEX_OK;
}

moex_status check_batch(const moex_paged_kv* kv, const moex_batch* b) {
  if (!b || !b->cu_q || !b->ctx_len || !b->page_table) return MOEX_EINVAL;
  if (b->n_seqs < 1 || b->n_seqs > (1 << 16) || b->n_tokens < 1 || b->n_tokens > (1 << 24)) return MOEX_EINVAL;
  if (b->max_q < 1 || b->max_q > b->n_tokens) return MOEX_EINVAL;
  if (b->table_width < 1 || b->table_stride < 0) return MOEX_EINVAL;
  // positions are 32-bit
  if (static_cast<int64_t>(b->table_width) * kv->page_size > (int64_t(1) << 30)) return MOEX_EUNSUPPORTED;
  return MOEX_OK;
}

}  // namespace

extern "C" {

moex_status moex_add_rms_norm(const void* x, int x_type, int64_t ldx, const float* residual, int64_t ldr,
                              const float* gamma, float eps, int T, int64_t H, float* sum, int64_t lds, void* y,
                              int y_type, int64_t ldy, int8_t* q, float* ds, moex_stream stream) {
  if (!x || !gamma || (!sum && !y && !q) || (q == nullptr) != (ds == nullptr)) return MOEX_EINVAL;
  if (!known_type(x_type) || (y && !known_type(y_type))) return MOEX_EUNSUPPORTED;
  if (T < 1 || H < QK || H % QK != 0 || !(eps > 0.f) || !std::isfinite(eps)) return MOEX_EINVAL;
  if (H > 32768) return MOEX_EUNSUPPORTED;
  if (ldx < H || (residual && ldr < H) || (sum && lds < H) || (y && ldy < H)) return MOEX_EINVAL;
  if (ldx % 4 != 0 || (residual && ldr % 4 != 0) || (sum && lds % 4 != 0) || (y && ldy % 4 != 0)) return MOEX_EALIGN;
  if (!aligned(x, row_align(x_type)) || !aligned(gamma, 16) || !aligned(residual, 16) || !aligned(sum, 16))
    return MOEX_EALIGN;
  if ((y && !aligned(y, row_align(y_type))) || !aligned(q, 16) || !aligned(ds, 8)) return MOEX_EALIGN;
  return launch_add_rms_norm(x, x_type, ldx, residual, ldr, gamma, eps, T, H, sum, lds, y, y_type, ldy, q, ds, stream);
}

moex_status moex_dequantize_q8_1(const int8_t* q, const float* ds, int T, int64_t K, void* y, int y_type,
                                 moex_stream stream) {
  if (!q || !ds || !y) return MOEX_EINVAL;
  if (!known_type(y_type)) return MOEX_EUNSUPPORTED;
  if (T < 1 || K < QK || K % QK != 0 || K > (1 << 20)) return MOEX_EINVAL;
  if (T * K / 1024 >= INT32_MAX) return MOEX_EUNSUPPORTED;  // CTAs of 1024 values
  if (!aligned(q, 16) || !aligned(ds, 8) || !aligned(y, 16)) return MOEX_EALIGN;
  return launch_dequantize_q8_1(q, ds, T, K, y, y_type, stream);
}

moex_status moex_route_experts(const void* logits, int type, int64_t ldl, const float* bias, int T, int E, int k,
                               int score, int groups, int top_groups, int group_top, int renorm, float scale,
                               int32_t* ids, float* w, moex_stream stream) {
  if (!logits || !ids || !w) return MOEX_EINVAL;
  if (!known_type(type) || (score != MOEX_SCORE_SOFTMAX && score != MOEX_SCORE_SIGMOID)) return MOEX_EUNSUPPORTED;
  if (T < 1 || E < 1 || E > 1024 || k < 1 || k > 16 || ldl < E || !std::isfinite(scale)) return MOEX_EINVAL;
  if (groups < 1 || groups > 32 || E % groups != 0 || top_groups < 1 || top_groups > groups) return MOEX_EINVAL;
  if (group_top < 1 || group_top > 2 || group_top > E / groups || k > top_groups * (E / groups)) return MOEX_EINVAL;
  return launch_route_experts(logits, type, ldl, bias, T, E, k, score, groups, top_groups, group_top, renorm, scale,
                              ids, w, stream);
}

moex_status moex_rope_kv_write(const void* qkv, int type, int64_t ld, const moex_paged_kv* kv, const moex_batch* batch,
                               int n_heads, const float* cos_sin, int64_t n_pos, int rot_dim, int interleaved, void* q,
                               int64_t ldq, moex_stream stream) {
  moex_status st = check_kv(kv);
  if (st != MOEX_OK) return st;
  st = check_batch(kv, batch);
  if (st != MOEX_OK) return st;
  if (!qkv || !q || n_heads < 1 || n_heads > 4096) return MOEX_EINVAL;
  if (!known_type(type)) return MOEX_EUNSUPPORTED;
  if (kv->head_dim % 16 != 0 || kv->head_dim > 512 || rot_dim % 16 != 0) return MOEX_EUNSUPPORTED;
  if (rot_dim < 0 || rot_dim > kv->head_dim || (rot_dim > 0) != (cos_sin != nullptr)) return MOEX_EINVAL;
  if (rot_dim > 0 && (n_pos < 1 || n_pos > INT32_MAX)) return MOEX_EINVAL;
  if (ld < static_cast<int64_t>(n_heads + 2 * kv->n_kv_heads) * kv->head_dim) return MOEX_EINVAL;
  if (ldq < static_cast<int64_t>(n_heads) * kv->head_dim) return MOEX_EINVAL;
  if (ld % 8 != 0 || ldq % 8 != 0 || !aligned(qkv, 16) || !aligned(q, 16) || !aligned(cos_sin, 16))
    return MOEX_EALIGN;
  return launch_rope_kv_write(qkv, type, ld, kv, batch, n_heads, cos_sin, n_pos, rot_dim, interleaved, q, ldq, stream);
}

size_t moex_paged_attention_workspace_bytes(const moex_paged_kv* kv, const moex_batch* batch, int n_heads) {
  if (!kv || !batch || kv->n_kv_heads < 1 || n_heads < kv->n_kv_heads || batch->n_tokens < 1) return 0;
  return paged_attention_ws_bytes(kv, batch, n_heads);
}

moex_status moex_paged_attention(const void* q, int64_t ldq, const moex_paged_kv* kv, const moex_batch* batch,
                                 int n_heads, float scale, int window, void* out, int out_type, int64_t ldo, float* lse,
                                 void* ws, size_t ws_bytes, moex_stream stream) {
  moex_status st = check_kv(kv);
  if (st != MOEX_OK) return st;
  st = check_batch(kv, batch);
  if (st != MOEX_OK) return st;
  if (!q || !out || n_heads < 1 || n_heads % kv->n_kv_heads != 0 || n_heads / kv->n_kv_heads > 128)
    return MOEX_EINVAL;
  if (kv->head_dim != 64 && kv->head_dim != 128) return MOEX_EUNSUPPORTED;
  if (out_type != kv->type && out_type != MOEX_F32) return MOEX_EUNSUPPORTED;
  if (!(scale > 0.f) || !std::isfinite(scale) || window < 0) return MOEX_EINVAL;
  if (ldq < static_cast<int64_t>(n_heads) * kv->head_dim || ldo < static_cast<int64_t>(n_heads) * kv->head_dim)
    return MOEX_EINVAL;
  // row indices (token within its sequence, head of the group) are 32-bit, those of the last tile's end too
  if (static_cast<int64_t>(batch->n_tokens) * n_heads > INT32_MAX - 2 * TILE_MT) return MOEX_EUNSUPPORTED;
  const size_t need = paged_attention_ws_bytes(kv, batch, n_heads);
  if (ws_bytes < need || (need > 0 && !ws)) return MOEX_ENOSPACE;
  if (ldq % 8 != 0 || ldo % 8 != 0 || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(ws, 16))
    return MOEX_EALIGN;
  return launch_paged_attention(q, ldq, kv, batch, n_heads, scale, window, out, out_type, ldo, lse, ws, stream);
}

}  // extern "C"
