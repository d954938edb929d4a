// Causal attention of new tokens over a paged cache.
#include "batch.cuh"
#include "internal.h"
#include "rows.cuh"

namespace moex {

struct AttnArgs {
  BatchView b;
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;  // or nullptr
  int64_t ldq, ldo;
  float scale;
  int n_heads, group, window, out_f32;
};

// One warp a (token, query head): lane l holds features l*D/32 .. of q, of
// each key and of the output, and walks the keys with a running maximum and sum.
template <int CT, int D>
__global__ void __launch_bounds__(128) attend_rows_kernel(const AttnArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int P = D / 32;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (w >= static_cast<int64_t>(a.b.n_tokens) * a.n_heads) return;
  const int tok = static_cast<int>(w / a.n_heads), h = static_cast<int>(w % a.n_heads), hk = h / a.group;
  using E = RowElem<CT>;
  using T = typename E::T;
  const int b = seq_of_token(a.b, tok);
  float q[P], o[P], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    q[i] = E::get(static_cast<const T*>(a.q)[tok * a.ldq + static_cast<int64_t>(h) * D + lane * P + i]);
    o[i] = 0.f;
  }
  SeqView s{0, 0, 0, true};
  if (b >= 0) s = seq_view(a.b, b);
  if (s.bad && lane == 0) flag_status(a.b.status, DEV_BAD_BATCH);
  const int pos = b >= 0 ? s.ctx - s.n + (tok - s.first) : -1;
  for (int j = a.window > 0 ? max(pos - a.window + 1, 0) : 0; j <= pos; ++j) {
    const int page = page_of(a.b, b, j);
    if (page < 0) continue;
    const int64_t off = kv_offset(a.b, page, hk, j) + lane * P;
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) x += q[i] * E::get(static_cast<const T*>(a.k)[off + i]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x *= a.scale;
    const float mn = fmaxf(m, x);
    if (mn == -INFINITY) continue;
    const float c = expf(m - mn), p = expf(x - mn);
    l = l * c + p;
    m = mn;
#pragma unroll
    for (int i = 0; i < P; ++i) o[i] = o[i] * c + p * E::get(static_cast<const T*>(a.v)[off + i]);
  }
  const float inv = l > 0.f ? __fdiv_rn(1.f, l) : 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int64_t at = tok * a.ldo + static_cast<int64_t>(h) * D + lane * P + i;
    if (a.out_f32)
      static_cast<float*>(a.out)[at] = o[i] * inv;
    else
      static_cast<T*>(a.out)[at] = static_cast<T>(o[i] * inv);
  }
  if (a.lse && lane == 0) a.lse[w] = l > 0.f ? m + logf(l) : -INFINITY;
}

size_t paged_attention_ws_bytes(const moex_paged_kv*, const moex_batch*, int) { return 0; }

template <int CT, int D>
static cudaError_t attend_launch(const AttnArgs& a, cudaStream_t s) {
  const int64_t warps = static_cast<int64_t>(a.b.n_tokens) * a.n_heads;
  return launch_pdl(attend_rows_kernel<CT, D>, dim3(static_cast<unsigned>((warps + 3) / 4)), dim3(128), 0, s, a);
}

moex_status launch_paged_attention(const void* q, int64_t ldq, const moex_paged_kv* kv, const moex_batch* batch,
                                   int n_heads, float scale, int window, void* out, int out_type, int64_t ldo,
                                   float* lse, void*, cudaStream_t s) {
  uint32_t* status = device_status_ptr();
  if (!status) return MOEX_ECUDA;
  const AttnArgs a{batch_view(kv, batch, status), q, kv->k, kv->v, out, lse, ldq, ldo, scale, n_heads,
                   n_heads / kv->n_kv_heads, window, out_type == MOEX_F32};
  if (kv->type == MOEX_BF16)
    return cuda_status(kv->head_dim == 64 ? attend_launch<MOEX_BF16, 64>(a, s) : attend_launch<MOEX_BF16, 128>(a, s));
  return cuda_status(kv->head_dim == 64 ? attend_launch<MOEX_F16, 64>(a, s) : attend_launch<MOEX_F16, 128>(a, s));
}

}  // namespace moex
