// Causal attention of new tokens over a paged cache: choice of the kernel, its
// workspace, and the joining of tiles that several CTAs worked on.
#include "attn.cuh"
#include "attn_launch.h"
#include "internal.h"

namespace moex {

// Tiles that ranges cut, one column of CTAs for each range that begins inside a
// tile and is the first to do so: the partials in the order of their keys, FP32.
// CTA c leaves its first tile in slot 2c when it begins inside it, and its last
// in slot 2c + 1 when it does not finish it.
template <int CT, int D, int MT>
__global__ void __launch_bounds__(128) attend_join_kernel(const AttnArgs a) {
  const int n_cta = gridDim.x;
  pdl_wait();
  pdl_launch_dependents();
  const RangeStart x = a.plan[blockIdx.x];
  if (x.u == 0) return;  // begins with a tile, or has no units
  const int64_t u0 = x.tile_u + x.u;
  const int c0 = static_cast<int>(range_of(x.tile_u, x.W, n_cta));
  if (range_begin(range_of(u0 - 1, x.W, n_cta), x.W, n_cta) > x.tile_u) return;  // an earlier range cut it first
  const int c1 = static_cast<int>(range_of(x.tile_u + x.units - 1, x.W, n_cta));
  const SeqView s = seq_view(a.b, x.b);
  const float* ml = a.part + static_cast<int64_t>(2 * n_cta) * MT * D;
  constexpr int V = D / 4;
  for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < x.rows * V; i += gridDim.y * blockDim.x) {
    const int r = i / V, c4 = 4 * (i % V);
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0; c <= c1; ++c) {
      if (range_begin(c, x.W, n_cta) == range_begin(c + 1, x.W, n_cta)) continue;  // no units, no partial
      const int64_t slot = 2 * static_cast<int64_t>(c) + (c == c0 ? 1 : 0), at = slot * MT + r;
      const float2 p = *reinterpret_cast<const float2*>(ml + 2 * at);
      const float4 v = *reinterpret_cast<const float4*>(a.part + part_offset<MT, D>(slot, r, c4));
      const float mn = fmaxf(m, p.x), ref = mn == -INFINITY ? 0.f : mn;
      const float f0 = fast_exp2(m - ref), f1 = fast_exp2(p.x - ref);
      m = mn;
      l = l * f0 + p.y * f1;
      acc.x = acc.x * f0 + v.x * f1, acc.y = acc.y * f0 + v.y * f1;
      acc.z = acc.z * f0 + v.z * f1, acc.w = acc.w * f0 + v.w * f1;
    }
    const float inv = l > 0.f ? __fdiv_rn(1.f, l) : 0.f;
    acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
    store_out4<CT>(a, row_offset(s, a.group, x.hk, x.t * MT + r, a.ldo, D) + c4, acc);
    if (a.lse && c4 == 0)
      a.lse[row_offset(s, a.group, x.hk, x.t * MT + r, a.n_heads, 1)] = l > 0.f ? m * LN2 + logf(l) : -INFINITY;
  }
}

namespace {

// CTAs of a launch and its workspace: their range starts, then two partial tiles each.
struct AttnGrid {
  bool tile;  // the tcgen05 kernel of 256-row tiles
  int ctas, mt;
  size_t plan_bytes, bytes;
};

AttnGrid grid_of(const moex_paged_kv* kv, const moex_batch* b, int n_heads) {
  AttnGrid g;
  g.tile = static_cast<int64_t>(b->max_q) * (n_heads / kv->n_kv_heads) > TILE_MIN_ROWS;
  g.mt = g.tile ? TILE_MT : STREAM_MT;
  g.ctas = (g.tile ? 1 : STREAM_CTAS_PER_SM) * sm_count();
  g.plan_bytes = (g.ctas * sizeof(RangeStart) + 255) / 256 * 256;
  g.bytes = g.plan_bytes + static_cast<size_t>(2 * g.ctas) * g.mt * (kv->head_dim + 2) * 4;
  return g;
}

template <int CT, int D>
cudaError_t launch_join(const AttnArgs& a, const AttnGrid& g, cudaStream_t s) {
  if (g.tile) return launch_pdl(attend_join_kernel<CT, D, TILE_MT>, dim3(g.ctas, 8), dim3(128), 0, s, a);
  return launch_pdl(attend_join_kernel<CT, D, STREAM_MT>, dim3(g.ctas), dim3(128), 0, s, a);
}

}  // namespace

size_t paged_attention_ws_bytes(const moex_paged_kv* kv, const moex_batch* batch, int n_heads) {
  return grid_of(kv, batch, n_heads).bytes;
}

moex_status launch_paged_attention(const void* q, int64_t ldq, const moex_paged_kv* kv, const moex_batch* batch,
                                   int n_heads, float scale, int window, void* out, int out_type, int64_t ldo,
                                   float* lse, void* ws, cudaStream_t s) {
  uint32_t* status = device_status_ptr();
  if (!status) return MOEX_ECUDA;
  const AttnGrid g = grid_of(kv, batch, n_heads);
  const AttnArgs a{batch_view(kv, batch, status),
                   q,
                   kv->k,
                   kv->v,
                   out,
                   lse,
                   static_cast<RangeStart*>(ws),
                   reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + g.plan_bytes),
                   ldq,
                   ldo,
                   scale * 1.4426950408889634f,
                   n_heads,
                   kv->n_kv_heads,
                   n_heads / kv->n_kv_heads,
                   window,
                   out_type == MOEX_F32};
  const cudaError_t e = g.tile ? launch_attend_tile(a, kv->type, kv->head_dim, g.ctas, s)
                               : launch_attend_stream(a, kv->type, kv->head_dim, g.ctas, s);
  if (e != cudaSuccess) return MOEX_ECUDA;
  if (kv->type == MOEX_BF16)
    return cuda_status(kv->head_dim == 64 ? launch_join<MOEX_BF16, 64>(a, g, s)
                                          : launch_join<MOEX_BF16, 128>(a, g, s));
  return cuda_status(kv->head_dim == 64 ? launch_join<MOEX_F16, 64>(a, g, s)
                                        : launch_join<MOEX_F16, 128>(a, g, s));
}

}  // namespace moex
