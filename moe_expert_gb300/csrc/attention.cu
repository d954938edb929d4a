// Causal attention of new tokens over a paged cache: choice of the kernel, its
// workspace, and the joining of tiles that several CTAs worked on.
#include "attn.cuh"
#include "attn_launch.h"
#include "internal.h"

namespace moex {

// Tiles that ranges cut, one column of CTAs for each range that begins inside a
// tile and is the first to do so, a CTA for 32 rows: the partials in the order of
// their keys, FP32.  CTA c of the first kernel leaves its first tile in slot 2c
// when it begins inside it, and its last in slot 2c + 1 when it does not finish
// it.  Latency bounds this kernel, so the rows' weights of up to 32 partials are
// formed first and the partials then read independently of one another.
template <int CT, int D, int MT>
__global__ void __launch_bounds__(128) attend_join_kernel(const AttnArgs a) {
  constexpr int R = MT < 32 ? MT : 32, F = 32, V = D / 4, ITEMS = R * V / 128;
  __shared__ float2 ml[F][R];          // (maximum, sum), then (weight, sum)
  __shared__ float rescale[R], total[R], top[R];
  __shared__ float4 rows[R][V + 1];
  const int n_cta = gridDim.x, r0 = blockIdx.y * R;
  pdl_wait();
  pdl_launch_dependents();
  const RangeStart x = a.plan[blockIdx.x];
  if (x.u == 0 || r0 >= x.rows) return;  // begins with a tile, or has no units
  const int64_t u0 = x.tile_u + x.u;
  if (range_begin(range_of(u0 - 1, x.W, n_cta), x.W, n_cta) > x.tile_u) return;  // an earlier range cut it first
  const int c0 = static_cast<int>(range_of(x.tile_u, x.W, n_cta));
  // with fewer units than CTAs a range is one unit or none
  const bool sparse = x.W < n_cta;
  const int parts = sparse ? x.units : static_cast<int>(range_of(x.tile_u + x.units - 1, x.W, n_cta)) - c0 + 1;
  auto slot_of = [&](int f) -> int64_t {
    const int64_t c = sparse ? range_of(x.tile_u + f, x.W, n_cta) : c0 + f;
    return 2 * c + (f == 0 ? 1 : 0);
  };
  const int nr = min(R, x.rows - r0);
  const float* stats = a.part + static_cast<int64_t>(2 * n_cta) * MT * D;
  float4 acc[ITEMS];
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int f0 = 0; f0 < parts; f0 += F) {
    const int nf = min(F, parts - f0);
    for (int i = threadIdx.x; i < nf * R; i += 128)
      if (i % R < nr)
        ml[i / R][i % R] = *reinterpret_cast<const float2*>(stats + 2 * (slot_of(f0 + i / R) * MT + r0 + i % R));
    __syncthreads();
    if (threadIdx.x < nr) {
      const int r = threadIdx.x;
      const float old = f0 ? top[r] : -INFINITY;
      float m = old, l = 0.f;
      for (int f = 0; f < nf; ++f) m = fmaxf(m, ml[f][r].x);
      const float ref = m == -INFINITY ? 0.f : m;
      for (int f = 0; f < nf; ++f) {
        const float w = fast_exp2(ml[f][r].x - ref);
        l += w * ml[f][r].y;
        ml[f][r].x = w;
      }
      const float k = fast_exp2(old - ref);
      rescale[r] = k;
      total[r] = (f0 ? total[r] * k : 0.f) + l;
      top[r] = m;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int r = (threadIdx.x + 128 * k) % R;
      const float old = r < nr ? rescale[r] : 0.f;
      acc[k].x *= old, acc[k].y *= old, acc[k].z *= old, acc[k].w *= old;
    }
#pragma unroll 4
    for (int f = 0; f < nf; ++f) {
      const float* part = a.part + part_offset<MT, D>(slot_of(f0 + f), r0, 0);
#pragma unroll
      for (int k = 0; k < ITEMS; ++k) {
        const int i = threadIdx.x + 128 * k;  // columns 4 (i / R) of row i % R
        if (i % R < nr) {
          const float4 v = *reinterpret_cast<const float4*>(part + 4 * i);
          const float w = ml[f][i % R].x;
          acc[k].x += w * v.x, acc[k].y += w * v.y, acc[k].z += w * v.z, acc[k].w += w * v.w;
        }
      }
    }
    __syncthreads();
  }
  // by way of shared memory, so that a row is written in one piece
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int i = threadIdx.x + 128 * k;
    rows[i % R][i / R] = acc[k];
  }
  __syncthreads();
  const SeqView s = seq_view(a.b, x.b);
  for (int i = threadIdx.x; i < nr * V; i += 128) {
    const int r = i / V, row = x.t * MT + r0 + r;
    const float l = total[r], inv = l > 0.f ? __fdiv_rn(1.f, l) : 0.f;
    float4 v = rows[r][i % V];
    v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
    store_out4<CT>(a, row_offset(s, a.group, x.hk, row, a.ldo, D) + 4 * (i % V), v);
    if (a.lse && i % V == 0)
      a.lse[row_offset(s, a.group, x.hk, row, a.n_heads, 1)] = l > 0.f ? top[r] * LN2 + logf(l) : -INFINITY;
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

HeadGroup head_group(int n, int n_tokens) {
  const int64_t rows = static_cast<int64_t>(n) * n_tokens + TILE_MT;  // a tile's row indices may pass the last row
  const bool fits = n > 1 && rows * n < (int64_t(1) << 32);
  return {n, fits ? static_cast<uint32_t>(((int64_t(1) << 32) + n - 1) / n) : 0u};
}

template <int CT, int D>
cudaError_t launch_join(const AttnArgs& a, const AttnGrid& g, cudaStream_t s) {
  if (g.tile) return launch_pdl(attend_join_kernel<CT, D, TILE_MT>, dim3(g.ctas, TILE_MT / 32), dim3(128), 0, s, a);
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
                   window,
                   out_type == MOEX_F32,
                   head_group(n_heads / kv->n_kv_heads, batch->n_tokens)};
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
