// Causal attention of new tokens over a paged cache: choice of the kernel, its
// workspace, and the joining of tiles that several CTAs worked on.
#include <algorithm>

#include "attn.cuh"
#include "attn_launch.h"
#include "internal.h"

namespace moex {

// Tiles that ranges cut, a CTA for each range that begins inside a
// tile of at most 16 rows and is the first to do so: the partials in the order of
// their keys, FP32.  CTA c of the first kernel leaves its first tile in slot 2c
// when it begins inside it, and its last in slot 2c + 1 when it does not finish
// it.  Latency bounds this kernel, so the rows' weights of up to 32 partials are
// formed first and the partials then read independently of one another.
constexpr int JOIN_ROWS = 16;

template <int CT, int D, int MT>
__global__ void __launch_bounds__(JOIN_ROWS * D / 4) attend_join_kernel(const AttnArgs a) {
  constexpr int R = JOIN_ROWS, F = 32, V = D / 4, WARPS = R * V / 32;  // a thread: four columns of a row
  __shared__ float weight[F][R + 1];
  __shared__ int slots[F];
  __shared__ float rescale[R], total[R], top[R];
  __shared__ float4 rows[R][V + 1];
  const int n_cta = gridDim.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const RangeStart x = a.plan[blockIdx.x];
  if (x.u == 0) return;  // begins with a tile, or has no units
  const int64_t u0 = x.tile_u + x.u;
  if (range_begin(range_of(u0 - 1, x.W, n_cta), x.W, n_cta) > x.tile_u) return;  // an earlier range cut it first
  const int c0 = static_cast<int>(range_of(x.tile_u, x.W, n_cta));
  // with fewer units than CTAs a range is one unit or none
  const bool sparse = x.W < n_cta;
  const int parts = sparse ? x.units : static_cast<int>(range_of(x.tile_u + x.units - 1, x.W, n_cta)) - c0 + 1;
  const int nr = min(R, x.rows);
  // thread: columns 4 (threadIdx.x / R) of one row, of every `ways`-th partial when the rows are few
  const int shift = nr > 8 ? 4 : nr > 4 ? 3 : nr > 2 ? 2 : nr - 1, ways = R >> shift;
  const int row = threadIdx.x & ((1 << shift) - 1), way = (threadIdx.x % R) >> shift;
  const float* stats = a.part + static_cast<int64_t>(2 * n_cta) * MT * D;
  const float* part = a.part + part_offset<MT, D>(0, row, 4 * (threadIdx.x / R));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int f0 = 0; f0 < parts; f0 += F) {
    const int nf = min(F, parts - f0);
    if (threadIdx.x < nf) {
      const int f = f0 + threadIdx.x;
      const int c = sparse ? static_cast<int>(range_of(x.tile_u + f, x.W, n_cta)) : c0 + f;
      slots[threadIdx.x] = 2 * c + (f == 0 ? 1 : 0);
    }
    __syncthreads();
    // a warp a row, a lane a partial
#pragma unroll 1
    for (int r = warp; r < nr; r += WARPS) {
      float2 p = make_float2(-INFINITY, 0.f);
      if (lane < nf)
        p = *reinterpret_cast<const float2*>(stats + 2 * (static_cast<int64_t>(slots[lane]) * MT + r));
      const float old = f0 ? top[r] : -INFINITY;
      float m = fmaxf(old, p.x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float ref = m == -INFINITY ? 0.f : m, wt = fast_exp2(p.x - ref);
      float l = wt * p.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      weight[lane][r] = wt;
      if (lane == 0) {
        const float k = fast_exp2(old - ref);
        rescale[r] = k;
        total[r] = (f0 ? total[r] * k : 0.f) + l;
        top[r] = m;
      }
    }
    __syncthreads();
    if (row < nr) {
      const float old = rescale[row];
      acc.x *= old, acc.y *= old, acc.z *= old, acc.w *= old;
#pragma unroll 4
      for (int f = way; f < nf; f += ways) {
        const float4 v = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(slots[f]) * MT * D);
        const float wt = weight[f][row];
        acc.x += wt * v.x, acc.y += wt * v.y, acc.z += wt * v.z, acc.w += wt * v.w;
      }
    }
    __syncthreads();
  }
  // by way of shared memory, so that a row is written in one piece
  rows[threadIdx.x % R][threadIdx.x / R] = acc;  // row + way << shift
  __syncthreads();
  const int r = threadIdx.x / V, c = threadIdx.x % V;
  if (r >= nr) return;
  const SeqView s{x.first, x.n, x.ctx, false};
  const float l = total[r], inv = l > 0.f ? __fdiv_rn(1.f, l) : 0.f;
  float4 v = rows[r][c];
  for (int y = 1; y < ways; ++y) {
    const float4 o = rows[r + (y << shift)][c];
    v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
  }
  v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
  store_out4<CT>(a, row_offset(s, a.group, x.hk, x.t * MT + r, a.ldo, D) + 4 * c, v);
  if (a.lse && c == 0)
    a.lse[row_offset(s, a.group, x.hk, x.t * MT + r, a.n_heads, 1)] = row_lse(top[r], l);
}

// The same for tiles of many rows, which few ranges cut: a thread has 16 columns
// of a row, and reads two partials of them, with their statistics, at a time.  blockIdx.y: 32 rows.
template <int CT, int D, int MT>
__global__ void __launch_bounds__(2 * D) attend_join_rows_kernel(const AttnArgs a) {
  const int n_cta = gridDim.x;
  pdl_wait();
  pdl_launch_dependents();
  const RangeStart x = a.plan[blockIdx.x];
  const int r = blockIdx.y * 32 + threadIdx.x % 32, c0 = 16 * (threadIdx.x / 32);
  if (x.u == 0 || r >= x.rows) return;  // begins with a tile, or has no units
  const int64_t u0 = x.tile_u + x.u;
  if (range_begin(range_of(u0 - 1, x.W, n_cta), x.W, n_cta) > x.tile_u) return;  // an earlier range cut it first
  const int first = static_cast<int>(range_of(x.tile_u, x.W, n_cta));
  const bool sparse = x.W < n_cta;  // a range is one unit or none
  const int parts = sparse ? x.units : static_cast<int>(range_of(x.tile_u + x.units - 1, x.W, n_cta)) - first + 1;
  const float* stats = a.part + static_cast<int64_t>(2 * n_cta) * MT * D;
  float acc[16], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll 1
  for (int f0 = 0; f0 < parts; f0 += 2) {
    float2 ml[2];
    float4 v[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int f = f0 + k;
      ml[k] = make_float2(-INFINITY, 0.f);
      if (f < parts) {
        const int c = sparse ? static_cast<int>(range_of(x.tile_u + f, x.W, n_cta)) : first + f;
        const int64_t slot = 2 * static_cast<int64_t>(c) + (f == 0 ? 1 : 0);
        ml[k] = *reinterpret_cast<const float2*>(stats + 2 * (slot * MT + r));
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[k][j] = *reinterpret_cast<const float4*>(a.part + part_offset<MT, D>(slot, r, c0 + 4 * j));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[k][j] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    const float mn = fmaxf(m, fmaxf(ml[0].x, ml[1].x)), ref = mn == -INFINITY ? 0.f : mn;
    const float k0 = fast_exp2(m - ref), w0 = fast_exp2(ml[0].x - ref), w1 = fast_exp2(ml[1].x - ref);
    m = mn;
    l = l * k0 + w0 * ml[0].y + w1 * ml[1].y;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      acc[4 * j] = acc[4 * j] * k0 + w0 * v[0][j].x + w1 * v[1][j].x;
      acc[4 * j + 1] = acc[4 * j + 1] * k0 + w0 * v[0][j].y + w1 * v[1][j].y;
      acc[4 * j + 2] = acc[4 * j + 2] * k0 + w0 * v[0][j].z + w1 * v[1][j].z;
      acc[4 * j + 3] = acc[4 * j + 3] * k0 + w0 * v[0][j].w + w1 * v[1][j].w;
    }
  }
  const SeqView s{x.first, x.n, x.ctx, false};
  const float inv = l > 0.f ? __fdiv_rn(1.f, l) : 0.f;
  const int64_t off = row_offset(s, a.group, x.hk, x.t * MT + r, a.ldo, D) + c0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = acc[8 * h + i] * inv;
    if (a.out_f32)
      store8<MOEX_F32>(a.out, off + 8 * h, o);
    else
      store8<CT>(a.out, off + 8 * h, o);
  }
  if (a.lse && c0 == 0)
    a.lse[row_offset(s, a.group, x.hk, x.t * MT + r, a.n_heads, 1)] = row_lse(m, l);
}

namespace {

// CTAs of a launch and its workspace: their range starts, then two partial tiles each.
struct AttnGrid {
  bool tile;  // the tcgen05 kernel of 256-row tiles
  bool cut;   // ranges may cut tiles
  int ctas, mt;
  size_t plan_bytes, bytes;
};

AttnGrid grid_of(const moex_paged_kv* kv, const moex_batch* b, int n_heads, int window) {
  AttnGrid g;
  g.tile = static_cast<int64_t>(b->max_q) * (n_heads / kv->n_kv_heads) >
           (kv->head_dim == 64 ? TILE_MIN_ROWS_64 : TILE_MIN_ROWS);
  g.mt = g.tile ? TILE_MT : STREAM_MT;
  g.ctas = (g.tile ? 1 : STREAM_CTAS_PER_SM) * sm_count();
  // The most keys that a tile can see, as far as the host knows.
  int64_t keys = static_cast<int64_t>(b->table_width) * kv->page_size;
  if (window > 0) keys = std::min(keys, static_cast<int64_t>(window) + b->max_q);
  // Short tiles are left whole: no second kernel and no workspace (two launches cost the
  // host about 2 us more than one), against ranges that are less equal.  Measured, device
  // time cut / whole: streaming, heads of 128, 64 sequences of up to 250 keys 14.8 / 11.7 us,
  // 300 keys 15.2 / 13.0, 500 keys 16.9 / 14.8, one sequence of 250 keys 8.7 / 7.2, 500 keys
  // 9.3 / 10.2; heads of 64, 64 sequences of up to 500 keys 14.1 / 11.8, 600 keys 14.8 / 13.3,
  // one of 500 8.3 / 7.4.  Large tiles, 0.5 a CTA,
  // 250 keys 18.1 / 13.8, 550 keys 20.7 / 19.1, 1250 keys 23.7 / 29.6; 1.9 a CTA, 600 keys
  // 36.1 / 33.2, 1300 keys 47.0 / 51.2; 3.5 a CTA, 1600 keys 82.3 / 79.6.
  if (g.tile) {
    const int64_t rows = static_cast<int64_t>(b->n_tokens) * (n_heads / kv->n_kv_heads);
    const int64_t tiles = kv->n_kv_heads * std::max<int64_t>(b->n_seqs, rows / TILE_MT);
    g.cut = keys > 384 && keys * g.ctas > 512 * tiles;
  } else {
    g.cut = keys * kv->head_dim > 288 * 128;
  }
  g.plan_bytes = g.bytes = 0;
  if (!g.cut) return g;
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
  if (g.tile)
    return launch_pdl(attend_join_rows_kernel<CT, D, TILE_MT>, dim3(g.ctas, TILE_MT / 32), dim3(2 * D), 0, s, a);
  return launch_pdl(attend_join_kernel<CT, D, STREAM_MT>, dim3(g.ctas), dim3(JOIN_ROWS * D / 4), 0, s, a);
}

}  // namespace

size_t paged_attention_ws_bytes(const moex_paged_kv* kv, const moex_batch* batch, int n_heads) {
  return grid_of(kv, batch, n_heads, 0).bytes;
}

moex_status launch_paged_attention(const void* q, int64_t ldq, const moex_paged_kv* kv, const moex_batch* batch,
                                   int n_heads, float scale, int window, void* out, int out_type, int64_t ldo,
                                   float* lse, void* ws, cudaStream_t s) {
  uint32_t* status = device_status_ptr();
  if (!status) return MOEX_ECUDA;
  if (window >= 1 << 30) window = 0;  // sees every position, and position - window may leave 32 bits
  const AttnGrid g = grid_of(kv, batch, n_heads, window);
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
                   g.cut,
                   head_group(n_heads / kv->n_kv_heads, batch->n_tokens)};
  const cudaError_t e = g.tile ? launch_attend_tile(a, kv->type, kv->head_dim, g.ctas, s)
                               : launch_attend_stream(a, kv->type, kv->head_dim, g.ctas, s);
  if (e != cudaSuccess) return MOEX_ECUDA;
  if (!g.cut) return MOEX_OK;
  if (kv->type == MOEX_BF16)
    return cuda_status(kv->head_dim == 64 ? launch_join<MOEX_BF16, 64>(a, g, s)
                                          : launch_join<MOEX_BF16, 128>(a, g, s));
  return cuda_status(kv->head_dim == 64 ? launch_join<MOEX_F16, 64>(a, g, s)
                                        : launch_join<MOEX_F16, 128>(a, g, s));
}

}  // namespace moex
