// New tokens into a paged cache: rotary embedding of queries and keys, keys
// and values to their slots, queries to a packed buffer.
#include "batch.cuh"
#include "internal.h"
#include "rows.cuh"

namespace moex {

struct KvWriteArgs {
  BatchView b;
  const void* qkv;
  const float* cos_sin;
  void* q;
  void* k;
  void* v;
  int64_t ld, ldq;
  int n_heads, n_kv_heads, D, rot, interleaved, n_pos;
};

// One CTA a token; a thread takes 16 features of a head at a time.  In the
// half-split form those are features j .. j+7 and j + rot/2 .. j + rot/2 + 7,
// so a pair's two members meet in one thread; otherwise 16 in a row.
template <int TYPE, int CT>
__global__ void __launch_bounds__(256) kv_write_kernel(const KvWriteArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int tok = blockIdx.x;
  const int per_head = a.D >> 4, rot_units = a.rot >> 4, half = a.rot >> 1;
  const int units = (a.n_heads + 2 * a.n_kv_heads) * per_head;
  float x[8], y[8];
  // feature offsets of a unit's two groups of eight, and their values
  auto fetch = [&](int u, int& h, int& j, int& i0, int& i1) {
    h = u / per_head, j = u - h * per_head;
    const bool split = j < rot_units && !a.interleaved;
    i0 = split ? 8 * j : 16 * j;
    i1 = split ? half + 8 * j : 16 * j + 8;
    load8<TYPE>(a.qkv, tok * a.ld + static_cast<int64_t>(h) * a.D + i0, x);
    load8<TYPE>(a.qkv, tok * a.ld + static_cast<int64_t>(h) * a.D + i1, y);
  };
  int h, j, i0, i1, u = threadIdx.x;
  if (u < units) fetch(u, h, j, i0, i1);  // under way while the token's place is looked up

  const int b = seq_of_token(a.b, tok);
  int pos = -1, page = -1;
  bool bad = b < 0;
  if (b >= 0) {
    const SeqView s = seq_view(a.b, b);
    pos = s.ctx - s.n + (tok - s.first);
    bad = s.bad || (a.rot > 0 && pos >= a.n_pos);
    if (bad) pos = -1;
    if (pos >= 0) page = page_of(a.b, b, pos);
  }
  if (bad && threadIdx.x == 0) flag_status(a.b.status, DEV_BAD_BATCH);

  while (u < units) {
    const bool is_q = h < a.n_heads, is_v = h >= a.n_heads + a.n_kv_heads;
    const bool turn = !is_v && j < rot_units;
    if (pos < 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.f;
    }
    if (turn && pos >= 0) {
      float c[8], s[8];
      load8<MOEX_F32>(a.cos_sin, static_cast<int64_t>(pos) * a.rot + 8 * j, c);
      load8<MOEX_F32>(a.cos_sin, static_cast<int64_t>(pos) * a.rot + half + 8 * j, s);
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = x[2 * i], r = x[2 * i + 1], p2 = y[2 * i], r2 = y[2 * i + 1];
          x[2 * i] = p * c[i] - r * s[i];
          x[2 * i + 1] = r * c[i] + p * s[i];
          y[2 * i] = p2 * c[4 + i] - r2 * s[4 + i];
          y[2 * i + 1] = r2 * c[4 + i] + p2 * s[4 + i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = x[i], r = y[i];
          x[i] = p * c[i] - r * s[i];
          y[i] = r * c[i] + p * s[i];
        }
      }
    }
    if (is_q) {
      const int64_t off = tok * a.ldq + static_cast<int64_t>(h) * a.D;
      store8<CT>(a.q, off + i0, x);
      store8<CT>(a.q, off + i1, y);
    } else if (page >= 0) {
      const int64_t off = kv_offset(a.b, page, is_v ? h - a.n_heads - a.n_kv_heads : h - a.n_heads, pos);
      store8<CT>(is_v ? a.v : a.k, off + i0, x);
      store8<CT>(is_v ? a.v : a.k, off + i1, y);
    }
    u += blockDim.x;
    if (u < units) fetch(u, h, j, i0, i1);
  }
}

template <int TYPE>
static cudaError_t write_launch(const KvWriteArgs& a, int ct, cudaStream_t s) {
  const int units = (a.n_heads + 2 * a.n_kv_heads) * (a.D / 16);
  // Many tokens: small CTAs, so that more tokens' look-ups and rows are under way.
  const int most = a.b.n_tokens > 2 * sm_count() ? 128 : 256;
  const dim3 grid(a.b.n_tokens), block(units < most ? (units + 31) / 32 * 32 : most);
  return ct == MOEX_BF16 ? launch_pdl(kv_write_kernel<TYPE, MOEX_BF16>, grid, block, 0, s, a)
                         : launch_pdl(kv_write_kernel<TYPE, MOEX_F16>, grid, block, 0, s, a);
}

moex_status launch_rope_kv_write(const void* qkv, int type, int64_t ld, const moex_paged_kv* kv,
                                 const moex_batch* batch, int n_heads, const float* cos_sin, int64_t n_pos,
                                 int rot_dim, int interleaved, void* q, int64_t ldq, cudaStream_t s) {
  uint32_t* status = device_status_ptr();
  if (!status) return MOEX_ECUDA;
  const KvWriteArgs a{batch_view(kv, batch, status), qkv, cos_sin, q, kv->k, kv->v, ld, ldq, n_heads, kv->n_kv_heads,
                      kv->head_dim, rot_dim, interleaved, static_cast<int>(n_pos)};
  switch (type) {
    case MOEX_BF16: return cuda_status(write_launch<MOEX_BF16>(a, kv->type, s));
    case MOEX_F16: return cuda_status(write_launch<MOEX_F16>(a, kv->type, s));
    default: return cuda_status(write_launch<MOEX_F32>(a, kv->type, s));
  }
}

}  // namespace moex
