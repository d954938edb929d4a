// A paged cache of Q8_0 blocks read back into pages of 16-bit values.
#include "batch.cuh"
#include "internal.h"
#include "kv_q8.cuh"
#include "rows.cuh"

namespace moex {

struct KvReadQ8Args {
  BatchView from, to;
  ScaleView sc;
  const int32_t* start;  // or nullptr
  const int8_t* k;
  const int8_t* v;
  void* k_out;
  void* v_out;
  int n_kv_heads, D;
};

constexpr int READ_THREADS = 128, READ_HEADS = 2;

// A thread has eight features of a position in READ_HEADS heads: its page and slot
// are looked up once, and the heads' reads (8 bytes and a scale, keys and values) are
// independent.  Neighbouring threads take neighbouring features, so stores are whole
// lines of 16 bytes a thread.  DRAM bounds it for many positions (4926 of 8 heads of
// 128 / 16384 of 8 heads of 64: 8.7 / 11.4 us, 87 / 67% of the copy rate; with heads of 64 the
// instructions too, 64% of the issue slots), the three reads
// one after the other (lengths, page, values) for few.  A position's page is asked for
// with the values of the one before (without, 256 threads: 9.4 / 12.1 us; with one head a
// thread 10.3 / 13.0, with four, not ahead, 10.0 / 12.4).
template <int CT>
__global__ void __launch_bounds__(READ_THREADS) kv_read_q8_kernel(const KvReadQ8Args a) {
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.x, most = min(a.from.table_width << a.from.page_shift, a.to.table_width << a.to.page_shift);
  const int said = a.from.ctx_len[b], from = a.start ? a.start[b] : 0;
  const int lo = max(from, 0), hi = clip(said, 0, most);
  if ((hi != said || lo != from) && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) flag_status(a.from.status, DEV_BAD_BATCH);
  const int vecs = a.D >> 3, step = READ_THREADS / vecs;  // positions of a CTA at a time
  const int at = threadIdx.x / vecs, c = 8 * (threadIdx.x - at * vecs);
  if (at >= step) return;
  const int64_t hop = static_cast<int64_t>(gridDim.y) * step;
  const int h0 = blockIdx.z * READ_HEADS;
  struct Place {
    int page, page_out;
  };
  auto place = [&](int64_t p) {
    return p < hi ? Place{page_of(a.from, b, static_cast<int>(p)), page_of(a.to, b, static_cast<int>(p))} : Place{-1, -1};
  };
  const int64_t p0 = static_cast<int64_t>(lo) + static_cast<int64_t>(blockIdx.y) * step + at;
  Place next = place(p0);
  for (int64_t p64 = p0; p64 < hi; p64 += hop) {
    const int p = static_cast<int>(p64);
    const Place now = next;
    const bool in_place = now.page >= 0 && now.page_out >= 0;
    uint2 q[READ_HEADS][2];
    __half d[READ_HEADS][2];
    if (in_place) {
      const int64_t in = kv_offset(a.from, now.page, h0, p) + c;
      const int64_t sc = scale_offset(a.sc, now.page, h0, p & ((1 << a.from.page_shift) - 1)) + c / QK;
#pragma unroll
      for (int n = 0; n < READ_HEADS; ++n) {
        const bool here = h0 + n < a.n_kv_heads;
        const int64_t i = here ? in + n * a.from.head_stride : in, s = here ? sc + n * a.sc.head_stride : sc;
        q[n][0] = *reinterpret_cast<const uint2*>(a.k + i), q[n][1] = *reinterpret_cast<const uint2*>(a.v + i);
        d[n][0] = a.sc.k[s], d[n][1] = a.sc.v[s];
      }
    }
    next = place(p64 + hop);  // under way with the values
    if (!in_place) continue;
    const int64_t out = kv_offset(a.to, now.page_out, h0, p) + c;
#pragma unroll
    for (int n = 0; n < READ_HEADS; ++n) {
      if (h0 + n >= a.n_kv_heads) break;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const float scale = __half2float(d[n][g]);
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = scale * byte_value(j < 4 ? q[n][g].x : q[n][g].y, j & 3);
        store8<CT>(g ? a.v_out : a.k_out, out + n * a.to.head_stride, f);
      }
    }
  }
}

moex_status launch_kv_read_q8(const moex_paged_kv_q8* src, int n_seqs, const int32_t* ctx_len, const int32_t* start,
                              const int32_t* table, int table_width, int64_t table_stride, const moex_paged_kv* dst,
                              const int32_t* dst_table, int dst_width, int64_t dst_table_stride, cudaStream_t s) {
  uint32_t* status = device_status_ptr();
  if (!status) return MOEX_ECUDA;
  const moex_paged_kv plane = q8_plane(src);
  moex_batch from{}, to{};
  from.n_seqs = to.n_seqs = n_seqs;
  from.ctx_len = to.ctx_len = ctx_len;
  from.page_table = table, from.table_width = table_width, from.table_stride = table_stride;
  to.page_table = dst_table, to.table_width = dst_width, to.table_stride = dst_table_stride;
  const KvReadQ8Args a{batch_view(&plane, &from, status), batch_view(dst, &to, status), scale_view(src), start,
                       static_cast<const int8_t*>(src->k), static_cast<const int8_t*>(src->v), dst->k, dst->v,
                       src->n_kv_heads, src->head_dim};
  const int step = READ_THREADS / (src->head_dim >> 3);
  const int64_t steps = (static_cast<int64_t>(table_width) * src->page_size + step - 1) / step;
  // a sequence's CTAs: all SMs several times over, shared among the sequences, whose lengths the host does not know.
  // Measured, 10 / 40 / 80 / 160 an SM: one sequence of 16384 among 63 of 100 220 / 90 / 57 / 48 us, one of 100000 alone,
  // heads of 64, 55.1 / 51.4 / 51.3 / 55.1.
  const int parts = (src->n_kv_heads + READ_HEADS - 1) / READ_HEADS;
  int64_t per = static_cast<int64_t>(sm_count()) * 80 / (static_cast<int64_t>(n_seqs) * parts);
  per = per < 8 ? 8 : per;
  const dim3 grid(static_cast<unsigned>(n_seqs), static_cast<unsigned>(steps < per ? steps : per),
                  static_cast<unsigned>(parts));
  return cuda_status(dst->type == MOEX_BF16
                         ? launch_pdl(kv_read_q8_kernel<MOEX_BF16>, grid, dim3(READ_THREADS), 0, s, a)
                         : launch_pdl(kv_read_q8_kernel<MOEX_F16>, grid, dim3(READ_THREADS), 0, s, a));
}

}  // namespace moex
