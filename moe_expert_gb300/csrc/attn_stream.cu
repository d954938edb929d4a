// Paged attention for few rows a key head (single tokens, drafts): the cache
// is streamed once, so DRAM bounds it.
//
// A CTA of four warps works on one tile of 16 rows; each warp runs alone
// over every fourth step of 16 keys (32 with heads of 64: 8 KB of cache either
// way), with its own copies in flight (cp.async, no CTA barrier in the loop), its
// own running maximum and sum, and the products on mma.sync m16n8k16: with 16
// rows a step is 32 such instructions, far below the tensor rate, and tcgen05's
// 128-row tiles would be mostly empty.  The copies run on from one tile into the next;
// the four warps' results meet in shared memory at the end of a tile.
#include "attn.cuh"
#include "attn_launch.h"
#include "internal.h"

namespace moex {
namespace {

constexpr int MT = STREAM_MT, DEAD = STREAM_DEAD;
constexpr int WARPS = 4, STAGES = 2;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <int CT>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (CT == MOEX_BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Shared memory: each warp's two stages (K then V), and the warps' outputs
// [WARPS][MT][D + 4] with their maxima and sums at the end of a tile.
template <int D>
struct Smem {
  static constexpr int STEP = D == 64 ? 32 : 16;  // keys of a step
  static constexpr int UK = WARPS * STEP;         // keys of a unit: a step of every warp
  static constexpr int PLANE = STEP * D * 2;   // bytes of a step's keys
  static constexpr int RING = WARPS * STAGES * 2 * PLANE;
  static constexpr int PITCH = D + 4;          // floats of an output row
  static constexpr int BYTES = RING + WARPS * MT * (PITCH + 2) * 4;
};

// The keys of a tile that a CTA's range holds, as one warp sees them: steps
// k0 + i * UK .. + STEP - 1.
template <int STEP, int UK>
struct WarpKeys {
  int units, k0, end, steps;
  __device__ __forceinline__ WarpKeys(const AttnArgs& a, const Cursor& c, int warp) {
    units = units_here(a, c);
    const int first = c.x.lo + c.u * UK;
    end = min(c.x.hi, first + units * UK);
    k0 = first + warp * STEP;
    steps = end > k0 ? (end - k0 + UK - 1) / UK : 0;
  }
};

// The bound on registers is that of the two CTAs an SM gets: with what the compiler
// takes by itself (128 for heads of 64) a few spill.
template <int CT, int D>
__global__ void __launch_bounds__(WARPS * 32, STREAM_CTAS_PER_SM) attend_stream_kernel(const AttnArgs a) {
  extern __shared__ __align__(128) uint8_t sm[];
  using S = Smem<D>;
  using E = RowElem<CT>;
  constexpr int STEP = S::STEP, UK = S::UK, RUNS = STEP / 8;  // runs of eight keys, each inside one page
  using Keys = WarpKeys<STEP, UK>;
  constexpr int CH = D / 8;     // 16-byte chunks of a row
  constexpr int KS = D / 16;    // k-steps of the first product
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, p2 = 2 * (lane & 3);
  pdl_wait();
  pdl_launch_dependents();  // the joining kernel's CTAs take the place of these as they end, and wait
  Cursor cur;
  __shared__ RangeScratch<WARPS * 32> scratch;
  find_range<MT, UK, DEAD, WARPS * 32>(a, blockIdx.x, gridDim.x, cur, scratch);
  if (cur.left <= 0) return;
  const uint32_t ring = smem_u32(sm) + warp * STAGES * 2 * S::PLANE;

  // ---- copies: a cursor of their own, a step ahead of the products
  __shared__ Cursor ahead_of[WARPS];
  Cursor& ahead = ahead_of[warp];
  if (lane == 0) ahead = cur;
  __syncwarp();
  int l_i = 0, l_steps = 0, l_k0 = 0, l_end = 0, l_hk = 0;  // the tile that copies are issued for
  bool l_more = true;
  int pg[RUNS];  // lane l: pages of the runs of step 32 * (l_i / 32) + l
  const int32_t* l_table = nullptr;
  auto fetch_pages = [&]() {
    const int j = l_k0 + (l_i + lane) * UK;
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      const int k = j + 8 * r;
      pg[r] = k + 7 >= ahead.x.from && k < l_end ? __ldg(l_table + (k >> a.b.page_shift)) : 0;
    }
  };
  // the next tile in which this warp has a step; its pages are asked for at once
  auto seek = [&](bool fresh) {
    for (;; fresh = false) {
      if (!fresh) {
        const int units = Keys(a, ahead, warp).units;
        __syncwarp();
        if (lane == 0) next_tile<MT, UK, DEAD>(a, ahead, units);
        __syncwarp();
      }
      l_more = ahead.left > 0;
      if (!l_more) return;
      const Keys w(a, ahead, warp);
      if (w.steps == 0) continue;
      l_i = 0, l_steps = w.steps, l_k0 = w.k0, l_end = w.end, l_hk = ahead.hk;
      l_table = a.b.table + ahead.b * a.b.table_stride;
      fetch_pages();
      return;
    }
  };
  uint32_t ok_ring = 0;  // RUNS bits a stage: the step's runs have a page
  auto load = [&](int stage) {
    if (l_more) {
      const int j = l_k0 + l_i * UK;
      int page[RUNS];
      uint32_t ok = (1u << RUNS) - 1;
      bool good = true;
#pragma unroll
      for (int r = 0; r < RUNS; ++r) {
        page[r] = __shfl_sync(0xffffffffu, pg[r], l_i & 31);
        good = good && static_cast<uint32_t>(page[r]) < static_cast<uint32_t>(a.b.n_pages);
      }
      if (!good) {
        if (lane == 0) flag_status(a.b.status, DEV_BAD_BATCH);
#pragma unroll
        for (int r = 0; r < RUNS; ++r)
          if (static_cast<uint32_t>(page[r]) >= static_cast<uint32_t>(a.b.n_pages)) {
            page[r] = -1;
            ok &= ~(1u << r);
          }
      }
      ok_ring = (ok_ring & ~(((1u << RUNS) - 1) << (RUNS * stage))) | ok << (RUNS * stage);
      const uint32_t dst = ring + stage * 2 * S::PLANE;
      const int r0 = ahead.x.from - j, r1 = l_end - j;  // the step's rows that are there
      constexpr int RPI = 32 / CH;  // rows an instruction covers
      const int c = lane % CH;
#pragma unroll
      for (int n = 0; n < STEP / RPI; ++n) {
        // the run of an instruction's rows is known when this is compiled: RPI divides 8
        const int r = n * RPI + lane / CH, run = n * RPI / 8;
        // zeros in place of keys outside: a value beside a probability of 0 must be finite
        const bool in = r >= r0 && r < r1 && page[run] >= 0;
        const int64_t off = in ? kv_offset(a.b, page[run], l_hk, j + r) + 8 * c : 0;
        const uint32_t at = dst + r * (D * 2) + ((c ^ (r & 7)) << 4);
        cp_async16(at, static_cast<const uint16_t*>(a.k) + off, in ? 16u : 0u);
        cp_async16(at + S::PLANE, static_cast<const uint16_t*>(a.v) + off, in ? 16u : 0u);
      }
      if (++l_i == l_steps)
        seek(false);
      else if ((l_i & 31) == 0)
        fetch_pages();
    }
    cp_commit();
  };
  seek(true);
  load(0);
  int stage = 0;

  // Q as the A operand: rows g and g + 8 of the tile, the same for every step
  uint32_t qf[KS][4];
  auto load_q = [&]() {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = cur.x.r0 + g + 8 * half;
      const bool in = r < cur.x.r1;
      const uint16_t* row =
          static_cast<const uint16_t*>(a.q) + (in ? row_offset(cur.s, a.group, cur.hk, r, a.ldq, D) : 0);
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        qf[i][half] = in ? *reinterpret_cast<const uint32_t*>(row + 16 * i + p2) : 0u;
        qf[i][2 + half] = in ? *reinterpret_cast<const uint32_t*>(row + 16 * i + 8 + p2) : 0u;
      }
    }
  };
  load_q();

  while (cur.left > 0) {
    const Tile x = cur.x;
    const Keys w(a, cur, warp);
    const int base = cur.s.ctx - cur.s.n;
    int top[2], bot[2];  // keys bot < j <= top are seen by the row
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = x.r0 + g + 8 * half;
      top[half] = r < x.r1 ? base + a.group.token(r) : -1;
      bot[half] = a.window > 0 ? top[half] - a.window : -1;
    }

    // m: the row's reference, its maximum but for prob_up
    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    for (int i = 0; i < w.steps; ++i) {
      const uint32_t ok = (ok_ring >> (RUNS * stage)) & ((1u << RUNS) - 1);
      __syncwarp();  // the stage refilled next has been read by every lane
      load(stage ^ 1);
      cp_wait<1>();
      __syncwarp();  // every lane's copies have landed
      const uint32_t kb = ring + stage * 2 * S::PLANE, vb = kb + S::PLANE;
      float s[RUNS][4];
#pragma unroll
      for (int nt = 0; nt < RUNS; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < RUNS / 2; ++kk) {
        const int r = 16 * kk + (lane >> 4) * 8 + (lane & 7), c = (lane >> 3) & 1;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t f[4];
          ldsm4(f, kb + r * (D * 2) + (((2 * ks + c) ^ (r & 7)) << 4));
          mma16816<CT>(s[2 * kk], qf[ks], f[0], f[1]);
          mma16816<CT>(s[2 * kk + 1], qf[ks], f[2], f[3]);
        }
      }
      const int j = w.k0 + i * UK;
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nt = 0; nt < RUNS; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int half = e >> 1, key = j + 8 * nt + p2 + (e & 1);
          const bool seen = key <= top[half] && key > bot[half] && ((ok >> nt) & 1u);
          s[nt][e] = seen ? s[nt][e] * a.scale_log2 : -INFINITY;
          mx[half] = fmaxf(mx[half], s[nt][e]);
        }
      float corr[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        mx[half] = fmaxf(mx[half], __shfl_xor_sync(0xffffffffu, mx[half], 1));
        mx[half] = fmaxf(mx[half], __shfl_xor_sync(0xffffffffu, mx[half], 2));
        mx[half] = fmaxf(m[half], mx[half] - prob_up<CT>(0.f));
        // a row that has seen no key keeps 0 as its reference, so that -inf - -inf does not arise
        const float ref = mx[half] == -INFINITY ? 0.f : mx[half];
        corr[half] = fast_exp2(m[half] - ref);
        m[half] = mx[half];
        l[half] *= corr[half];
#pragma unroll
        for (int nt = 0; nt < RUNS; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float pv = fast_exp2(s[nt][2 * half + e] - ref);
            s[nt][2 * half + e] = pv;
            l[half] += pv;
          }
      }
      if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
        for (int i2 = 0; i2 < D / 8; ++i2) {
          o[i2][0] *= corr[0], o[i2][1] *= corr[0], o[i2][2] *= corr[1], o[i2][3] *= corr[1];
        }
      }
#pragma unroll
      for (int kk = 0; kk < RUNS / 2; ++kk) {
        // probabilities rounded to the cache type (attn.cuh): the A operand of the second product
        const uint32_t pf[4] = {E::pack(s[2 * kk][0], s[2 * kk][1]), E::pack(s[2 * kk][2], s[2 * kk][3]),
                                E::pack(s[2 * kk + 1][0], s[2 * kk + 1][1]),
                                E::pack(s[2 * kk + 1][2], s[2 * kk + 1][3])};
        const int r = 16 * kk + ((lane >> 3) & 1) * 8 + (lane & 7), c = lane >> 4;
#pragma unroll
        for (int nt = 0; nt < D / 16; ++nt) {
          uint32_t f[4];
          ldsm4_t(f, vb + r * (D * 2) + (((2 * nt + c) ^ (r & 7)) << 4));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float(&od)[4] = o[2 * nt + h];
            mma16816<CT>(od, pf, f[2 * h], f[2 * h + 1]);
          }
        }
      }
      stage ^= 1;
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
      l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
    }
    float* jo = reinterpret_cast<float*>(sm + S::RING);
    float* jm = jo + WARPS * MT * S::PITCH;  // [WARPS][MT][2]
    __syncthreads();                         // the previous tile's results have been read
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = g + 8 * half;
      if (x.r0 + r < x.r1) {
#pragma unroll
        for (int nt = 0; nt < D / 8; ++nt)
          *reinterpret_cast<float2*>(jo + (warp * MT + r) * S::PITCH + 8 * nt + p2) =
              make_float2(o[nt][2 * half], o[nt][2 * half + 1]);
        if ((lane & 3) == 0)
          *reinterpret_cast<float2*>(jm + (warp * MT + r) * 2) = make_float2(m[half], l[half]);
      }
    }
    const SeqView seq = cur.s;
    const int hk = cur.hk, first_u = cur.u;
    next_tile<MT, UK, DEAD>(a, cur, w.units);
    if (cur.left > 0) load_q();  // arrives while the tile's results are joined
    __syncthreads();
    const bool whole = w.units == x.units;
    const int slot = 2 * blockIdx.x + (first_u == 0 ? 1 : 0);
    for (int i = threadIdx.x; i < (x.r1 - x.r0) * (D / 4); i += WARPS * 32) {
      const int r = i / (D / 4), c = 4 * (i % (D / 4));
      float mm = -INFINITY;
#pragma unroll
      for (int i2 = 0; i2 < WARPS; ++i2) mm = fmaxf(mm, jm[(i2 * MT + r) * 2]);
      const float ref = mm == -INFINITY ? 0.f : mm;
      float ll = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i2 = 0; i2 < WARPS; ++i2) {
        const float2 ml = *reinterpret_cast<const float2*>(jm + (i2 * MT + r) * 2);
        const float f = fast_exp2(ml.x - ref);
        const float4 v = *reinterpret_cast<const float4*>(jo + (i2 * MT + r) * S::PITCH + c);
        ll += f * ml.y;
        acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
      }
      if (whole) {
        const float inv = ll > 0.f ? __fdiv_rn(1.f, ll) : 0.f;
        acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
        store_out4<CT>(a, row_offset(seq, a.group, hk, x.r0 + r, a.ldo, D) + c, acc);
        if (a.lse && c == 0)
          a.lse[row_offset(seq, a.group, hk, x.r0 + r, a.n_heads, 1)] = row_lse(mm, ll);
      } else {
        *reinterpret_cast<float4*>(a.part + part_offset<MT, D>(slot, r, c)) = acc;
        if (c == 0) {
          float* ml = a.part + static_cast<int64_t>(2 * gridDim.x) * MT * D + (static_cast<int64_t>(slot) * MT + r) * 2;
          ml[0] = mm;
          ml[1] = ll;
        }
      }
    }
  }
}

template <int CT, int D>
cudaError_t launch(const AttnArgs& a, int ctas, cudaStream_t s) {
  const cudaError_t e = ensure_smem(reinterpret_cast<const void*>(attend_stream_kernel<CT, D>), Smem<D>::BYTES);
  if (e != cudaSuccess) return e;
  return launch_pdl(attend_stream_kernel<CT, D>, dim3(ctas), dim3(WARPS * 32), Smem<D>::BYTES, s, a);
}

}  // namespace

cudaError_t launch_attend_stream(const AttnArgs& a, int type, int D, int ctas, cudaStream_t s) {
  if (type == MOEX_BF16) return D == 64 ? launch<MOEX_BF16, 64>(a, ctas, s) : launch<MOEX_BF16, 128>(a, ctas, s);
  return D == 64 ? launch<MOEX_F16, 64>(a, ctas, s) : launch<MOEX_F16, 128>(a, ctas, s);
}

}  // namespace moex
