// Paged attention over a cache of Q8_0 blocks: the cache is streamed once as it
// lies there, 34 bytes a block of 32 values, so DRAM bounds it.
//
// The division of the work is that of the 16-bit streaming kernel (attn.cuh): a
// CTA works on one tile of MT = 8 NT rows, each of its warps alone over every
// WARPS-th step of STEP keys, with its own copies in flight and its own running
// maximum and sum.  What is different is the arithmetic:
//
//   S^T = K Q^T   keys are the 16 rows of an mma.sync m16n8k16 and query rows its 8
//                 columns, so that a single token's few rows (1 to 8 heads a key
//                 head) leave little empty, and a converted key serves every NT.
//                 The products of a block are summed alone and then multiplied by
//                 the key's scale, in FP32: no value is rounded.
//   O^T = V^T P^T values are the A operand too (ldmatrix.trans on pairs of bytes
//                 brings two features of two keys into a register), so P^T is the B
//                 operand: S^T's fragment transposed by movmatrix.  The value's scale
//                 goes into P, block by block, before its one rounding to FP16
//                 (2^-11 of it, below a step of the values).
//
// int8 q becomes FP16 without arithmetic: the byte q + 128 alone in a half is the
// subnormal (q + 128) 2^-24, exactly.  The 128 are taken off a key inside the
// product, which starts from -128 sum(q) of the block (a tile's queries give it
// once); off a value by a subtraction, exactly, since what a product with P would
// lose there (2^-23 of 128 P) may be more than a small sum of values can bear.
//
// FP16 holds 2^-24 to 2^16, scales as much: the reference for the exponentials is
// taken over score + exponent of the key's largest value scale, less 15, so the
// largest product lies below 2^15.  It is moved only when a product would pass that,
// and then by GROW more, which leaves FP16's 11 bits down to 2^(GROW - 29) of the
// largest.  Queries are multiplied by the power of two that puts a row's largest value
// into [2^14, 2^15): BF16's values that this takes below FP16's range are 2^-38 of
// the row's largest.
//
// Measured, device time: 64 single tokens over contexts to 16384, 4 query heads a key
// head, 98 us, 90% of the copy rate (copies alone 93 us); three over up to 100001 keys
// 41 us (copies alone 33); one token over 1003 keys, its page table cut to 63 pages of 16,
// 6.6 us (2048 pages 9.2 us: ranges and the joining kernel).
#include <cooperative_groups.h>

#include <cfloat>

#include "attn.cuh"
#include "attn_q8.h"
#include "internal.h"

namespace moex {
namespace {

constexpr int DEAD = Q8_DEAD;
// One step of a warp in flight while another is read.  (Two in flight: 117 us in place of 103 for 64 tokens over contexts to
// 16384, 48 in place of 42 for three to 100001; three: 112 and 42.)
constexpr int WARPS = Q8_WARPS, STAGES = 2;
constexpr float GROW = 4.f;

// Shared memory: each warp's two stages (keys, values, their scales).  At the end of a tile
// the stage that is free takes the warp's output, eight rows at a time.
template <int D, int NT>
struct Smem {
  static constexpr int MT = 8 * NT, NB = D / QK;
  static constexpr int STEP = q8_step(D), UK = WARPS * STEP;
  static constexpr int PLANE = STEP * D;          // bytes of a step's keys
  static constexpr int SCALES = STEP * NB * 2;    // and of their scales
  static constexpr int STAGE = 2 * (PLANE + SCALES);
  static constexpr int PITCH = D + 4;             // floats of an output row
  static constexpr int BYTES = WARPS * STAGES * STAGE;
  static_assert(STAGE % 128 == 0 && 8 * PITCH * 4 <= STAGE, "eight rows of output in a stage");
};

// Byte offset of 16-byte chunk c of a step's row: eight rows' same chunk, which ldmatrix
// reads at a time, lies in eight different groups of banks.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
  if constexpr (D == 128) return row * 128 + ((c ^ (row & 7)) << 4);
  return (row >> 1) * 128 + ((((row & 1) * 4 + c) ^ ((row >> 1) & 3)) << 4);
}

// Copies without a size, and of a row's scales (bytes 0: zeros, and src is not read).
__device__ __forceinline__ void cp_async_row(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_async_scales(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_async_scales(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(in ? BYTES : 0)
               : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}

// Bytes 0 and 2 of a word of int8 as the halves (q + 128) 2^-24, and bytes 1 and 3: (w & 0x00FF00FF) ^ 0x00800080,
// one instruction with both constants in registers (an instruction holds one, and the compiler would use two).
struct ByteHalves {
  uint32_t low, flip;
  __device__ __forceinline__ ByteHalves() {
    asm volatile("mov.b32 %0, 0x00FF00FF;" : "=r"(low));
    asm volatile("mov.b32 %0, 0x00800080;" : "=r"(flip));
  }
  __device__ __forceinline__ uint32_t even(uint32_t w) const {
    uint32_t h;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(h) : "r"(w), "r"(low), "r"(flip));
    return h;
  }
  __device__ __forceinline__ uint32_t odd(uint32_t w) const { return even(w >> 8); }
};
__device__ __forceinline__ uint32_t less_128(uint32_t h) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(h), "r"(0x00800080u));
  return d;
}
constexpr uint32_t MINUS_128 = 0x80808080u;  // two halves of -128 * 2^-24

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
// d = a b + c; c's rows g and g + 8 the same where it is given as two numbers
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, float c0, float c1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// The FP16 scales of a row's blocks, as they lie in shared memory.
template <int NB>
struct RowScales {
  uint32_t w[NB / 2];
  __device__ __forceinline__ void load(uint32_t at) {
    if constexpr (NB == 4) {
      const uint2 v = lds64(at);
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = lds32(at);
    }
  }
  __device__ __forceinline__ float get(int b) const {
    const __half2 h = *reinterpret_cast<const __half2*>(&w[b >> 1]);
    return b & 1 ? __high2float(h) : __low2float(h);
  }
  // A power of two above every scale's magnitude, as its exponent (-14 for zeros and subnormal ones, 17 for those that
  // are not finite).
  __device__ __forceinline__ float exponent() const {
    constexpr uint32_t MAGNITUDE = 0x7FFF7FFFu;
    uint32_t m = w[0] & MAGNITUDE;
    if constexpr (NB == 4) m = __vmaxu2(m, w[1] & MAGNITUDE);
    m = __vmaxu2(m, m >> 16);
    return __uint_as_float(0x4B000000u | (m >> 10 & 0x1Fu)) - 8388622.f;  // 2^23 + n, less 2^23 + 14
  }
};

// The keys of a tile that a CTA's range holds, as one warp sees them: steps
// k0 + i * UK .. + STEP - 1.
template <int STEP, int UK>
struct WarpKeys {
  int units, k0, end, steps;
  __device__ __forceinline__ WarpKeys(const Cursor& c, int units_, int warp) : units(units_) {
    const int first = c.x.lo + c.u * UK;
    end = min(c.x.hi, first + units * UK);
    k0 = first + warp * STEP;
    steps = end > k0 ? (end - k0 + UK - 1) / UK : 0;
  }
};

// CL: a cluster works on a tile, each CTA on an equal share of its keys, and the shares
// are joined in distributed shared memory: no ranges, no workspace, no second kernel.
// The clusters stand for sequence, key head and `row_tiles` tiles of rows; where a
// sequence has more, its clusters take them in turn.
template <int QT, int D, int NT, bool CL>
__global__ void __launch_bounds__(WARPS * 32, q8_ctas(D, NT)) attend_stream_q8_kernel(const AttnArgs a, const ScaleView sc,
                                                                                     const int row_tiles) {
  extern __shared__ __align__(128) uint8_t sm[];
  using S = Smem<D, NT>;
  constexpr int MT = S::MT, NB = S::NB, STEP = S::STEP, UK = S::UK;
  constexpr int RUNS = STEP / 8, KK = STEP / 16;  // runs of eight keys, each inside one page; groups of 16
  using Keys = WarpKeys<STEP, UK>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_launch_dependents();  // the joining kernel's CTAs take the place of these as they end, and wait
  Cursor cur;
  const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  const int peers = CL ? static_cast<int>(cluster.num_blocks()) : 1, peer = CL ? static_cast<int>(cluster.block_rank()) : 0;
  auto share = [&](int units) { return (units + peers - 1) / peers; };
  auto units_of = [&](const Cursor& c) {
    return CL ? max(min(share(c.x.units), c.x.units - c.u), 0) : units_here(a, c);
  };
  auto advance = [&](Cursor& c, int done) {
    if constexpr (CL) {
      c.t += row_tiles;
      c.left = c.t * MT < c.s.n * a.group.n;
      if (c.left > 0) c.x = tile_of<MT, UK>(c.s, a.group, a.window, c.t);
      c.u = peer * share(c.x.units);
    } else {
      next_tile<MT, UK, DEAD>(a, c, done);
    }
  };
  if constexpr (CL) {
    const int tile = blockIdx.x / peers, per_seq = a.n_kv_heads * row_tiles;
    cur.b = tile / per_seq;
    cur.hk = tile % per_seq / row_tiles;
    cur.t = tile % row_tiles;
    cur.s = seq_view(a.b, cur.b);
    if (tile % per_seq == 0 && peer == 0 && threadIdx.x == 0 && (cur.s.bad || uncovered(a.b, cur.b)))
      flag_status(a.b.status, DEV_BAD_BATCH);
    if (cur.t * MT >= cur.s.n * a.group.n) return;  // with the whole cluster
    cur.left = 1;
    cur.x = tile_of<MT, UK>(cur.s, a.group, a.window, cur.t);
    cur.u = peer * share(cur.x.units);
  } else {
    __shared__ RangeScratch<WARPS * 32> scratch;
    find_range<MT, UK, DEAD, WARPS * 32>(a, blockIdx.x, gridDim.x, cur, scratch);
    if (cur.left <= 0) return;
  }
  __shared__ float part[CL ? 8 : 1][CL ? D : 1];  // a cluster's: this CTA's eight rows,
  __shared__ float2 part_stats[8];                // and their references and sums
  const uint32_t ring = smem_u32(sm) + warp * STAGES * S::STAGE;

  // ---- copies: a cursor of their own, a step ahead of the products
  __shared__ Cursor ahead_of[WARPS];
  __shared__ uint32_t out_at[WARPS];    // at the end of a tile: each warp's free stage,
  __shared__ float2 stats[WARPS][8];    // and its rows' references and sums
  Cursor& ahead = ahead_of[warp];
  if (lane == 0) ahead = cur;
  __syncwarp();
  constexpr int CH = D / 16, RPI = 32 / CH;  // 16-byte chunks of a row, rows an instruction covers
  const uint32_t page_stride = static_cast<uint32_t>(a.b.page_stride), row_stride = static_cast<uint32_t>(a.b.row_stride);
  const uint32_t sc_page = 2 * static_cast<uint32_t>(sc.page_stride), sc_row = 2 * static_cast<uint32_t>(sc.row_stride);
  const uint32_t slots = (1u << a.b.page_shift) - 1;
  const int64_t to_vs = reinterpret_cast<const char*>(sc.v) - reinterpret_cast<const char*>(sc.k);
  // where this lane's chunk of rows 0 .. RPI - 1 goes, in the warp's first stage
  const uint32_t to0 = ring + chunk_at<D>(lane / CH, lane % CH);
  const int s_row = lane % STEP;  // scales: a lane a row; with steps of 16 keys the upper lanes take the values'
  int l_i = 0, l_steps = 0, l_j = 0, l_end = 0, l_from = 0, l_hk = 0;  // the tile that copies are issued for; its next step
  const int8_t *l_kp = nullptr, *l_vp = nullptr;                      // this lane's chunk in slot 0 of page 0
  const char* l_sp = nullptr;                                         // and its row's scales
  bool l_more = true;
  int pg[RUNS];        // lane l: pages of the runs of step 32 * (l_i / 32) + l
  uint32_t l_all = 0;  // bit l: that step's keys are all there
  const int32_t* l_table = nullptr;
  auto fetch_pages = [&]() {
    const int j = l_j + lane * UK;
    bool all = j >= l_from && j + STEP <= l_end;
#pragma unroll
    for (int r = 0; r < RUNS; ++r) {
      const int k = j + 8 * r;
      pg[r] = k + 7 >= l_from && k < l_end ? __ldg(l_table + (k >> a.b.page_shift)) : 0;
    }
#pragma unroll
    for (int r = 0; r < RUNS; ++r) all = all && static_cast<uint32_t>(pg[r]) < static_cast<uint32_t>(a.b.n_pages);
    l_all = __ballot_sync(0xffffffffu, all);
  };
  // the next tile in which this warp has a step; its pages are asked for at once
  auto seek = [&](bool fresh) {
    for (;; fresh = false) {
      if (!fresh) {
        const int units = units_of(ahead);
        __syncwarp();
        if (lane == 0) advance(ahead, units);
        __syncwarp();
      }
      l_more = ahead.left > 0;
      if (!l_more) return;
      const Keys w(ahead, units_of(ahead), warp);
      if (w.steps == 0) continue;
      l_i = 0, l_steps = w.steps, l_j = w.k0, l_end = w.end, l_from = ahead.x.from, l_hk = ahead.hk;
      const int64_t lane_off = l_hk * a.b.head_stride + (lane / CH) * a.b.row_stride + 16 * (lane % CH);
      l_kp = static_cast<const int8_t*>(a.k) + lane_off;
      l_vp = static_cast<const int8_t*>(a.v) + lane_off;
      l_sp = reinterpret_cast<const char*>((STEP == 16 && lane >= 16 ? sc.v : sc.k) + l_hk * sc.head_stride +
                                           (s_row & 7) * sc.row_stride);
      l_table = a.b.table + ahead.b * a.b.table_stride;
      fetch_pages();
      return;
    }
  };
  uint32_t ok_ring = 0;  // RUNS bits a stage: the step's runs have a page
  auto load = [&](int stage) {
    if (l_more) {
      const int at_step = l_i & 31;
      uint32_t page[RUNS];
#pragma unroll
      for (int r = 0; r < RUNS; ++r) page[r] = __shfl_sync(0xffffffffu, pg[r], at_step);
      // scales of row s_row: its run's page and slot
      uint32_t s_page = page[0];
#pragma unroll
      for (int run = 1; run < RUNS; ++run) s_page = s_row >> 3 == run ? page[run] : s_page;
      const uint32_t s_dst = ring + stage * S::STAGE + 2 * S::PLANE + lane * (NB * 2);
      const char* const s_src = l_sp + static_cast<uint64_t>(s_page) * sc_page +
                                static_cast<uint64_t>((l_j + (s_row & ~7)) & slots) * sc_row;
      if (l_all >> at_step & 1u) {
        ok_ring |= ((1u << RUNS) - 1) << (RUNS * stage);
        const uint32_t at0 = to0 + stage * S::STAGE, at1 = at0 ^ 64u;  // (stages are multiples of 128 bytes)
#pragma unroll
        for (int run = 0; run < RUNS; ++run) {
          // products of 32-bit numbers, which fold the additions in
          const uint64_t slot = (l_j + 8 * run) & slots;
          const int8_t* kp = l_kp + static_cast<uint64_t>(page[run]) * page_stride + slot * row_stride;
          const int8_t* vp = l_vp + static_cast<uint64_t>(page[run]) * page_stride + slot * row_stride;
#pragma unroll
          for (int n = 0; n < 8 / RPI; ++n) {
            // rows 8 run + n RPI + lane / CH
            const uint32_t at = (D == 128 && n & 1 ? at1 : at0) + (8 * run + n * RPI) * D;
            cp_async_row(at, kp);
            cp_async_row(at + S::PLANE, vp);
            kp += static_cast<uint64_t>(RPI) * row_stride;
            vp += static_cast<uint64_t>(RPI) * row_stride;
          }
        }
        cp_async_scales<NB * 2>(s_dst, s_src);
        if (STEP == 32) cp_async_scales<NB * 2>(s_dst + S::SCALES, s_src + to_vs);
      } else {
        const int r0 = l_from - l_j, r1 = l_end - l_j;  // the step's rows that are there
        uint32_t ok = 0;
#pragma unroll
        for (int r = 0; r < RUNS; ++r) ok |= (page[r] < static_cast<uint32_t>(a.b.n_pages) ? 1u : 0u) << r;
        if (ok != (1u << RUNS) - 1 && lane == 0) flag_status(a.b.status, DEV_BAD_BATCH);
        ok_ring = (ok_ring & ~(((1u << RUNS) - 1) << (RUNS * stage))) | ok << (RUNS * stage);
        // zeros in place of keys outside: a scale beside a probability of 0 must be finite
#pragma unroll
        for (int n = 0; n < STEP / RPI; ++n) {
          // the run of an instruction's rows is known when this is compiled: RPI divides 8
          const int r = n * RPI + lane / CH, run = n * RPI / 8;
          const bool in = r >= r0 && r < r1 && (ok >> run & 1u);
          const int64_t off = in ? kv_offset(a.b, page[run], l_hk, l_j + r) + 16 * (lane % CH) : 0;
          const uint32_t at = ring + stage * S::STAGE + chunk_at<D>(r, lane % CH);
          cp_async16(at, static_cast<const int8_t*>(a.k) + off, in ? 16u : 0u);
          cp_async16(at + S::PLANE, static_cast<const int8_t*>(a.v) + off, in ? 16u : 0u);
        }
        const bool in = s_row >= r0 && s_row < r1 && (ok >> (s_row >> 3) & 1u);
        const char* const src = in ? s_src : reinterpret_cast<const char*>(sc.k);
        cp_async_scales<NB * 2>(s_dst, src, in);
        if (STEP == 32) cp_async_scales<NB * 2>(s_dst + S::SCALES, in ? src + to_vs : src, in);
      }
      l_j += UK;
      if (++l_i == l_steps)
        seek(false);
      else if ((l_i & 31) == 0)
        fetch_pages();
    }
    cp_commit();
  };
  const ByteHalves bytes;
  seek(true);
  load(0);
  int stage = 0;
  // ldmatrix rows of a block: keys 0-7 and 8-15 of its first 16 features, then of the others
  uint32_t frag[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) frag[b] = chunk_at<D>(lane & 15, 2 * b + (lane >> 4));

  // Q as the B operand, the same for every step: column g of each eight rows, features 32 b + 16 h + 4 t .. + 3 in
  // the order of a key word's halves, times the row's power of two.  bias[][]: -128 2^-24 times a block's sum, for
  // columns 2t and 2t + 1; unit[][]: what takes the powers of two off a score again, times its scale.
  uint32_t qf[NT][NB][2][2];
  float unit[NT][2], bias[NT][NB][2];
  auto load_q = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = cur.x.r0 + 8 * nt + g;
      const bool in = r < cur.x.r1;
      const auto* row = static_cast<const uint16_t*>(a.q) + (in ? row_offset(cur.s, a.group, cur.hk, r, a.ldq, D) : 0);
      uint2 v[NB][2];
      float top = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          v[b][h] = in ? *reinterpret_cast<const uint2*>(row + QK * b + 16 * h + 4 * t) : make_uint2(0u, 0u);
          const float2 f0 = RowElem<QT>::unpack(v[b][h].x), f1 = RowElem<QT>::unpack(v[b][h].y);
          top = fmaxf(top, fmaxf(fmaxf(fabsf(f0.x), fabsf(f0.y)), fmaxf(fabsf(f1.x), fabsf(f1.y))));
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // exponent fields: 2^14 <= top * up < 2^15 (less for rows that are FP32's smallest), down = 1 / up
      const int field = min(268 - static_cast<int>(__float_as_uint(top) >> 23), 253);
      const float up = __uint_as_float(static_cast<uint32_t>(field) << 23);
      const float down = __uint_as_float(static_cast<uint32_t>(254 - field) << 23) * a.scale_log2;
      // (a row beyond 2^113 / scale has scores that leave all but one probability 0 whatever the factor; one of 0 would
      // make a masked score NaN)
      unit[nt][0] = fmaxf(fminf(__shfl_sync(0xffffffffu, down, 8 * t) * 16777216.f, FLT_MAX), FLT_MIN);
      unit[nt][1] = fmaxf(fminf(__shfl_sync(0xffffffffu, down, 8 * t + 4) * 16777216.f, FLT_MAX), FLT_MIN);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 f0 = RowElem<QT>::unpack(v[b][h].x), f1 = RowElem<QT>::unpack(v[b][h].y);
          qf[nt][b][h][0] = RowElem<MOEX_F16>::pack(f0.x * up, f1.x * up);
          qf[nt][b][h][1] = RowElem<MOEX_F16>::pack(f0.y * up, f1.y * up);
        }
        float sum[4];
        mma_f16(sum, MINUS_128, MINUS_128, MINUS_128, MINUS_128, qf[nt][b][0][0], qf[nt][b][0][1], 0.f, 0.f);
        mma_f16(sum, MINUS_128, MINUS_128, MINUS_128, MINUS_128, qf[nt][b][1][0], qf[nt][b][1][1]);
        bias[nt][b][0] = sum[0], bias[nt][b][1] = sum[1];
      }
    }
  };
  load_q();

  while (cur.left > 0) {
    const Tile x = cur.x;
    const Keys w(cur, units_of(cur), warp);
    const int base = cur.s.ctx - cur.s.n;
    // steps clear_lo .. + clear_n - 1 hold keys that every row sees, and need no mask (rows past the last are not stored)
    const int all_bot = a.window > 0 ? max(base + a.group.token(x.r1 - 1) - a.window + 1, x.from) : x.from;
    const int all_top = min(base + a.group.token(x.r0) + 1, w.end);
    const int clear_lo = all_bot > w.k0 ? (all_bot - w.k0 + UK - 1) / UK : 0;
    const int clear_n = all_top - w.k0 >= STEP ? max((all_top - w.k0 - STEP) / UK + 1 - clear_lo, 0) : 0;

    // ref: what is taken off a score (0 for a row that has seen no key); lim: the largest score + exponent that it allows
    float o[NT][NB][2][4], ref[NT][2], lim[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      ref[nt][0] = ref[nt][1] = 0.f;
      lim[nt][0] = lim[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][b][0][e] = o[nt][b][1][e] = 0.f;
    }
    for (int i = 0; i < w.steps; ++i) {
      const uint32_t ok = (ok_ring >> (RUNS * stage)) & ((1u << RUNS) - 1);
      __syncwarp();  // the stage refilled next has been read by every lane
      load(stage ^ 1);
      cp_wait<1>();
      __syncwarp();  // every lane's copies have landed
      const uint32_t kb = ring + stage * S::STAGE, vb = kb + S::PLANE, ks = vb + S::PLANE, vs = ks + S::SCALES;

      // ---- scores of keys 16 kk + g and + 8, rows 2t and 2t + 1 of each eight
      float s[KK][NT][4];
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        const int r = 16 * kk + g;
        RowScales<NB> d0, d1;
        d0.load(ks + r * (NB * 2));
        d1.load(ks + (r + 8) * (NB * 2));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[kk][nt][0] = s[kk][nt][1] = s[kk][nt][2] = s[kk][nt][3] = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          uint32_t k4[4];  // rows g and g + 8: features 4t .. + 3, then 16 + 4t .. + 3, of the block
          ldsm4(k4, kb + frag[b] + kk * 16 * D);
          const float e0 = d0.get(b), e1 = d1.get(b);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float acc[4];
            mma_f16(acc, bytes.even(k4[0]), bytes.even(k4[1]), bytes.odd(k4[0]), bytes.odd(k4[1]), qf[nt][b][0][0],
                    qf[nt][b][0][1], bias[nt][b][0], bias[nt][b][1]);
            mma_f16(acc, bytes.even(k4[2]), bytes.even(k4[3]), bytes.odd(k4[2]), bytes.odd(k4[3]), qf[nt][b][1][0],
                    qf[nt][b][1][1]);
            s[kk][nt][0] += e0 * acc[0], s[kk][nt][1] += e0 * acc[1];
            s[kk][nt][2] += e1 * acc[2], s[kk][nt][3] += e1 * acc[3];
          }
        }
      }
      if (static_cast<unsigned>(i - clear_lo) >= clear_n || ok != (1u << RUNS) - 1) {
        const int j = w.k0 + i * UK;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int run = 2 * kk + (e >> 1), key = j + 8 * run + g, r = x.r0 + 8 * nt + 2 * t + (e & 1);
              const int top = r < x.r1 ? base + a.group.token(r) : -1;  // keys top - window < key <= top are seen
              const bool seen = key <= top && !(a.window > 0 && key <= top - a.window) && (ok >> run & 1u);
              if (!seen) s[kk][nt][e] = -INFINITY;
            }
      }

      // ---- maxima over the step's keys, each with the exponent of its value scales
      RowScales<NB> dv[KK][2];
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mx[nt][0] = mx[nt][1] = -INFINITY;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          dv[kk][h].load(vs + (16 * kk + 8 * h + g) * (NB * 2));
          const float e = dv[kk][h].exponent();
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mx[nt][0] = fmaxf(mx[nt][0], fmaf(s[kk][nt][2 * h], unit[nt][0], e));
            mx[nt][1] = fmaxf(mx[nt][1], fmaf(s[kk][nt][2 * h + 1], unit[nt][1], e));
          }
        }
      bool past = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) past = past || mx[nt][0] > lim[nt][0] || mx[nt][1] > lim[nt][1];
      if (__any_sync(0xffffffffu, past)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = mx[nt][e];
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            if (v > lim[nt][e]) {
              const float to = v + GROW - 15.f;
              const float corr = lim[nt][e] == -INFINITY ? 0.f : fast_exp2(ref[nt][e] - to);  // from nothing: 0 stays 0
              ref[nt][e] = to;
              lim[nt][e] = v + GROW;
              l[nt][e] *= corr;
#pragma unroll
              for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h) o[nt][b][h][e] *= corr, o[nt][b][h][2 + e] *= corr;
            }
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = fast_exp2(fmaf(s[kk][nt][e], unit[nt][e & 1], -ref[nt][e & 1]));
            s[kk][nt][e] = p;
            l[nt][e & 1] += p;
          }

      // ---- features 32 b + 16 h + 2g and + 1 of keys 16 kk + 2t, + 1, + 8, + 9
#pragma unroll
      for (int kk = 0; kk < KK; ++kk)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float e0 = dv[kk][0].get(b), e1 = dv[kk][1].get(b);
          uint32_t v4[4];
          ldsm4_t(v4, vb + frag[b] + kk * 16 * D);
          uint32_t f[2][4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            f[i >> 1][2 * (i & 1)] = less_128(bytes.even(v4[i])), f[i >> 1][2 * (i & 1) + 1] = less_128(bytes.odd(v4[i]));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float(&p)[4] = s[kk][nt];
            const uint32_t b0 = transpose8x8(RowElem<MOEX_F16>::pack(p[0] * e0, p[1] * e0));
            const uint32_t b1 = transpose8x8(RowElem<MOEX_F16>::pack(p[2] * e1, p[3] * e1));
#pragma unroll
            for (int h = 0; h < 2; ++h) mma_f16(o[nt][b][h], f[h][0], f[h][1], f[h][2], f[h][3], b0, b1);
          }
        }
      stage ^= 1;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], i);
    const SeqView seq = cur.s;
    const int hk = cur.hk;
    const bool whole = w.units == x.units;
    const int slot = 2 * blockIdx.x + (cur.u == 0 ? 1 : 0);
    const uint32_t mine = static_cast<uint32_t>((stage ^ 1) * S::STAGE);
    advance(cur, w.units);
    out_at[warp] = mine;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (nt > 0) __syncthreads();  // the rows before have been read
      float* jo = reinterpret_cast<float*>(sm + warp * STAGES * S::STAGE + mine);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 2 * t + e;
        if (x.r0 + 8 * nt + r < x.r1) {
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              *reinterpret_cast<float2*>(jo + r * S::PITCH + QK * b + 16 * h + 2 * g) =
                  make_float2(o[nt][b][h][e], o[nt][b][h][2 + e]);
          if (g == 0) stats[warp][r] = make_float2(lim[nt][e] == -INFINITY ? -INFINITY : ref[nt][e], l[nt][e]);
        }
      }
      if (nt == NT - 1 && cur.left > 0) load_q();  // arrives while the tile's results are joined
      __syncthreads();
      for (int i = threadIdx.x; i < min(8, x.r1 - x.r0 - 8 * nt) * (D / 4); i += WARPS * 32) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4)), row = x.r0 + 8 * nt + r;
        float mm = -INFINITY;
#pragma unroll
        for (int i2 = 0; i2 < WARPS; ++i2) mm = fmaxf(mm, stats[i2][r].x);
        const float mref = mm == -INFINITY ? 0.f : mm;
        float ll = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i2 = 0; i2 < WARPS; ++i2) {
          const float2 ml = stats[i2][r];
          float f = fast_exp2(ml.x - mref);
          const float4 v =
              *reinterpret_cast<const float4*>(sm + i2 * STAGES * S::STAGE + out_at[i2] + (r * S::PITCH + c) * 4);
          ll += f * ml.y;
          f *= 16777216.f;  // the values' 2^-24
          acc.x += f * v.x, acc.y += f * v.y, acc.z += f * v.z, acc.w += f * v.w;
        }
        if constexpr (CL) {
          *reinterpret_cast<float4*>(&part[r][c]) = acc;
          if (c == 0) part_stats[r] = make_float2(mm, ll);
        } else if (whole) {
          const float inv = ll > 0.f ? __fdiv_rn(1.f, ll) : 0.f;
          acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
          store_out4<QT>(a, row_offset(seq, a.group, hk, row, a.ldo, D) + c, acc);
          if (a.lse && c == 0) a.lse[row_offset(seq, a.group, hk, row, a.n_heads, 1)] = row_lse(mm, ll);
        } else {
          *reinterpret_cast<float4*>(a.part + part_offset<MT, D>(slot, 8 * nt + r, c)) = acc;
          if (c == 0) {
            float* ml = a.part + static_cast<int64_t>(2 * gridDim.x) * MT * D +
                        (static_cast<int64_t>(slot) * MT + 8 * nt + r) * 2;
            ml[0] = mm;
            ml[1] = ll;
          }
        }
      }
      if constexpr (CL) {
        cluster.sync();
        // four columns of a row a thread, over the cluster
        for (int i = peer * WARPS * 32 + threadIdx.x; i < min(8, x.r1 - x.r0 - 8 * nt) * (D / 4); i += peers * WARPS * 32) {
          const int r = i / (D / 4), c = 4 * (i % (D / 4)), row = x.r0 + 8 * nt + r;
          float2 ml[Q8_CLUSTER];
          float4 v[Q8_CLUSTER];
          float mm = -INFINITY;
#pragma unroll
          for (int k = 0; k < Q8_CLUSTER; ++k) {
            ml[k] = make_float2(-INFINITY, 0.f);
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k < peers) {
              ml[k] = *cluster.map_shared_rank(&part_stats[r], k);
              v[k] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(&part[r][c], k));
            }
          }
#pragma unroll
          for (int k = 0; k < Q8_CLUSTER; ++k) mm = fmaxf(mm, ml[k].x);
          const float mref = mm == -INFINITY ? 0.f : mm;
          float ll = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < Q8_CLUSTER; ++k) {
            const float f = fast_exp2(ml[k].x - mref);
            ll += f * ml[k].y;
            acc.x += f * v[k].x, acc.y += f * v[k].y, acc.z += f * v[k].z, acc.w += f * v[k].w;
          }
          const float inv = ll > 0.f ? __fdiv_rn(1.f, ll) : 0.f;
          acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
          store_out4<QT>(a, row_offset(seq, a.group, hk, row, a.ldo, D) + c, acc);
          if (a.lse && c == 0) a.lse[row_offset(seq, a.group, hk, row, a.n_heads, 1)] = row_lse(mm, ll);
        }
        cluster.sync();  // the shares have been read
      }
    }
    __syncthreads();  // the stages take copies again
  }
}

template <int QT, int D, int NT>
cudaError_t launch(const AttnArgs& a, const ScaleView& sc, const Q8Grid& g, cudaStream_t s) {
  constexpr int BYTES = Smem<D, NT>::BYTES;
  if (g.cluster == 0) {
    const auto kernel = attend_stream_q8_kernel<QT, D, NT, false>;
    const cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kernel), BYTES);
    return e != cudaSuccess ? e : launch_pdl(kernel, dim3(g.ctas), dim3(WARPS * 32), BYTES, s, a, sc, 1);
  }
  const auto kernel = attend_stream_q8_kernel<QT, D, NT, true>;
  const cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kernel), BYTES);
  return e != cudaSuccess ? e : launch_cluster(kernel, dim3(g.ctas), dim3(WARPS * 32), g.cluster, BYTES, s, a, sc, g.row_tiles);
}

template <int QT>
cudaError_t launch_type(const AttnArgs& a, const ScaleView& sc, int D, const Q8Grid& g, cudaStream_t s) {
  if (D == 64) return g.mt == 8 ? launch<QT, 64, 1>(a, sc, g, s) : launch<QT, 64, 2>(a, sc, g, s);
  return g.mt == 8 ? launch<QT, 128, 1>(a, sc, g, s) : launch<QT, 128, 2>(a, sc, g, s);
}

template <int D, int NT>
int clusters(int size) {
  const auto kernel = reinterpret_cast<const void*>(attend_stream_q8_kernel<MOEX_BF16, D, NT, true>);
  return ensure_smem(kernel, Smem<D, NT>::BYTES) == cudaSuccess
             ? resident_clusters(kernel, WARPS * 32, size, Smem<D, NT>::BYTES)
             : q8_ctas(D, NT) * sm_count() / size;
}

}  // namespace

int q8_clusters(int D, int mt, int size) {
  if (D == 64) return mt == 8 ? clusters<64, 1>(size) : clusters<64, 2>(size);
  return mt == 8 ? clusters<128, 1>(size) : clusters<128, 2>(size);
}

cudaError_t launch_attend_stream_q8(const AttnArgs& a, const ScaleView& sc, int q_type, int D, const Q8Grid& g,
                                    cudaStream_t s) {
  return q_type == MOEX_BF16 ? launch_type<MOEX_BF16>(a, sc, D, g, s) : launch_type<MOEX_F16>(a, sc, D, g, s);
}

}  // namespace moex
