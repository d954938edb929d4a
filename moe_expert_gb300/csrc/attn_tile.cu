// Paged attention for many rows a key head (prompts and chunks) on tcgen05.
//
// A CTA (one an SM) works on a tile of 256 rows as two groups of 128, over
// blocks of 128 keys.  With S = Q K^T and O = P V:
//   - S of a group: 128 x 128 FP32 in TMEM; P (16-bit) replaces it in place and
//     is the A operand of the second product, so neither touches shared memory;
//   - O of a group: 128 x D FP32 in TMEM.  4 * 128 columns hold both groups.
// Both groups use one copy of every key block: 64 KB of cache feed 4 products of
// 128 x 128 x 128.
// Warps: 0 issues the MMAs; 1-3 copy keys, values and queries; 4-7 and 8-11 are
// the softmax of the two groups, one row a thread, so maxima and sums need no
// exchange (192 registers: a row's 128 scores stay in them).  A block of keys
// comes by cp.async, or by TMA where pages are long enough.
// A block that the sequence or its window does not fill, or that has a page out
// of range, comes by cp.async with zeros in place of what no row sees or is not
// there, since a value beside a probability of 0 must be finite.
// The MMA order is PV0(j), QK0(j+1), PV1(j), QK1(j+1): while one group's
// products run the other's softmax does.  A row's reference for the exponentials
// follows its maximum only when that grows by more than 2^8, so O is rescaled
// rarely; sums and O are exact for any reference.
// Measured, 2048 tokens over 14336 keys, 32 heads of 128, 8 key heads, pages of
// 64: 323-344 us with the joining kernel on ten boxes, 1497-1596 TFLOP/s (floor
// 268 us); the tensor pipe works 70% of the kernel's time.  The chain softmax - PV
// - QK of a group, about 2800 cycles a block against 2048 of tensor work for both
// groups, sets the pace.  Slower: two threads a row (375 us), P handed over in
// halves (363 us), the same softmax in 176 registers beside four copying warps
// (408 us).
#include "attn.cuh"
#include "attn_launch.h"
#include "internal.h"
#include "tc.cuh"

namespace moex {
namespace {

constexpr int MT = TILE_MT, UK = TILE_UK, DEAD = TILE_DEAD;
constexpr int MIN_BOX = 32, MAX_BOX = 64;  // slots of a TMA box
constexpr int THREADS = 384, LOADERS = 3, SOFTMAX0 = 4;  // warps 1-3 copy, 4-11 softmax
constexpr float GROW = 8.f;  // log2 of the growth of a maximum that rescales O

template <int D>
struct Lay {
  static constexpr int HALF = 128 * 128;              // 128 rows of 64 elements, 128-byte swizzle
  static constexpr int STAGE = (D / 64) * HALF;       // 128 keys (or values)
  static constexpr int NS = D == 64 ? 8 : 5;          // stages: K0 V0 K1 V1 ...
  static constexpr int Q = 0;                         // [group][half]
  static constexpr int RING = 2 * STAGE;
  static constexpr int BARS = RING + NS * STAGE;
  static constexpr int N_BARS = 2 * NS + 2 + 10 + 1;
  static constexpr int CURSORS = BARS + N_BARS * 8;
  static constexpr int FLAGS = CURSORS + (SOFTMAX0 + 2) * sizeof(Cursor);  // TMEM address, abort flag
  static constexpr int BYTES = FLAGS + 8;
};

// Whether the phase is complete, at once (try_wait may suspend the thread first).
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// A place in a ring of N stages that K and V take in turn: the stage and the
// parity of its current use.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      parity ^= 1;
    }
  }
  __device__ __forceinline__ void next2() {
    slot += 2;
    if (slot >= N) {
      slot -= N;
      parity ^= 1;
    }
  }
};

// Shared-memory writes of this thread before reads by the tensor core.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
template <int R>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// The larger of three, and FP32 arithmetic on pairs.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Writes 64 bytes of each lane's row (16 FP32 values, or 32 rounded to 16 bits):
// the 4 x 4 sixteen-byte pieces of four lanes are exchanged, so that four lanes
// write 64 bytes of one row and a store touches 8 rows, not 32.  off: the row's
// element offset, -1 for none.
template <int TYPE>
__device__ __forceinline__ void store_rows(void* out, int64_t off, int col, const uint32_t* v, int lane) {
  uint32_t w[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (TYPE == MOEX_F32)
        w[i][j] = v[4 * i + j];
      else
        w[i][j] = RowElem<TYPE>::pack(__uint_as_float(v[8 * i + 2 * j]), __uint_as_float(v[8 * i + 2 * j + 1]));
    }
  // transpose over the lane's two low bits: piece i of lane k <-> piece k of lane i
#pragma unroll
  for (int b = 1; b < 4; b <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!(i & b)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool up = lane & b;
          const uint32_t send = up ? w[i][j] : w[i | b][j];
          const uint32_t got = __shfl_xor_sync(0xffffffffu, send, b);
          if (up)
            w[i][j] = got;
          else
            w[i | b][j] = got;
        }
      }
  constexpr int PIECE = TYPE == MOEX_F32 ? 4 : 8;  // elements of 16 bytes
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t o = __shfl_sync(0xffffffffu, off, (lane & ~3) | i);  // the row of lane 4 * (lane / 4) + i
    if (o >= 0) {
      void* p = TYPE == MOEX_F32 ? static_cast<void*>(static_cast<float*>(out) + o + col + PIECE * (lane & 3))
                                 : static_cast<void*>(static_cast<uint16_t*>(out) + o + col + PIECE * (lane & 3));
      *reinterpret_cast<uint4*>(p) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
    }
  }
}

// A word with its n lowest bits set (none below 0, all above 32).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

template <int CT, int D>
__global__ void __launch_bounds__(THREADS, 1)
    attend_tile_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const int tma) {
  extern __shared__ __align__(1024) uint8_t sm[];
  using L = Lay<D>;
  using E = RowElem<CT>;
  constexpr int CH = D / 8;  // 16-byte chunks of a row
  constexpr int NS = L::NS;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + L::FLAGS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::FLAGS + 4);
  // The range is walked by the MMA warp, by each copying warp, and by each softmax
  // group together; the cursors stay out of the registers.
  Cursor* cursors = reinterpret_cast<Cursor*>(sm + L::CURSORS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(sm + L::BARS);
  uint64_t* kv_empty = kv_full + NS;
  uint64_t* q_full = kv_empty + NS;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* o_empty = o_full + 2;
  uint64_t* meet = o_empty + 2;  // the warps of a softmax group
  uint64_t* done = meet + 2;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < NS; ++i) {
      mbar_init(&kv_full[i], LOADERS);
      mbar_init(&kv_empty[i], 1);  // a commit
    }
    mbar_init(q_full, LOADERS);
    mbar_init(q_empty, 1);
    for (int g = 0; g < 2; ++g) {
      mbar_init(&s_full[g], 1);
      mbar_init(&p_full[g], 4);
      mbar_init(&o_full[g], 1);
      mbar_init(&o_empty[g], 4);
      mbar_init(&meet[g], 4);
    }
    mbar_init(done, 1);
    fence_mbar_init();
  }
  if (warp == SOFTMAX0) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  pdl_wait();
  Cursor& cur = cursors[warp < SOFTMAX0 ? warp : SOFTMAX0 + (warp - SOFTMAX0) / 4];
  RangeScratch<THREADS>& scratch = *reinterpret_cast<RangeScratch<THREADS>*>(sm + L::Q);  // not in use yet
  const bool counted = a.b.n_seqs <= WARP_SEQS;
  if (counted) {
    // a warp a sequence
    for (int b = warp; b < a.b.n_seqs; b += THREADS / 32) {
      const int64_t u = seq_units_warp<MT, UK, DEAD>(seq_view(a.b, b), a.group, a.window);
      if (lane == 0) scratch.counted[b] = u;
    }
    __syncthreads();
  }
  if (!counted || warp == 0) {
    Cursor at;
    find_range<MT, UK, DEAD, THREADS>(a, blockIdx.x, gridDim.x, at, scratch, counted);
    if (warp == 0 && lane < SOFTMAX0 + 2) cursors[lane] = at;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t smb = smem_u32(sm);

  // A wait of a whole warp: all of its lanes go on, or none.
  auto warp_wait = [&](uint64_t* bar, uint32_t parity, uint32_t bit) {
    if (__all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag))) return true;
    if (!*abort_flag) flag_status(a.b.status, bit);
    *abort_flag = 1;
    return false;
  };
  auto advance = [&](int units) {
    __syncwarp();
    if (lane == 0) next_tile<MT, UK, DEAD>(a, cur, units);
    __syncwarp();
  };

  if (warp < SOFTMAX0) regs_down<120>();
  if (tma && threadIdx.x == 32) {
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  if (warp >= 1 && warp < SOFTMAX0) {
    // ------------------------------------------------ keys, values, queries
    // A block is 16 runs of 8 keys, each inside one page; warp w copies runs
    // w - 1, w + 2, ...
    constexpr int RPI = 32 / CH;      // rows an instruction covers: 2 or 4
    constexpr int PER_RUN = 8 / RPI;  // instructions a run takes
    constexpr int RUNS = (16 + LOADERS - 1) / LOADERS;
    const int lw = warp - 1, c = lane % CH, r0 = lane / CH;
    uint32_t dst0[PER_RUN];
#pragma unroll
    for (int i = 0; i < PER_RUN; ++i) {
      const int r = i * RPI + r0;
      dst0[i] = (c >> 3) * L::HALF + r * 128 + (((c & 7) ^ r) << 4);
    }
    const int64_t rows = RPI * a.b.row_stride, mine_at = r0 * a.b.row_stride + 8 * c;
    Ring<NS> ring;
    int told_slot = 0, untold = 0;  // stages under way that the MMA warp does not know of
    bool filled = false;            // the ring has been filled once: stages have to be waited for
    auto announce = [&](int keep) {
      fence_async_smem();
      __syncwarp();
      for (; untold > keep; --untold) {
        if (lane == 0) mbar_arrive(&kv_full[told_slot]);
        told_slot = told_slot + 1 == NS ? 0 : told_slot + 1;
      }
    };
    bool ok = true;
    for (int tile = 0; cur.left > 0 && ok; ++tile) {
      const int units = units_here(a, cur);
      const int first = cur.x.lo + cur.u * UK, hi = cur.x.hi, hk = cur.hk;
      const int32_t* table = a.b.table + cur.b * a.b.table_stride;
      // lane l < 16: the page of run l of a block, read a block ahead and looked at when its turn comes;
      // a run wholly in front of the window or behind the keys has none
      auto has_page = [&](int j) { return lane < 16 && j + 7 >= cur.x.from && j < hi; };
      auto fetch_page = [&](int j) {
        j += 8 * lane;
        return has_page(j) ? __ldg(table + (j >> a.b.page_shift)) : -1;
      };
      int pg = fetch_page(first);
      for (int i = 0; i < units; ++i) {
        const int j0 = first + i * UK, j = j0 + 8 * lane;
        // the offset of the run's first row, -1 for none
        int64_t mine = -1;
        if (pg >= 0 && pg < a.b.n_pages)
          mine = kv_offset(a.b, pg, hk, j);
        else if (has_page(j))
          flag_status(a.b.status, DEV_BAD_BATCH);
        const int pages = pg;  // of this block's runs
        const bool whole = __all_sync(0xffffffffu, lane >= 16 || (mine >= 0 && j >= cur.x.from)) && j0 + UK <= hi;
        if (i + 1 < units) pg = fetch_page(j0 + UK);
        int64_t off[RUNS];
#pragma unroll
        for (int n = 0; n < RUNS; ++n) off[n] = __shfl_sync(0xffffffffu, mine, (lw + LOADERS * n) & 15);
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          if (filled && !__all_sync(0xffffffffu, mbar_test(&kv_empty[ring.slot], ring.parity ^ 1))) {
            // about to wait: hand over everything that is under way first
            cp_wait<0>();
            announce(0);
            ok = warp_wait(&kv_empty[ring.slot], ring.parity ^ 1, DEV_TIMEOUT_PIPE);
            if (!ok) break;
          }
          const uint32_t dst = smb + L::RING + ring.slot * L::STAGE;
          if (whole && tma) {
            // every key of the block is there: boxes of a page's slots and 64 features, a lane a box
            if (untold) {
              cp_wait<0>();
              announce(0);
            }
            if (lw == 0) {
              if (lane == 0) mbar_arrive_expect_tx(&kv_full[ring.slot], L::STAGE);
              __syncwarp();
              const int box = min(1 << a.b.page_shift, MAX_BOX), part = lane % (D / 64), key = lane / (D / 64) * box;
              const int page = __shfl_sync(0xffffffffu, pages, (key >> 3) & 15);
              if (key < UK)
                tma_load_4d(dst + part * L::HALF + key * 128, kv ? &vmap : &kmap, 64 * part,
                            (j0 + key) & ((1 << a.b.page_shift) - 1), hk, page, &kv_full[ring.slot]);
            } else if (lane == 0) {
              mbar_arrive(&kv_full[ring.slot]);
            }
            ring.next();
            told_slot = ring.slot;
            filled = filled || ring.slot == 0;
            continue;
          }
          const uint16_t* src = static_cast<const uint16_t*>(kv ? a.v : a.k) + mine_at;
          if (whole) {
#pragma unroll
            for (int n = 0; n < RUNS; ++n) {
              const int run = lw + LOADERS * n;
              const uint16_t* p = src + off[n];
              if (run < 16) {
#pragma unroll
                for (int k = 0; k < PER_RUN; ++k) cp_async16(dst + dst0[k] + run * 1024, p + k * rows, 16u);
              }
            }
          } else {
#pragma unroll 1
            for (int run = lw; run < 16; run += LOADERS) {
              const int64_t at = __shfl_sync(0xffffffffu, mine, run);
              const int k0 = cur.x.from - j0 - 8 * run - r0, k1 = hi - j0 - 8 * run - r0;
#pragma unroll
              for (int k = 0; k < PER_RUN; ++k) {
                const bool in = at >= 0 && k * RPI >= k0 && k * RPI < k1;
                cp_async16(dst + dst0[k] + run * 1024, in ? src + at + k * rows : src - mine_at, in ? 16u : 0u);
              }
            }
          }
          cp_commit();
          ++untold;
          ring.next();
          filled = filled || ring.slot == 0;
          if (untold > 2) {
            cp_wait<2>();
            announce(2);
          }
        }
        if (!ok) break;
        if (i == 0) {
          // the tile's queries, when the previous tile's are done with
          cp_wait<0>();
          announce(0);
          if (tile > 0) ok = warp_wait(q_empty, (tile - 1) & 1, DEV_TIMEOUT_PIPE);
          if (!ok) break;
          // 32 rows at a time: lane l finds where row l is, then the warp copies RPI rows an instruction
          const int q_rows = cur.x.r1 - cur.x.r0;
          for (int b0 = 32 * lw; b0 < q_rows; b0 += 32 * LOADERS) {
            const int64_t at =
                b0 + lane < q_rows ? row_offset(cur.s, a.group, hk, cur.x.r0 + b0 + lane, a.ldq, D) : -1;
            const uint32_t qdst = smb + L::Q + (b0 >> 7) * L::STAGE + (c >> 3) * L::HALF + (b0 & 127) * 128;
#pragma unroll 4
            for (int k = 0; k < 32 / RPI; ++k) {
              const int r = k * RPI + r0;
              const int64_t off = __shfl_sync(0xffffffffu, at, r);
              cp_async16(qdst + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                         static_cast<const uint16_t*>(a.q) + (off >= 0 ? off + 8 * c : 0), off >= 0 ? 16u : 0u);
            }
          }
          cp_commit();
          cp_wait<0>();
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(q_full);
        }
      }
      advance(units);
    }
    cp_wait<0>();
    if (ok) announce(0);
    if (*abort_flag) {
      // some wait ran out: boxes may still be under way, and nobody waits for them any more
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 200000ull) {
      }
    }
  } else if (warp == 0) {
      // ------------------------------------------------ MMA issue
      constexpr uint32_t IDESC_S = idesc_16_f32(128, 128, CT == MOEX_BF16, false);
      constexpr uint32_t IDESC_O = idesc_16_f32(128, D, CT == MOEX_BF16, true);
      const uint64_t qd = smem_desc_sw128(smb + L::Q);
      const uint64_t kd = smem_desc_sw128(smb + L::RING);
      const uint64_t vd = smem_desc_mn_sw128(smb + L::RING, L::HALF);
      Ring<NS> kr, vr;  // the stages of the next keys and values
      vr.next();
      uint32_t qp = 0, pp[2] = {0, 0}, op[2] = {1, 1};  // parities; the first O finds its columns free
      bool ok = true;
      auto first = [&](int g, int slot) {  // S_g = Q_g K^T
        const uint64_t kb = kd + slot * (L::STAGE >> 4), qb = qd + g * (L::STAGE >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * L::HALF + (ks & 3) * 32) >> 4;
          mma_f16_ss_elect(tmem + g * 128, qb + off, kb + off, IDESC_S, ks != 0);
        }
        mma_commit_elect(&s_full[g]);
      };
      auto second = [&](int g, int slot, bool acc) {  // O_g (+)= P_g V
        const uint64_t vb = vd + slot * (L::STAGE >> 4);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_f16_ts_elect(tmem + 256 + g * 128, tmem + g * 128 + 8 * ks, vb + ks * (2048 >> 4), IDESC_O, acc || ks != 0);
      };
      while (cur.left > 0 && ok) {
        const int units = units_here(a, cur);
        const int groups = cur.x.r1 - cur.x.r0 > 128 ? 2 : 1;
        ok = warp_wait(q_full, qp, DEV_TIMEOUT_MMA) && warp_wait(&kv_full[kr.slot], kr.parity, DEV_TIMEOUT_MMA);
        if (!ok) break;
        qp ^= 1;
        tc_fence_after();
        first(0, kr.slot);
        if (groups == 2) first(1, kr.slot);
        mma_commit_elect(&kv_empty[kr.slot]);
        if (units == 1) mma_commit_elect(q_empty);
        for (int i = 0; i < units; ++i) {
          const bool more = i + 1 < units;
          kr.next2();
          ok = warp_wait(&kv_full[vr.slot], vr.parity, DEV_TIMEOUT_MMA);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (!ok || g >= groups) break;
            if (i == 0) {
              ok = warp_wait(&o_empty[g], op[g], DEV_TIMEOUT_MMA);
              op[g] ^= 1;
            }
            ok = ok && warp_wait(&p_full[g], pp[g], DEV_TIMEOUT_MMA);
            if (!ok) break;
            pp[g] ^= 1;
            tc_fence_after();
            second(g, vr.slot, i > 0);
            if (g == groups - 1) mma_commit_elect(&kv_empty[vr.slot]);
            if (more) {
              if (g == 0) {
                ok = warp_wait(&kv_full[kr.slot], kr.parity, DEV_TIMEOUT_MMA);
                if (!ok) break;
                tc_fence_after();
              }
              first(g, kr.slot);
            } else {
              mma_commit_elect(&o_full[g]);
            }
          }
          if (!ok) break;
          if (more) mma_commit_elect(&kv_empty[kr.slot]);
          if (i + 2 == units) mma_commit_elect(q_empty);
          vr.next2();
        }
        advance(units);
      }
      // the CTA leaves its TMEM and shared memory only when nothing reads them any more
      mma_commit_elect(done);
      mbar_wait(done, 0, nullptr);
      __syncwarp();
  } else {
    // ------------------------------------------------ softmax
    regs_up<192>();
    const int g = (warp - SOFTMAX0) / 4;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lanes 32 * (warp % 4)
    const uint32_t ts = tmem + lanes + g * 128, to = tmem + lanes + 256 + g * 128;
    const int row = g * 128 + (warp & 3) * 32 + lane;
    uint32_t sp = 0, op = 0, mp = 0;  // parities
    bool ok = true;
    // the group's four warps, with a bounded wait
    auto together = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&meet[g]);
      ok = warp_wait(&meet[g], mp, DEV_TIMEOUT_MMA);
      mp ^= 1;
      return ok;
    };
    while (cur.left > 0) {
      const int units = units_here(a, cur);
      if (cur.x.r1 - cur.x.r0 > g * 128) {
        const int r = cur.x.r0 + row;
        const bool in = r < cur.x.r1;
        const int first = cur.x.lo + cur.u * UK, end = cur.x.hi;
        const int32_t* table = a.b.table + cur.b * a.b.table_stride;
        const int top = in ? cur.s.ctx - cur.s.n + a.group.token(r) : -1;
        const int bot = a.window > 0 ? top - a.window : -1;
        float m = -INFINITY, l = 0.f;
        // lane c < 16: the page of keys j + 8 c .. + 7 of a block, read a block ahead (0 where there is none)
        auto fetch_page = [&](int j) {
          j += 8 * lane;
          return lane < 16 && j < end ? __ldg(table + (j >> a.b.page_shift)) : 0;
        };
        int pg = fetch_page(first);
        for (int i = 0; i < units; ++i) {
          const int j0 = first + i * UK;
          // runs of eight keys without a page (also such as no row sees: masked twice)
          const uint32_t bad = __ballot_sync(0xffffffffu, pg < 0 || pg >= a.b.n_pages);
          if (i + 1 < units) pg = fetch_page(first + (i + 1) * UK);
          ok = warp_wait(&s_full[g], sp, DEV_TIMEOUT_MMA);
          if (!ok) break;
          sp ^= 1;
          tc_fence_after();
          uint32_t s[UK / 32][32];
#pragma unroll
          for (int q = 0; q < UK / 32; ++q) tmem_ld32(ts + 32 * q, s[q]);
          tmem_ld_wait();
          // every key seen by every row of the warp?
          const bool clean = __all_sync(0xffffffffu, j0 + UK - 1 <= top && j0 > bot) && bad == 0;
          if (!clean) {
            const int hi = top - j0, lo = bot - j0;  // keys lo < c <= hi of the block are seen
#pragma unroll
            for (int q = 0; q < UK / 32; ++q) {
              // one bit a key
              uint32_t seen = low_bits(hi + 1 - 32 * q) & ~low_bits(lo + 1 - 32 * q);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if ((bad >> (4 * q + k)) & 1u) seen &= ~(0xFFu << (8 * k));
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((seen >> e) & 1u)) s[q][e] = 0xff800000u;  // -inf
            }
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 32; e += 2)
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = max3(mx[q], __uint_as_float(s[q][e]), __uint_as_float(s[q][e + 1]));
          const float top_s = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * a.scale_log2 - prob_up<CT>(GROW);
          const bool grow = top_s > m + GROW || (i == 0 && top_s > m) || (m == -INFINITY && top_s > m);
          if (__any_sync(0xffffffffu, grow)) {
            const float mn = grow ? top_s : m;
            const float f = mn == -INFINITY ? 1.f : fast_exp2(m - mn);
            m = mn;
            l *= f;
            if (i > 0) {
#pragma unroll 1
              for (int q = 0; q < D / 16; ++q) {
                uint32_t o[16];
                tmem_ld16(to + 16 * q, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(to + 16 * q, o);
              }
            }
          }
          const float ref = m == -INFINITY ? 0.f : m;
          const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2), ref2 = pack2(-ref, -ref);
          uint64_t sum[2] = {0, 0};  // pairs of FP32 sums
#pragma unroll
          for (int q = 0; q < UK / 32; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float p0, p1;
              unpack2(fma2(pack2(__uint_as_float(s[q][2 * e]), __uint_as_float(s[q][2 * e + 1])), scale2, ref2), p0, p1);
              p0 = fast_exp2(p0);
              p1 = fast_exp2(p1);
              sum[e & 1] = add2(sum[e & 1], pack2(p0, p1));
              pk[e] = E::pack(p0, p1);
            }
            tmem_st16(ts + 16 * q, pk);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[g]);
          {
            float s0, s1;
            unpack2(add2(sum[0], sum[1]), s0, s1);
            l += s0 + s1;
          }
        }
        if (!ok) break;
        // the tile's (or the range's) output
        const bool whole = units == cur.x.units;
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (cur.u == 0 ? 1 : 0);
        const int64_t off = in ? row_offset(cur.s, a.group, cur.hk, r, a.ldo, D) : -1;
        const int64_t lse_at = row_offset(cur.s, a.group, cur.hk, in ? r : 0, a.n_heads, 1);
        ok = warp_wait(&o_full[g], op, DEV_TIMEOUT_MMA);
        if (!ok) break;
        op ^= 1;
        tc_fence_after();
        const float inv = whole ? (l > 0.f ? __fdiv_rn(1.f, l) : 0.f) : 1.f;
        float* part = a.part + part_offset<MT, D>(slot, row, 0);
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          tmem_ld32(to + 32 * q, o);
          tmem_ld_wait();
          if (q == D / 32 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_empty[g]);
          }
          if (!whole) {
            // lanes side by side: a warp's store is 512 bytes in a row
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(part + (8 * q + e / 4) * 128) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
            if (a.out_f32) {
              store_rows<MOEX_F32>(a.out, off, 32 * q, o, lane);
              store_rows<MOEX_F32>(a.out, off, 32 * q + 16, o + 16, lane);
            } else {
              store_rows<CT>(a.out, off, 32 * q, o, lane);
            }
          }
        }
        if (in) {
          if (!whole)
            *reinterpret_cast<float2*>(a.part + 2 * static_cast<int64_t>(gridDim.x) * MT * D + (slot * MT + row) * 2) =
                make_float2(m, l);
          else if (a.lse)
            a.lse[lse_at] = row_lse(m, l);
        }
      }
      if (!together()) break;  // the cursor has been read
      if (warp == SOFTMAX0 + 4 * g && lane == 0) next_tile<MT, UK, DEAD>(a, cur, units);
      if (!together()) break;
    }
  }
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == SOFTMAX0) tmem_dealloc(tmem, 512);
}

// Tensor map of a plane: features, slots of a page, key heads, pages.  Pages of
// fewer than MIN_BOX slots have none, since shorter boxes are bound by the box rate
// (the chunk measured above took 350 us with cp.async at any page size, by TMA
// 325 us with pages of 64, 353 us with 32, 450 us with 16; packed prompts with pages
// of 32 61.4 and 59.8 us), nor have strides of 0; then the copies are cp.async
// throughout.
bool plane_map(CUtensorMap* m, const void* base, const AttnArgs& a, int D, int n_pages) {
  const EncodeTiledFn fn = encode_tiled_fn();
  if (!fn || (1 << a.b.page_shift) < MIN_BOX || a.b.row_stride <= 0 || a.b.page_stride <= 0 || (a.n_kv_heads > 1 && a.b.head_stride <= 0)) return false;
  const cuuint32_t page = 1u << a.b.page_shift;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), page, static_cast<cuuint64_t>(a.n_kv_heads),
                              static_cast<cuuint64_t>(n_pages)};
  const int64_t head_stride = a.n_kv_heads > 1 ? a.b.head_stride : a.b.row_stride;
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(a.b.row_stride) * 2, static_cast<cuuint64_t>(head_stride) * 2,
                                 static_cast<cuuint64_t>(a.b.page_stride) * 2};
  const cuuint32_t box[4] = {64, page < MAX_BOX ? page : MAX_BOX, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CT, int D>
cudaError_t launch(const AttnArgs& a, int ctas, cudaStream_t s) {
  const cudaError_t e = ensure_smem(reinterpret_cast<const void*>(attend_tile_kernel<CT, D>), Lay<D>::BYTES);
  if (e != cudaSuccess) return e;
  CUtensorMap kmap = {}, vmap = {};
  const int tma = plane_map(&kmap, a.k, a, D, a.b.n_pages) && plane_map(&vmap, a.v, a, D, a.b.n_pages);
  return launch_pdl(attend_tile_kernel<CT, D>, dim3(ctas), dim3(THREADS), Lay<D>::BYTES, s, a, kmap, vmap, tma);
}

}  // namespace

cudaError_t launch_attend_tile(const AttnArgs& a, int type, int D, int ctas, cudaStream_t s) {
  if (type == MOEX_BF16) return D == 64 ? launch<MOEX_BF16, 64>(a, ctas, s) : launch<MOEX_BF16, 128>(a, ctas, s);
  return D == 64 ? launch<MOEX_F16, 64>(a, ctas, s) : launch<MOEX_F16, 128>(a, ctas, s);
}

}  // namespace moex
