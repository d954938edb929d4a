// What the paged attention kernels share: their arguments, the division of a
// ragged batch into equal shares, and the joining of partial results.
//
// The new tokens of a sequence and the `group` query heads of one key head
// make one list of n * group rows (row r: token r / group, head r % group), so
// every key and value is read once for all of them.  Rows are cut into tiles of
// MT, the keys a tile sees into units of UK, and all units of the batch, in the
// order sequence, key head, tile, keys, into one contiguous range a CTA:
// CTA c of G takes units floor(c W / G) .. floor((c+1) W / G) of W, whatever the
// lengths.  A tile inside one range is finished by its CTA; one that crosses a
// border leaves FP32 partials (unnormalised output, maximum, sum) in the
// workspace, which a second kernel joins in the order of the keys.  Starting a
// tile costs about as much as some units (its queries, its output), so every
// tile counts DEAD units more than it has, in front of its own: the share of a
// CTA with many short tiles holds fewer keys.
//
// Scores, maxima, sums and outputs are FP32.  Probabilities are rounded to the
// cache type for the product with the values: the 16-bit tensor instructions take
// no wider operand beside 16-bit values, and carrying the rest in a second product
// would double that half of the work.  Each is off by at most 2^-8 (BF16) or 2^-11
// (FP16) of itself, as a value of the cache is, whatever the output's type; the sum
// takes them unrounded.
#pragma once

#include "batch.cuh"
#include "rows.cuh"

namespace moex {

// Query heads of a key head, and division of a row index by it: r / n is the
// high word of r * ceil(2^32 / n) as long as r * n < 2^32 (the product is above
// r 2^32 / n by less than r < 2^32 / n); magic 0 where rows may be more.
struct HeadGroup {
  int n;
  uint32_t magic;
  __device__ __forceinline__ int token(int row) const {
    if (n == 1) return row;
    return magic ? static_cast<int>(__umulhi(static_cast<uint32_t>(row), magic)) : row / n;
  }
};

// Where a CTA's range begins, for the kernel that joins the tiles cut there.
struct RangeStart {
  int64_t W, tile_u;     // units of the batch; units before the tile's own
  int b, hk, t, u;       // sequence, key head, tile, unit inside the tile
  int units, rows;       // of the tile
  int first, n, ctx, pad;  // of the sequence
};

struct AttnArgs {
  BatchView b;
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;         // or nullptr
  struct RangeStart* plan;  // [G]
  float* part;        // [2 G] tiles of MT x D (part_offset), then [2 G][MT][2]
  int64_t ldq, ldo;
  float scale_log2;   // scale * log2(e): scores are kept in powers of two
  int n_heads, n_kv_heads, window, out_f32;
  int cut;            // whether ranges may cut tiles; otherwise a tile is its first unit's CTA's, and plan and part are null
  HeadGroup group;
};

// A copy of 16 bytes to shared memory; bytes 0: zeros, and src is not read.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr float LN2 = 0.6931471805599453f;

// 2^x within 2^-22 of it, far below the probabilities' rounding; 0 below 2^-126.
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Powers of two that a row's reference for the exponentials lies below its
// maximum, when the maximum may pass it by another 2^grow.  FP16 has most of its
// range above 1 and holds no more than 2^15: taken up, a probability of 2^-29 of
// the largest (with grow 0) still has FP16's 11 bits, where it would be dropped from
// the output, though not from the sum, below 2^-25.  BF16 has FP32's range.
template <int CT>
constexpr float prob_up(float grow) {
  return CT == MOEX_F16 ? 15.f - grow : 0.f;
}

// Log of a row's sum l of exponentials relative to 2^m: -inf for a row without
// keys; a NaN among the scores is in l, though the maximum passes over it.
__device__ __forceinline__ float row_lse(float m, float l) { return l == 0.f ? -INFINITY : m * LN2 + logf(l); }

// One tile of a sequence's rows and the keys that its rows see.
struct Tile {
  int r0, r1;  // rows
  int lo, hi;  // keys [lo, hi)
  int from;    // the first key that a row sees: those in front of it may be anything, and their pages gone
  int units;   // at least one, so that rows without keys are written too
};

template <int MT, int UK>
__device__ __forceinline__ Tile tile_of(const SeqView& s, const HeadGroup& group, int window, int t) {
  Tile x;
  x.r0 = t * MT;
  x.r1 = min(s.n * group.n, x.r0 + MT);
  const int base = s.ctx - s.n;
  x.hi = max(base + group.token(x.r1 - 1) + 1, 0);
  x.from = window > 0 ? min(max(base + group.token(x.r0) - window + 1, 0), x.hi) : 0;
  // whole runs of eight keys for the copies; in the kernel of large tiles whole blocks, so that a block
  // begins where a box of the cache does
  constexpr int ALIGN = MT >= 128 ? UK : 16;
  x.lo = x.from & ~(ALIGN - 1);
  x.units = max((x.hi - x.lo + UK - 1) / UK, 1);
  return x;
}

// Units of a sequence and key head: few tiles by one thread; many by a warp,
// its lanes taking them in turn.
constexpr int FEW_TILES = 6;
template <int MT, int UK, int DEAD>
__device__ __forceinline__ int seq_units_few(const SeqView& s, const HeadGroup& group, int window) {
  int u = 0;
#pragma unroll 1
  for (int t = 0; t * MT < s.n * group.n; ++t) u += tile_of<MT, UK>(s, group, window, t).units + DEAD;
  return u;
}
template <int MT, int UK, int DEAD>
__device__ __forceinline__ int64_t seq_units_warp(const SeqView& s, const HeadGroup& group, int window) {
  const int tiles = (s.n * group.n + MT - 1) / MT;
  int64_t u = 0;
  for (int t = threadIdx.x & 31; t < tiles; t += 32) u += tile_of<MT, UK>(s, group, window, t).units + DEAD;
  if (!__any_sync(0xffffffffu, u >> 25)) return __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(u));
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
  return u;
}

// (32-bit division where the numbers allow it: there are at most a few hundred CTAs.)
__device__ __forceinline__ int64_t range_begin(int64_t c, int64_t W, int G) {
  const int64_t n = c * W;
  return n >> 32 ? n / G : static_cast<uint32_t>(n) / static_cast<uint32_t>(G);
}
// The CTA whose range holds unit u.
__device__ __forceinline__ int64_t range_of(int64_t u, int64_t W, int G) {
  const int64_t n = (u + 1) * G - 1;
  return (n | W) >> 32 ? n / W : static_cast<uint32_t>(n) / static_cast<uint32_t>(W);
}

// Where a CTA is in the list of units.
struct Cursor {
  int64_t left;    // units of this CTA's range from here on, the next tile's dead ones taken off
  int b, hk, t, u; // sequence, key head, tile, unit inside the tile
  SeqView s;
  Tile x;
};

// To the first unit of the next tile; `done` units of this one were in the range.
template <int MT, int UK, int DEAD>
__device__ __forceinline__ void next_tile(const AttnArgs& a, Cursor& cur, int done) {
  cur.left -= done + DEAD;
  cur.u = 0;
  if (cur.left <= 0) return;
  ++cur.t;
  if (cur.t * MT >= cur.s.n * a.group.n) {
    cur.t = 0;
    if (++cur.hk == a.n_kv_heads) {
      cur.hk = 0;
      do {
        cur.s = seq_view(a.b, ++cur.b);
      } while (cur.s.n == 0);
    }
  }
  cur.x = tile_of<MT, UK>(cur.s, a.group, a.window, cur.t);
}

// Units of the tile that are this CTA's, from the cursor on.
__device__ __forceinline__ int units_here(const AttnArgs& a, const Cursor& cur) {
  return a.cut ? static_cast<int>(min(cur.left, static_cast<int64_t>(cur.x.units - cur.u))) : cur.x.units;
}

// Inclusive sum over the warp's lanes.
__device__ __forceinline__ int64_t warp_scan(int64_t v) {
  const int lane = threadIdx.x & 31;
  if (__any_sync(0xffffffffu, v >> 25)) {
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    return v;
  }
  int x = static_cast<int>(v);  // 32 of these fit 32 bits
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Units of each lane's sequence and one key head; one of many tiles is counted by the whole warp.
template <int MT, int UK, int DEAD>
__device__ __forceinline__ int64_t lane_units(const AttnArgs& a, const SeqView& s) {
  const bool few = s.n * a.group.n <= FEW_TILES * MT;
  int64_t v = few ? seq_units_few<MT, UK, DEAD>(s, a.group, a.window) : 0;
#pragma unroll 1
  for (uint32_t many = __ballot_sync(0xffffffffu, !few); many; many &= many - 1) {
    const int src = __ffs(many) - 1;
    const SeqView w{0, __shfl_sync(0xffffffffu, s.n, src), __shfl_sync(0xffffffffu, s.ctx, src), false};
    const int64_t u = seq_units_warp<MT, UK, DEAD>(w, a.group, a.window);
    if ((threadIdx.x & 31) == src) v = u;
  }
  return v;
}

// Every CTA finds the batch's number of units and its own range; the cursor is
// at the range's first unit, and so is the CTA's entry of the plan.  For up to
// WARP_SEQS sequences a warp needs no other, a lane a sequence, and a kernel may
// leave it to one warp; for more, all threads of the CTA have to call it.
constexpr int WARP_SEQS = 32;
template <int THREADS>
struct RangeScratch {  // in shared memory, used before the function returns only
  int64_t warp_sum[2][THREADS / 32];
  int64_t before, units;
  SeqView s;
  int b;
  int64_t counted[WARP_SEQS];  // units of a sequence and key head, when the CTA's warps counted them
};
template <int MT, int UK, int DEAD, int THREADS>
__device__ __forceinline__ void find_range(const AttnArgs& a, int cta, int n_cta, Cursor& cur,
                                           RangeScratch<THREADS>& sh, bool counted = false) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t total, u0, before, units;  // of the batch; the range's first; before and in its sequence
  if (a.b.n_seqs <= WARP_SEQS) {
    SeqView s{0, 0, 0, false};
    if (lane < a.b.n_seqs) {
      s = seq_view(a.b, lane);
      if (cta == 0 && (s.bad || uncovered(a.b, lane))) flag_status(a.b.status, DEV_BAD_BATCH);
    }
    int64_t mine = 0;
    if (!counted)
      mine = a.n_kv_heads * lane_units<MT, UK, DEAD>(a, s);
    else if (lane < a.b.n_seqs)
      mine = a.n_kv_heads * sh.counted[lane];
    const int64_t sum = warp_scan(mine);
    total = __shfl_sync(0xffffffffu, sum, 31);
    u0 = range_begin(cta, total, n_cta);
    const uint32_t past = __ballot_sync(0xffffffffu, sum > u0);
    const int src = past ? __ffs(past) - 1 : 0;
    units = __shfl_sync(0xffffffffu, mine, src);
    before = __shfl_sync(0xffffffffu, sum, src) - units;
    cur.b = src;
    cur.s = SeqView{__shfl_sync(0xffffffffu, s.first, src), __shfl_sync(0xffffffffu, s.n, src),
                    __shfl_sync(0xffffffffu, s.ctx, src), false};
  } else {
    int64_t mine = 0, first = 0;
    SeqView s{0, 0, 0, false};
    total = 0;
    // pass 0 finds W (and keeps the one block of a small batch); pass 1 the place of the range's first unit.
    // `it` counts the blocks of both passes: neighbouring blocks use different halves of warp_sum, also where
    // one pass ends and the other begins, so a half is written again only after a barrier behind its readers.
    int it = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      const int64_t want = pass ? range_begin(cta, total, n_cta) : 0;
      int64_t run = 0;
#pragma unroll 1
      for (int base = 0; base < a.b.n_seqs; base += THREADS, ++it) {
        const int b = base + threadIdx.x;
        if (pass == 0 || a.b.n_seqs > THREADS) {
          s = SeqView{0, 0, 0, false};
          if (b < a.b.n_seqs) {
            s = seq_view(a.b, b);
            if (cta == 0 && pass == 0 && (s.bad || uncovered(a.b, b))) flag_status(a.b.status, DEV_BAD_BATCH);
          }
          mine = a.n_kv_heads * lane_units<MT, UK, DEAD>(a, s);
          const int64_t x = warp_scan(mine);
          if (lane == 31) sh.warp_sum[it & 1][warp] = x;
          __syncthreads();
          const int warps = min((a.b.n_seqs - base + 31) / 32, THREADS / 32);
          first = run;
          for (int w = 0; w < warps; ++w) {
            const int64_t ws = sh.warp_sum[it & 1][w];
            if (w < warp) first += ws;
            run += ws;
          }
          first += x - mine;
        }
        if (pass == 1 && mine > 0 && first <= want && want < first + mine) {
          sh.b = b;
          sh.s = s;
          sh.before = first;
          sh.units = mine;
        }
      }
      if (pass == 0)
        total = run;
      else
        __syncthreads();
    }
    u0 = range_begin(cta, total, n_cta);
    before = sh.before;
    units = sh.units;
    cur.b = sh.b;
    cur.s = sh.s;
  }
  cur.left = range_begin(cta + 1, total, n_cta) - u0;
  if (cur.left == 0) {
    if (lane == 0 && a.cut) a.plan[cta] = RangeStart{total, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    return;
  }
  int64_t off = u0 - before;
  const int64_t per =
      units >> 32 ? units / a.n_kv_heads : static_cast<uint32_t>(units) / static_cast<uint32_t>(a.n_kv_heads);
  cur.hk = static_cast<int>((off | per) >> 32 ? off / per : static_cast<uint32_t>(off) / static_cast<uint32_t>(per));
  off -= cur.hk * per;
  cur.t = 0;
  // the tile: 32 at a time, every warp for itself
#pragma unroll 1
  for (int t0 = 0; cur.s.n * a.group.n > MT; t0 += 32) {
    const int t = t0 + lane;
    const int n = t * MT < cur.s.n * a.group.n ? tile_of<MT, UK>(cur.s, a.group, a.window, t).units + DEAD : 0;
    const int64_t sum = warp_scan(n);
    const uint32_t past = __ballot_sync(0xffffffffu, sum > off);
    if (past) {
      const int src = __ffs(past) - 1;
      cur.t = t0 + src;
      off -= __shfl_sync(0xffffffffu, sum - n, src);
      break;
    }
    off -= __shfl_sync(0xffffffffu, sum, 31);
  }
  cur.x = tile_of<MT, UK>(cur.s, a.group, a.window, cur.t);
  const int64_t tile_u = u0 - off + DEAD;
  off -= DEAD;
  if (off < 0) cur.left += off;  // the range begins among the tile's dead units
  cur.u = static_cast<int>(max(off, int64_t(0)));
  if (!a.cut) {
    if (cur.u > 0) next_tile<MT, UK, DEAD>(a, cur, cur.x.units - cur.u);
    return;
  }
  if (lane == 0)  // of every warp that is here: the same values
    a.plan[cta] = RangeStart{total, tile_u, cur.b, cur.hk, cur.t, cur.u, cur.x.units, cur.x.r1 - cur.x.r0,
                             cur.s.first, cur.s.n, cur.s.ctx, 0};
}

// Offset of row r of a tile's sequence and key head in a packed [token][head][D] buffer.
__device__ __forceinline__ int64_t row_offset(const SeqView& s, const HeadGroup& group, int hk, int r, int64_t ld, int D) {
  const int i = group.token(r);
  return (s.first + i) * ld + static_cast<int64_t>(hk * group.n + (r - i * group.n)) * D;
}

// Float offset of columns c .. c + 3 (c a multiple of 4) of a row of partial
// tile `slot`: 32 rows' pieces lie side by side, as a warp of one row a lane
// writes them.
template <int MT, int D>
__device__ __forceinline__ int64_t part_offset(int64_t slot, int row, int c) {
  constexpr int R = MT < 32 ? MT : 32;
  return (slot * MT + row / R * R) * D + (c / 4 * R + row % R) * 4;
}

template <int CT>
__device__ __forceinline__ void store_out4(const AttnArgs& a, int64_t off, float4 v) {
  if (a.out_f32)
    store4<MOEX_F32>(a.out, off, v);
  else
    store4<CT>(a.out, off, v);
}

}  // namespace moex
