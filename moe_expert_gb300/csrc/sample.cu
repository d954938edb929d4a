// A token a row of logits: temperature, top-k, top-p and min-p at a given
// random number.
//
// A row is one cluster's: each CTA keeps its slice of the logits in shared
// memory, so they are read from memory once whatever the settings ask for, and
// what the CTAs have to know of one another (the largest logit, histograms, the
// few tokens around a cut, masses) goes through distributed shared memory.
//
// No sort: a cut (the last token of the first top_k, or of those that reach
// top_p) is a weight (a count, a mass) up to which the falling order is followed.
// A histogram over the distance to the largest logit names the bin in which the
// weight is reached, and the few tokens of that bin are ranked against one another;
// where they are many (equal logits), finer histograms over (logit, index) as one
// 64-bit number come first, each 2^8 finer, so nine at most.  The token itself is
// found by running sums: CTA, warp's chunk, thread, four logits.
//
// e = exp((x - largest) / T) is taken as an integer in units of 2^-43: sums over
// 2^18 tokens are exact in 64 bits and do not depend on any order, at less than
// FP32's error of e itself (a tail of 2^18 tokens below 2^-44 of the likeliest
// one's probability, 2^-26 of its mass together, counts as 0).
//
// Latency bounds few rows (steps of a cluster one after the other: 3 to 5 joint
// barriers), instructions and the shared memory of a row, which lets some 50 rows of 128256
// run at a time, many.  Measured, device time: one row of 128256, top-k 50 and top-p
// 0.95, 8.7 us; top-p alone 17.9 us; 64 rows of 128256 by settings of their own, top-p,
// 53.4 us (48 rows 42.3); 200 rows of 50001 BF16, min-p, 16.9 us.
#include <cooperative_groups.h>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace cg = cooperative_groups;

namespace moex {

struct SampleArgs {
  const void* logits;
  const float* u;
  int32_t* ids;
  float* prob;  // or nullptr
  int64_t ldl;
  int V, chunk;  // chunk: logits of a warp; a slice has WARPS of them
  moex_sampling set;
  uint32_t* status;
};

namespace {

constexpr int BINS = 256, MAX_CLUSTER = 8;
constexpr int CAP = 192;   // tokens that are ranked against one another, two threads each
constexpr int LIST = 512;  // tokens of a bin that a CTA keeps

// Order of the tokens as one 64-bit number, larger first: the logit's bits as an
// ordered integer, then the complement of the index.
__device__ __forceinline__ uint32_t logit_key(float x) {
  const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);  // -0 and 0 are equal logits
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ uint64_t rank_key(float x, int i) {
  return static_cast<uint64_t>(logit_key(x)) << 32 | ~static_cast<uint32_t>(i);
}

// Powers of two that x lies below the largest logit, times 1 / T (0, and not NaN, for +inf below +inf).
__device__ __forceinline__ float depth(float x, float top, float c) { return fmaxf((top - x) * c, 0.f); }

__device__ __forceinline__ float exp2_below(float y) {  // 2^-y
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-y));
  return e;
}
// A sum of up to 100 masses in units of 2^-43, as hi * 2^23 + lo: an FP32 number added to 8, rounded down, has its bits
// down to 2^-20 in the low word, and what is left, added to 2^-20, those down to 2^-43, rounded to the nearest.  The words'
// bits are added, and the two numbers' own taken off at the end.
struct MassSum {
  uint32_t hi = 0, lo = 0, n = 0;
  __device__ __forceinline__ float add(float e) {  // e to the nearest unit, which is what was added
    const float t = __fadd_rd(e, 8.f), less = t - (8.f + 0x1p-20f), r = e - less;
    hi += __float_as_uint(t), lo += __float_as_uint(r), ++n;
    return less + r;
  }
  __device__ __forceinline__ uint64_t whole() const {
    return (static_cast<uint64_t>(hi - n * __float_as_uint(8.f)) << 23) + (lo - n * __float_as_uint(0x1p-20f));
  }
};
__device__ __forceinline__ uint64_t mass_of(float e) {
  MassSum s;
  s.add(e);
  return s.whole();
}
__device__ __forceinline__ float in_units(float e) {
  MassSum s;
  return s.add(e);
}

// Sixteenths of a power of two downwards from 1, as a mass's own bits give them: bin b of e = 2^-(b / 8) (1 - r 2^-24),
// b % 8 the upper three bits of r's 23; BINS - 1 for what lies beyond.  A bin's sum has to be that of its tokens' masses to
// the last unit, so that a cut which the sum puts into a bin is found among the bin's tokens: e is a whole number of units
// here (below 2^-20 FP32 holds finer ones), which the sum's own four additions leave: rounding by two more took 64 rows of
// 128256 54.3 us in place of 53.4, in a second pass, for cuts below 2^-20 only, 55.2.
__device__ __forceinline__ uint32_t below_one(float e) { return 0x3F800000u - __float_as_uint(e); }

// x in [0, 1) in units of 2^-64, exactly from 2^-41 on: shares of 64-bit sums are then integer products (FP64 arithmetic
// in every thread took 3 us of a row).
__device__ __forceinline__ uint64_t fraction(float x) {
  const uint32_t b = __float_as_uint(x);
  const int up = static_cast<int>(b >> 23) - 86;
  const uint64_t m = b & 0x7FFFFFu | 0x800000u;
  return up >= 0 ? m << up : up > -24 ? m >> -up : 0;
}

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

struct Shared {
  union {
    uint32_t hist[3][BINS];  // weights of the bins
    struct {
      uint64_t all[CAP], mass[CAP];  // the row's tokens of a cut's bin
    };
  };
  uint64_t list[LIST];                             // this CTA's
  uint64_t best[MAX_CLUSTER], total[MAX_CLUSTER];  // of every CTA, written by each
  uint64_t range[2];                               // lowest and highest in the bin
  uint64_t part[32], found[4];
  uint64_t sum, skipped;                           // mass of the slice; of a bin's tokens in front of those listed
  uint32_t n_list;
};

// Threads of a CTA: FEW where every CTA has an SM of its own, MANY, three CTAs an SM where slices are of 16384 logits at most
// (two with rows of 151936, one with rows of 262144), otherwise.  Measured, device time,
// one row of 128256 FP32 logits with top-k 50 and top-p 0.95 / with top-p alone: 384 threads 8.7 / 21.4 us, 512
// 8.7 / 19.3, 768 10.1 / 20.7, 1024 10.9 / 21.2; 64 rows with top-p alone / 200 rows of 50001 with min-p: 384 threads
// three an SM 55.1 / 17.1 us, 512 two an SM 52.6 / 21.4.
constexpr int FEW = 512, MANY = 384;
static_assert(2 * CAP <= MANY && MANY <= FEW && BINS <= MANY, "two threads a ranked token, one a bin");

template <int TYPE, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) sample_kernel(const SampleArgs a) {
  constexpr int WARPS = THREADS / 32, PER = (LIST + THREADS - 1) / THREADS;
  constexpr bool NARROW = TYPE == MOEX_F32;
  extern __shared__ __align__(16) float xs[];
  __shared__ Shared sh;
  const cg::cluster_group cluster = cg::this_cluster();
  const int peers = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int row = blockIdx.x / peers, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cluster.barrier_arrive();  // a peer's shared memory may be written once the peer runs
  pdl_wait();
  pdl_launch_dependents();

  // ---- the slice: `here` logits from index `from` on (from may be below 0: rows begin anywhere, reads at 16 bytes)
  using T = typename RowElem<TYPE>::T;
  constexpr int N = 16 / sizeof(T);
  const T* x = static_cast<const T*>(a.logits) + row * a.ldl;
  const int here = WARPS * a.chunk, from = rank * here - static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  float most = -INFINITY;  // of this thread
  auto edge = [&](int i) { return i >= 0 && i < a.V ? RowElem<TYPE>::get(x[i]) : -INFINITY; };
  if constexpr (N == 4) {
    // copies of whole fours, all in flight at once
    for (int j = 4 * threadIdx.x; j < here; j += 4 * THREADS) {
      const int i = from + j;
      if (i >= 0 && i + 4 <= a.V)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(xs + j)), "l"(x + i) : "memory");
      else
        *reinterpret_cast<float4*>(xs + j) = make_float4(edge(i), edge(i + 1), edge(i + 2), edge(i + 3));
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 4
    for (int j = 4 * threadIdx.x; j < here; j += 4 * THREADS) {
      const float4 v = *reinterpret_cast<const float4*>(xs + j);
      most = fmaxf(fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)), most);
      if (isnan(v.x + v.y + v.z + v.w))  // NaN is masked too (and infinities of both signs come by here)
        *reinterpret_cast<float4*>(xs + j) =
            make_float4(fmaxf(v.x, -INFINITY), fmaxf(v.y, -INFINITY), fmaxf(v.z, -INFINITY), fmaxf(v.w, -INFINITY));
    }
  } else {
#pragma unroll 4
    for (int j = N * threadIdx.x; j < here; j += N * THREADS) {
      const int i = from + j;
      float f[N];
      if (i >= 0 && i + N <= a.V) {
        load8<TYPE>(x, i, f);
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k) f[k] = edge(i + k);
      }
#pragma unroll
      for (int k = 0; k < N; ++k) {
        f[k] = fmaxf(f[k], -INFINITY);
        most = fmaxf(most, f[k]);
      }
#pragma unroll
      for (int k = 0; k < N; k += 4) *reinterpret_cast<float4*>(xs + j + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
    }
  }
  // The largest number of the cluster, each CTA's put into every one's shared memory.
  auto largest = [&](uint64_t v) {
    v = warp_max(v);
    if (lane == 0) sh.part[warp] = v;
    __syncthreads();
    if (warp == 0) {
      v = warp_max(lane < WARPS ? sh.part[lane] : 0);
      if (lane < peers) *cluster.map_shared_rank(&sh.best[rank], lane) = v;
    }
    cluster.sync();
    return warp_max(lane < peers ? sh.best[lane] : 0);
  };
  cluster.barrier_wait();
  const uint32_t top_key = static_cast<uint32_t>(largest(logit_key(most)));
  const float top = key_logit(top_key);

  const float u = a.u[row], temp = a.set.temperature ? a.set.temperature[row] : a.set.temperature_all;
  const float p = a.set.top_p ? a.set.top_p[row] : a.set.top_p_all;
  const float m = a.set.min_p ? a.set.min_p[row] : a.set.min_p_all;
  const int top_k = a.set.top_k ? a.set.top_k[row] : a.set.top_k_all;
  const bool bad = isnan(u) || !(temp >= 0.f) || isinf(temp) || isnan(p) || isnan(m), none = bad || top == -INFINITY;
  if (none || temp == 0.f) {
    int first = -1;
    if (!none) {  // the first of the largest
      uint64_t at = 0;
      for (int j = threadIdx.x; j < here; j += THREADS)
        if (xs[j] == top) at = max(at, static_cast<uint64_t>(~static_cast<uint32_t>(from + j)));
      cluster.sync();  // the largest logits have been read
      first = static_cast<int>(~static_cast<uint32_t>(largest(at)));
    }
    if (rank == 0 && threadIdx.x == 0) {
      if (bad) flag_status(a.status, DEV_BAD_TOKEN);
      a.ids[row] = first;
      if (a.prob) a.prob[row] = none ? 0.f : 1.f;
    }
    return;  // nothing of a peer is read from here on
  }
  const uint64_t best = static_cast<uint64_t>(top_key) << 32 | 0xFFFFFFFFu;
  const float c = fminf(__fdiv_rn(1.4426950408889634f, temp), 3e38f);
  const float least = fminf(fmaxf(m, 0.f), 1.f);
  const float at_u = fminf(fmaxf(u, 0.f), 0x1.fffffep-1f);
  auto want_of = [](float share, uint64_t total) {  // the least weight that `share` (below 1) of the total asks for, 1 at least
    const uint64_t f = fraction(fmaxf(share, 0.f));
    return max(static_cast<uint64_t>(__umul64hi(total, f)) + (total * f != 0 ? 1 : 0), uint64_t(1));
  };
  auto e_of = [&](float v) { return exp2_below(depth(v, top, c)); };
  // Counts go by the distance to the largest logit at temperature 1, in bins of 1/STEPS of a power of two that are twice as
  // wide from 64 steps on, and again from 192 and 448: 41 in a logit are told apart, and where the cut lies further down,
  // another 41 from the largest there on.  (Bins of an eighth to 22 in a logit, then finer ones over the numbers: top-k 40 of
  // a row whose largest logit lies 30 above the others 60 us in place of 8, 60 above 60 in place of 32; 1000 of 256 rows of
  // 32000 43 in place of 47.)  Masses go by below_one.
  constexpr float STEPS = 16.f, BASE = 64.f;
  float origin = top;  // or the largest of the tokens that the last bin held
  auto count_bin = [&](float v) {
    const float y = fminf(depth(v, origin, 1.4426950408889634f * STEPS), 15.f * BASE - 1.f) + BASE;
    return static_cast<int>((__float_as_uint(y) - __float_as_uint(BASE)) >> 17);
  };
  auto count_edge = [&](int bin) { return (__uint_as_float(__float_as_uint(BASE) + (static_cast<uint32_t>(bin) << 17)) - BASE) / STEPS; };
  auto mass_bin = [&](float v) { return static_cast<int>(min(below_one(in_units(e_of(v))) >> 20, BINS - 1u)); };
  // Logits between which a bin lies, with room for roundings: those outside need no closer look.
  auto near_bin = [&](bool by_count, int bin, float& low, float& high) {
    low = -INFINITY, high = INFINITY;
    const float from = by_count ? origin : top, k = by_count ? 1.4426950408889634f : c;
    if (isinf(from)) return;
    float y0, y1;
    if (by_count) {
      y0 = count_edge(bin), y1 = count_edge(bin + 1);
    } else {
      y0 = (bin >> 3) - log2f(1.f - (bin & 7) / 16.f), y1 = (bin >> 3) - log2f(1.f - ((bin & 7) + 1) / 16.f);
    }
    // FP32's largest relative error of a difference, a product and the exponential, many times over
    high = from - (y0 - 1e-4f * y0 - 1e-4f) / k;
    if (bin < BINS - 1) low = from - (y1 + 1e-4f * y1 + 1e-4f) / k;
    high += 1e-6f * fabsf(high), low -= 1e-6f * fabsf(low);
  };
  // A slice's logits in fours: f(index of the first, the four).
  auto fours = [&](auto&& f) {
#pragma unroll 2
    for (int j = 4 * threadIdx.x; j < here; j += 4 * THREADS) {
      const float4 v = *reinterpret_cast<const float4*>(xs + j);
      const float w[4] = {v.x, v.y, v.z, v.w};
      f(j, w);
    }
  };
  // The few of them in [low, high], one by one: f(index, logit).
  auto between = [&](float low, float high, auto&& f) {
#pragma unroll 2
    for (int j = 4 * threadIdx.x; j < here; j += 4 * THREADS) {
      const float4 v = *reinterpret_cast<const float4*>(xs + j);
      const float w[4] = {v.x, v.y, v.z, v.w};
      uint32_t in = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) in |= w[k] >= low && w[k] <= high ? 1u << k : 0u;
      for (; in; in &= in - 1) {
        const float u = xs[j + __ffs(in) - 1];
        if (u > -INFINITY) f(from + j + __ffs(in) - 1, u);
      }
    }
  };
  // Over all CTAs, a thread a bin: its weight, and that of the bins in front with it; the total.  planes: words of 15
  // bits, or 0: counts and sums of r's lower 20 bits (`crowded` where such a sum may have left its word).
  uint64_t bin_w = 0, bin_sum = 0, bin_n = 0;
  auto read_bins = [&](int planes, bool& crowded) {
    bin_w = bin_n = 0;
    if (threadIdx.x < BINS) {
      uint32_t most_n = 0;
      uint64_t word[3] = {0, 0, 0};
      const int words = planes == 0 ? 2 : planes;
      for (int i = 0; i < words; ++i) {
        uint32_t h[MAX_CLUSTER];  // every CTA's asked for before the first is looked at
#pragma unroll
        for (int r = 0; r < MAX_CLUSTER; ++r) h[r] = r < peers ? *cluster.map_shared_rank(&sh.hist[i][threadIdx.x], r) : 0u;
        uint64_t sum = 0;
#pragma unroll
        for (int r = 0; r < MAX_CLUSTER; ++r) sum += h[r], most_n = i == 0 ? max(most_n, h[r]) : most_n;
        if (i == 0) word[0] = sum;
        if (i == 1) word[1] = sum;
        if (i == 2) word[2] = sum;
      }
      bin_n = word[0];
      if (planes == 0) {
        crowded = most_n >= 1u << 12;
        // units of 2^-43: (n (2^24 - upper three bits of r) - sum) 2^(19 - b / 8), which leaves no remainder
        const uint64_t e = word[0] * ((1u << 24) - ((threadIdx.x & 7u) << 20)) - word[1];
        const int up = 19 - (static_cast<int>(threadIdx.x) >> 3);
        bin_w = up >= 0 ? e << up : e >> -up;
        if (warp == BINS / 32 - 1) {
          const uint64_t mass = warp_sum(lane < peers ? *cluster.map_shared_rank(&sh.sum, lane) : 0);
          if (lane == 31) bin_w = mass;  // of all; less the other bins, below
        }
      } else {
        bin_w = word[0] + (word[1] << 15) + (word[2] << 30);
      }
    }
    bin_sum = bin_w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t v = __shfl_up_sync(0xffffffffu, bin_sum, o);
      if (lane >= o) bin_sum += v;
    }
    if (lane == 31) sh.part[warp] = bin_sum;
    __syncthreads();
    uint64_t total = 0;
    for (int i = 0; i < BINS / 32; ++i) {
      if (i < warp) bin_sum += sh.part[i];
      total += sh.part[i];
    }
    if (planes == 0 && threadIdx.x == BINS - 1) {
      // the last bin's is what the others leave of all
      bin_sum = bin_w;
      bin_w -= total - bin_w;
      sh.found[0] = bin_sum;
    }
    if (planes == 0) {
      __syncthreads();
      total = sh.found[0];
      __syncthreads();
    }
    return total;
  };
  auto clear = [&]() {
    for (int i = threadIdx.x; i < 3 * BINS; i += THREADS) sh.hist[i / BINS][i % BINS] = 0;
    if (threadIdx.x == 0) sh.n_list = 0, sh.sum = 0, sh.skipped = 0, sh.range[0] = ~uint64_t(0), sh.range[1] = 0;
    __syncthreads();
  };
  auto add_mass = [&](int b, uint64_t w) {
    const uint32_t w0 = w & 0x7FFFu, w1 = w >> 15 & 0x7FFFu, w2 = static_cast<uint32_t>(w >> 30);
    if (w0) atomicAdd(&sh.hist[0][b], w0);
    if (w1) atomicAdd(&sh.hist[1][b], w1);
    if (w2) atomicAdd(&sh.hist[2][b], w2);
  };
  // All CTAs' lists in sh.all with their masses, when they are CAP at most; their number.
  auto gather = [&]() {
    // every warp has the lists' lengths, a lane a CTA, and copies every WARPS-th list
    const int len = lane < peers ? static_cast<int>(*cluster.map_shared_rank(&sh.n_list, lane)) : 0;
    int end = len;
#pragma unroll
    for (int o = 1; o < MAX_CLUSTER; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += v;
    }
    const int n = __shfl_sync(0xffffffffu, end, MAX_CLUSTER - 1);
    if (n > CAP) return n;
    for (int r = warp; r < peers; r += WARPS) {
      const int k = __shfl_sync(0xffffffffu, len, r), front = __shfl_sync(0xffffffffu, end, r) - k;
      const uint64_t* list = cluster.map_shared_rank(&sh.list[0], r);
      for (int i = lane; i < k; i += 32) {
        const uint64_t key = list[i];
        sh.all[front + i] = key;
        sh.mass[front + i] = mass_of(e_of(key_logit(static_cast<uint32_t>(key >> 32))));
      }
    }
    __syncthreads();
    return n;
  };

  uint64_t last = 0;  // the last token of the order that stays
  // One cut: the first top_k, or the tokens up to top_p of the mass, of those from `last` on.
  auto cut = [&](bool by_count) {
    uint64_t lo = last, hi = best, above = 0, want = by_count ? top_k : 0;
    // What a bin's mass is counted by: its tokens and the sum of their r, 20 bits of which lie below a bin's size, if
    // no bin has 2^12 tokens of a CTA; else 15 bits a word (`wide`).  A token whose e is below (1 - top_p) / V cannot
    // stay (all such together are less than what may go, since the likeliest one's e is 1), and is not binned.
    bool fine = false, wide = last != 0;
    const uint32_t far = min(below_one(fminf((1.f - fmaxf(p, 0.f)) / a.V * 0.99f, 1.f)), (BINS - 1u) << 20);
    int shift = 0;
    bool listed = false;
    uint64_t held[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) held[i] = 0;
    float near_low = -INFINITY, near_high = INFINITY;
    for (int level = 0; level < 11; ++level) {
      clear();
      auto bin_at = [&](float v, uint64_t key) {
        return fine ? static_cast<int>((hi - key) >> shift) : by_count ? count_bin(v) : mass_bin(v);
      };
      auto count = [&](uint64_t key) {
        const float v = key_logit(static_cast<uint32_t>(key >> 32));
        if (by_count)
          atomicAdd(&sh.hist[0][bin_at(v, key)], 1u);
        else
          add_mass(bin_at(v, key), mass_of(e_of(v)));
      };
      if (by_count && !fine) {
        fours([&](int, const float(&v)[4]) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (v[k] > -INFINITY && v[k] <= origin) atomicAdd(&sh.hist[0][count_bin(v[k])], 1u);
        });
      } else if (!wide) {
        MassSum sum;  // of all the slice's logits
        fours([&](int, const float(&v)[4]) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t d = below_one(sum.add(e_of(v[k])));
            if (d < far) {
              atomicAdd(&sh.hist[0][d >> 20], 1u);
              atomicAdd(&sh.hist[1][d >> 20], d & 0xFFFFFu);
            }
          }
        });
        const uint64_t here_mass = warp_sum(sum.whole());
        if (lane == 0) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.sum), here_mass);
      } else if (listed) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (held[i] >= lo && held[i] <= hi) count(held[i]);
      } else {
        between(near_low, near_high, [&](int i, float v) {
          const uint64_t key = rank_key(v, i);
          if (key >= lo && key <= hi) count(key);
        });
      }
      cluster.sync();
      bool crowded = false;
      const int words = by_count ? 1 : wide || fine ? 3 : 0;
      const uint64_t total = read_bins(words, crowded);
      if (__syncthreads_or(crowded)) {
        wide = true;
        cluster.sync();  // the bins have been read
        continue;
      }
      if (!by_count && !fine) want = want_of(p, total);
      if (!fine && want >= above + total) return;  // all of them stay
      if (threadIdx.x < BINS && above + bin_sum >= want && above + bin_sum - bin_w < want) {
        sh.found[0] = threadIdx.x;
        sh.found[1] = above + bin_sum - bin_w;
        sh.found[2] = bin_w;
        sh.found[3] = bin_n;
      }
      __syncthreads();
      const int bin = static_cast<int>(sh.found[0]);
      above = sh.found[1];
      // Of a bin that holds more tokens than are ranked, those near the place that its mass in front of the cut points to,
      // and the mass of the others in front of these; all of it where the cut is not among them.  This saves a flat row its
      // finer histogram (one row of 262144 28.2 us in place of 32.7, 64 of 128256 53.8 in place of 58.1), but not rows
      // of 16 bits, where a bin holds a few different logits only (one of 262144 BF16 40.3 in place of 35.3), and is no
      // gain for counts (1000 of 256 rows of 32000 44.2 in place of 43.0).
      bool narrow = false;
      float low_in = -INFINITY, high_in = INFINITY;
      if (!fine) {
        near_bin(by_count, bin, near_low, near_high);
        narrow = NARROW && words == 0 && sh.found[3] > CAP && near_low > -INFINITY && near_high < INFINITY;
        if (narrow) {
          const float at = __fdiv_rn(__ull2float_rn(want - above), __ull2float_rn(sh.found[2]));
          const float half = __fdiv_rn(0.375f * CAP, __ull2float_rn(sh.found[3])), width = near_high - near_low;
          high_in = near_high - (at - half) * width, low_in = near_high - (at + half) * width;
        }
      }
      uint64_t low = ~uint64_t(0), high = 0, skipped = 0;
      // tokens that no lists hold are not listed (with three words they are not counted)
      const bool list = words == 3 || sh.found[3] <= static_cast<uint64_t>(LIST) * peers;
      auto keep = [&](uint64_t key) {
        if (list || narrow) {
          const uint32_t n = atomicAdd(&sh.n_list, 1u);
          if (n < LIST) sh.list[n] = key;
        }
        low = min(low, key), high = max(high, key);
      };
      int n;
      for (;;) {
        if (listed) {
#pragma unroll
          for (int i = 0; i < PER; ++i)
            if (held[i] >= lo && held[i] <= hi && bin_at(0.f, held[i]) == bin) keep(held[i]);
        } else {
          between(narrow ? low_in : near_low, near_high, [&](int i, float v) {
            const uint64_t key = rank_key(v, i);
            if (key >= lo && key <= hi && bin_at(v, key) == bin) {
              if (narrow && v > high_in)
                skipped += mass_of(e_of(v));
              else
                keep(key);
            }
          });
        }
        if (low <= high) {
          atomicMin(reinterpret_cast<unsigned long long*>(&sh.range[0]), low);
          atomicMax(reinterpret_cast<unsigned long long*>(&sh.range[1]), high);
        }
        if (skipped) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.skipped), skipped);
        cluster.sync();
        n = list || narrow ? gather() : CAP + 1;
        if (!narrow) break;
        if (n <= CAP) {
          const uint64_t front = above + warp_sum(lane < peers ? *cluster.map_shared_rank(&sh.skipped, lane) : 0);
          uint64_t in = 0;
          for (int k = lane; k < n; k += 32) in += sh.mass[k];
          if (front < want && front + warp_sum(in) >= want) {
            above = front;
            break;
          }
        }
        narrow = false, skipped = 0;
        cluster.sync();  // the lists have been read
        if (threadIdx.x == 0) sh.n_list = 0;
        __syncthreads();
      }
      if (n > CAP) {  // finer: over the numbers in this bin, which this CTA has in its list if they are not too many
        const bool again = by_count && !fine && bin == BINS - 1 && origin == top;  // the same bins from the bin's largest on
        fine = wide = !again;
        listed = !again && list && sh.n_list <= LIST;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int at = threadIdx.x + i * THREADS;
          held[i] = listed && at < static_cast<int>(sh.n_list) ? sh.list[at] : 0;
        }
        const Shared* s = cluster.map_shared_rank(&sh, lane < peers ? lane : 0);
        const uint64_t peer_lo = s->range[0], peer_hi = s->range[1];
        lo = ~warp_max(~peer_lo), hi = warp_max(peer_hi);
        shift = max(0, 64 - __clzll(static_cast<long long>(hi - lo)) - 8);
        if (again) origin = key_logit(static_cast<uint32_t>(hi >> 32));
        cluster.sync();  // the lists and ranges have been read
        continue;
      }
      // two threads a token: the weight in front of it
      const int i = threadIdx.x >> 1;
      uint64_t before = 0;
      const uint64_t key = i < n ? sh.all[i] : 0;
      if (i < n)
        for (int k = threadIdx.x & 1; k < n; k += 2)
          if (sh.all[k] > key) before += by_count ? 1 : sh.mass[k];
      before += __shfl_xor_sync(0xffffffffu, before, 1);
      if (threadIdx.x == 0) sh.found[0] = ~uint64_t(0);
      __syncthreads();
      if (i < n && above + before < want) atomicMin(reinterpret_cast<unsigned long long*>(&sh.found[0]), key);
      __syncthreads();
      last = sh.found[0];
      return;
    }
  };

  if (top_k > 0 && top_k <= CAP / 2) {
    // A bin that holds, with those in front, top_k threads' largest logits holds top_k tokens: all up to it are few
    // and are gathered, and the rest is the work of the cluster's first CTA.
    clear();
    if (most > -INFINITY) atomicAdd(&sh.hist[0][count_bin(most)], 1u);
    cluster.sync();
    bool crowded = false;
    const uint64_t total = read_bins(1, crowded), want = min(static_cast<uint64_t>(top_k), total);
    if (threadIdx.x < BINS && bin_sum >= want && bin_sum - bin_w < want) sh.found[0] = threadIdx.x;
    __syncthreads();
    // (with fewer threads than tokens asked for, all that are not masked)
    const int bin = total < static_cast<uint64_t>(top_k) ? BINS - 1 : static_cast<int>(sh.found[0]);
    float near_low, near_high;
    near_bin(true, bin, near_low, near_high);
    between(near_low, INFINITY, [&](int i, float v) {
      if (count_bin(v) > bin) return;
      const uint32_t n = atomicAdd(&sh.n_list, 1u);
      if (n < LIST) sh.list[n] = rank_key(v, i);
    });
    cluster.sync();
    const int n = gather();
    if (n <= CAP) {
      cluster.barrier_arrive();  // the others' lists have been read
      if (rank == 0) {
        // ranks, masses in front, the cut at top_p and min_p, and the running sum by index, all against one another
        const int i = threadIdx.x >> 1, half = threadIdx.x & 1;
        const uint64_t key = i < n ? sh.all[i] : 0, own = i < n ? sh.mass[i] : 0;
        uint64_t before = 0;
        int in_front = 0;
        if (i < n)
          for (int k = half; k < n; k += 2)
            if (sh.all[k] > key) before += sh.mass[k], ++in_front;
        before += __shfl_xor_sync(0xffffffffu, before, 1);
        in_front += __shfl_xor_sync(0xffffffffu, in_front, 1);
        bool stays = i < n && in_front < top_k;
        if (p < 1.f) {
          const uint64_t s = warp_sum(stays && half == 0 ? own : 0);
          if (lane == 0) sh.part[warp] = s;
          __syncthreads();
          uint64_t all = 0;
          for (int w = 0; w < WARPS; ++w) all += sh.part[w];
          stays = stays && before < want_of(p, all);
        }
        stays = stays && e_of(key_logit(static_cast<uint32_t>(key >> 32))) >= least;
        __syncthreads();
        if (half == 0 && i < n && !stays) sh.mass[i] = 0;
        __syncthreads();
        uint64_t all = 0, run = 0;
        for (int k = half; k < n; k += 2) {
          const uint64_t e = sh.mass[k];
          all += e;
          if (~static_cast<uint32_t>(sh.all[k]) < ~static_cast<uint32_t>(key)) run += e;
        }
        all += __shfl_xor_sync(0xffffffffu, all, 1);
        run += __shfl_xor_sync(0xffffffffu, run, 1);
        const uint64_t t = __umul64hi(all, fraction(at_u));
        if (half == 0 && stays && run <= t && t < run + own) {
          a.ids[row] = static_cast<int>(~static_cast<uint32_t>(key));
          if (a.prob) a.prob[row] = __fdiv_rn(__ull2float_rn(own), __ull2float_rn(all));
        }
      }
      cluster.barrier_wait();
      return;
    }
    cluster.sync();  // too many in one bin: the lists have been read
  }
  if (top_k > 0) {
    cut(true);
    if (p < 1.f) cluster.sync();  // what the cut left in shared memory has been read
  }
  if (p < 1.f) cut(false);

  // ---- what stays: masses by warp's chunk, CTA and cluster, then the token
  const float last_x = last ? key_logit(static_cast<uint32_t>(last >> 32)) : -INFINITY;
  // min_p's border, with room for roundings: logits below need no closer look
  const float low_x = isinf(top) || least == 0.f ? last_x : fmaxf(last_x, top - (-log2f(least) + 1e-3f) * 1.001f / c - 1e-6f * fabsf(top));
  // Up to the last token's index its own logit stays, behind it only larger ones (none, as a comparison with NaN, above
  // infinity).
  const float above_x = last ? key_logit(static_cast<uint32_t>(last >> 32) + 1) : -INFINITY;
  const int last_j = static_cast<int>(~static_cast<uint32_t>(last)) - from;
  auto kept = [&](float v, float border) {  // e of a logit, where it stays
    const float e = e_of(v);
    return v >= border && e >= least ? e : 0.f;
  };
  uint64_t sum = 0;
  {
    MassSum all;
#pragma unroll 2
    for (int j = warp * a.chunk + 4 * lane; j < (warp + 1) * a.chunk; j += 128) {
      const float4 v = *reinterpret_cast<const float4*>(xs + j);
      float w[4] = {v.x, v.y, v.z, v.w};
      if (!__any_sync(0xffffffffu, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) >= low_x)) continue;
      const float border = j <= last_j ? last_x : above_x;
      if (j <= last_j && last_j < j + 3) {  // one four of the row
#pragma unroll
        for (int k = 1; k < 4; ++k)
          if (j + k > last_j && !(w[k] >= above_x)) w[k] = -INFINITY;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) all.add(kept(w[k], border));
    }
    sum = warp_sum(all.whole());
  }
  if (lane == 0) sh.part[warp] = sum;
  __syncthreads();
  if (warp == 0) {
    const uint64_t t = warp_sum(lane < WARPS ? sh.part[lane] : 0);
    if (lane < peers) *cluster.map_shared_rank(&sh.total[rank], lane) = t;
  }
  cluster.sync();  // nothing of a peer is read or written from here on
  uint64_t total = 0, front = 0;
  for (int r = 0; r < peers; ++r) {
    const uint64_t t = sh.total[r];
    if (r < rank) front += t;
    total += t;
  }
  const uint64_t want = __umul64hi(total, fraction(at_u));  // below the total: at_u is below 1
  if (want < front || want >= front + sh.total[rank]) return;
  int w = 0;
  while (want >= front + sh.part[w]) front += sh.part[w++];
  __syncthreads();  // part is used again
  const int per = a.chunk / 32 / WARPS + (a.chunk / 32 % WARPS != 0), j0 = w * a.chunk + threadIdx.x * per;
  uint64_t own = 0;
  for (int k = 0; k < per; ++k)
    if (threadIdx.x * per + k < a.chunk) own += mass_of(kept(xs[j0 + k], j0 + k <= last_j ? last_x : above_x));
  uint64_t run = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t v = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += v;
  }
  if (lane == 31) sh.part[warp] = run;
  __syncthreads();
  for (int k = 0; k < warp; ++k) run += sh.part[k];
  run += front;
  if (run <= want || run - own > want) return;
  run -= own;
  for (int k = 0; k < per; ++k) {
    const uint64_t e = threadIdx.x * per + k < a.chunk ? mass_of(kept(xs[j0 + k], j0 + k <= last_j ? last_x : above_x)) : 0;
    if (run <= want && want < run + e) {
      a.ids[row] = from + j0 + k;
      if (a.prob) a.prob[row] = __fdiv_rn(__ull2float_rn(e), __ull2float_rn(total));
    }
    run += e;
  }
}

template <int TYPE, int THREADS, int CTAS>
cudaError_t launch(SampleArgs a, int n_rows, int cluster, cudaStream_t s) {
  // (a row that begins off 16 bytes takes up to 7 places more)
  const int warps = THREADS / 32, per_warp = (a.V + 7 + cluster * warps - 1) / (cluster * warps);
  a.chunk = (per_warp + 127) / 128 * 128;
  const size_t smem = static_cast<size_t>(warps) * a.chunk * 4;
  const cudaError_t e = ensure_smem(reinterpret_cast<const void*>(sample_kernel<TYPE, THREADS, CTAS>), smem);
  if (e != cudaSuccess) return e;
  return launch_cluster(sample_kernel<TYPE, THREADS, CTAS>, dim3(static_cast<unsigned>(n_rows * cluster)), dim3(THREADS), cluster,
                        smem, s, a);
}

template <int TYPE>
cudaError_t launch(const SampleArgs& a, int n_rows, cudaStream_t s) {
  // CTAs of a row: slices of at most 16384 logits, while a cluster has CTAs (up to 131072 logits; of 32768 beyond: 64 rows
  // of 151936 67 us, of 262144 189); with few rows, as many CTAs as a cluster has, while every CTA of every
  // row has an SM of its own (FEW's registers let one run on an SM; 16 rows of 128256 in 16 clusters of 8, where 15 run at
  // a time: 13.2 us, by MANY 10.7; 37 rows of 5000 in clusters of 4, where 36 do: 7.6, of 2: 5.2).
  const auto alone = [](int cluster) {
    return resident_clusters(reinterpret_cast<const void*>(sample_kernel<TYPE, FEW, 1>), FEW, cluster, 0);
  };
  int cluster = 1;
  while (cluster < MAX_CLUSTER && cluster * 16384 < a.V) cluster *= 2;
  while (cluster < MAX_CLUSTER && a.V > 1024 * cluster && n_rows <= alone(2 * cluster)) cluster *= 2;
  return n_rows <= alone(cluster) ? launch<TYPE, FEW, 1>(a, n_rows, cluster, s) : launch<TYPE, MANY, 3>(a, n_rows, cluster, s);
}

}  // namespace

moex_status launch_sample(const void* logits, int type, int64_t ldl, int n_rows, int V, const float* u,
                          const moex_sampling* settings, int32_t* ids, float* prob, cudaStream_t s) {
  uint32_t* status = device_status_ptr();
  if (!status) return MOEX_ECUDA;
  const SampleArgs a{logits, u, ids, prob, ldl, V, 0, *settings, status};
  switch (type) {
    case MOEX_BF16: return cuda_status(launch<MOEX_BF16>(a, n_rows, s));
    case MOEX_F16: return cuda_status(launch<MOEX_F16>(a, n_rows, s));
    default: return cuda_status(launch<MOEX_F32>(a, n_rows, s));
  }
}

}  // namespace moex
