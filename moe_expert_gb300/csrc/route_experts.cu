// Routing to experts: softmax or sigmoid scores, a bias that only moves the
// selection, groups of experts, top-k, renormalised weights.
#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace moex {

struct RouteArgs {
  const void* logits;
  const float* bias;  // or nullptr
  int32_t* ids;
  float* w;
  int64_t ldl;
  float scale;
  int T, k, sigmoid, groups, top_groups, group_top, renorm, group_size;
  int lane_shift;  // log2 of the lanes a group takes
  int vec;         // rows can be read four at a time
};

// Ranks are compared as 32-bit keys whose unsigned order is the order of the
// floats; 0 = not selectable (no such expert, group left out, taken already),
// 1 = masked (below every rank, even -inf).
constexpr uint32_t KEY_NONE = 0, KEY_MASKED = 1;
__device__ __forceinline__ uint32_t rank_key(float f) {
  if (isnan(f)) return KEY_MASKED;
  const uint32_t u = __float_as_uint(f + 0.f);  // -0 ties with +0
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_rank(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// Score of one logit; 0 for a masked one.  `top` and `sum` are the token's
// largest logit and sum of exponentials (softmax).
__device__ __forceinline__ float score_of(float x, int sigmoid, float top, float sum) {
  if (!(x > -INFINITY)) return 0.f;  // -inf, NaN
  if (sigmoid) return __fdiv_rn(1.f, 1.f + expf(-x));
  // an infinite logit ties with the maximum: its exponent is 0, not inf - inf
  return __fdiv_rn(expf(x == top ? 0.f : x - top), sum);
}

// One warp a token.  A group takes 2^lane_shift neighbouring lanes and a lane
// PER experts in a row (the last ones of a group may be none), so that a
// group's rank meets in a few neighbouring lanes and the order of lanes is the
// order of experts.  The selection: a bound that k keys reach, the few keys that
// reach it compacted to one a lane, and each one's place by counting the keys
// before it; the selected experts' scores are computed again from their logits.
// Instructions bound it: 8192 x 256, 8 groups, top-8 takes 9.2 us (1.3 us at the
// copy rate); k arg-max rounds over all keys took 12.4 us there.
// FP32 throughout; expf and IEEE division.
template <int TYPE, int PER>
__global__ void __launch_bounds__(128) route_experts_kernel(const RouteArgs a) {
  __shared__ uint2 found[4][32];  // a warp's candidates: key, expert
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (t >= a.T) return;
  constexpr uint32_t ALL = 0xffffffffu;
  const typename RowElem<TYPE>::T* row = static_cast<const typename RowElem<TYPE>::T*>(a.logits) + t * a.ldl;
  const int g = lane >> a.lane_shift, in_group = (lane & ((1 << a.lane_shift) - 1)) * PER;
  const int e0 = g * a.group_size + in_group;                                // the lane's first expert
  const int n = g < a.groups ? min(max(a.group_size - in_group, 0), PER) : 0;  // and how many it has

  float x[PER];
  float top = -INFINITY;
  if (PER >= 4 && a.vec) {
#pragma unroll
    for (int i = 0; i + 3 < PER; i += 4) {
      float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (i < n) v = load4<TYPE>(row, e0 + i);
      x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = i < n ? RowElem<TYPE>::get(row[e0 + i]) : -INFINITY;
  }
  float sum = 0.f;
  if (!a.sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) top = fmaxf(top, x[i]);  // ignores NaN
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(ALL, top, o));
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += x[i] > -INFINITY ? expf(x[i] == top ? 0.f : x[i] - top) : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(ALL, sum, o);
  }
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const float s = score_of(x[i], a.sigmoid, top, sum);
    key[i] = i >= n ? KEY_NONE : x[i] > -INFINITY ? rank_key(s + (a.bias ? a.bias[e0 + i] : 0.f)) : KEY_MASKED;
  }

  if (a.groups > 1) {
    // the group's best two ranks, then its key in every lane of it
    uint32_t b1 = KEY_NONE, b2 = KEY_NONE;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      b2 = max(b2, min(b1, key[i]));
      b1 = max(b1, key[i]);
    }
    for (int o = 1; o < (1 << a.lane_shift); o <<= 1) {
      const uint32_t o1 = __shfl_xor_sync(ALL, b1, o), o2 = __shfl_xor_sync(ALL, b2, o);
      b2 = max(max(b2, o2), min(b1, o1));
      b1 = max(b1, o1);
    }
    uint32_t mine = b1;
    if (b1 > KEY_MASKED) mine = rank_key(key_rank(b1) + (a.group_top == 2 && b2 > KEY_MASKED ? key_rank(b2) : 0.f));
    int before = 0;  // groups that come first
    for (int h = 0; h < a.groups; ++h) {
      const uint32_t other = __shfl_sync(ALL, mine, h << a.lane_shift);
      before += other > mine || (other == mine && h < g);
    }
    if (before >= a.top_groups) {
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = KEY_NONE;
    }
  }

  // A bound below the k-th largest key: the k-th largest of the lanes' own
  // maxima (equal ones taken together, which only lowers it).
  uint32_t best = key[0];
#pragma unroll
  for (int i = 1; i < PER; ++i) best = max(best, key[i]);
  uint32_t bound = 0;
  for (int r = 0; r < a.k; ++r) {
    bound = __reduce_max_sync(ALL, best);
    if (best == bound) best = KEY_NONE;
  }
  bound = max(bound, KEY_MASKED);
  // The keys from there on, usually a few more than k, one a lane, in the order of experts.
  int count = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) count += key[i] >= bound;
  int at = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(ALL, at, o);
    if (lane >= o) at += y;
  }
  const int total = __shfl_sync(ALL, at, 31);
  at -= count;
  int my_id = 0, rank = lane;
  if (total <= 32) {
    uint2* mine = found[threadIdx.x >> 5];
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] >= bound) mine[at++] = make_uint2(key[i], e0 + i);
    __syncwarp();
    const uint2 c = lane < total ? mine[lane] : make_uint2(KEY_NONE, 0);
    my_id = static_cast<int>(c.y);
    // its place: the keys above it, and the equal ones before it
    rank = lane < total ? 0 : 32;
    for (int j = 0; j < total; ++j) {
      const uint32_t other = __shfl_sync(ALL, c.x, j);
      rank += other > c.x || (other == c.x && j < lane);
    }
  } else {
    // many equal keys: one arg-max a round
#pragma unroll 1
    for (int r = 0; r < a.k; ++r) {
      best = key[0];
#pragma unroll
      for (int i = 1; i < PER; ++i) best = max(best, key[i]);
      const uint32_t m = __reduce_max_sync(ALL, best);
      const int leader = __ffs(__ballot_sync(ALL, best == m)) - 1;
      int which = 0;
#pragma unroll
      for (int i = PER - 1; i >= 0; --i)
        if (key[i] == m) which = i;
      const int e = __shfl_sync(ALL, e0 + which, leader);
      if (lane == r) my_id = e;
      if (lane == leader) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
          if (i == which) key[i] = KEY_NONE;
      }
    }
  }
  const bool chosen = rank < a.k;
  float w = chosen ? score_of(RowElem<TYPE>::get(row[my_id]), a.sigmoid, top, sum) : 0.f;
  if (a.renorm) {
    float all = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(ALL, all, o);
    w = all > 0.f ? __fdiv_rn(w, all) : 0.f;
  }
  if (chosen) {
    a.ids[t * a.k + rank] = my_id;
    a.w[t * a.k + rank] = w * a.scale;
  }
}

template <int TYPE>
static cudaError_t route_launch(const RouteArgs& a, int per, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.T) + 3) / 4)), block(128);
  if (per <= 4) return launch_pdl(route_experts_kernel<TYPE, 4>, grid, block, 0, s, a);
  if (per <= 8) return launch_pdl(route_experts_kernel<TYPE, 8>, grid, block, 0, s, a);
  if (per <= 16) return launch_pdl(route_experts_kernel<TYPE, 16>, grid, block, 0, s, a);
  if (per <= 32) return launch_pdl(route_experts_kernel<TYPE, 32>, grid, block, 0, s, a);
  return launch_pdl(route_experts_kernel<TYPE, 64>, grid, block, 0, s, a);
}

moex_status launch_route_experts(const void* logits, int type, int64_t ldl, const float* bias, int T, int E, int k,
                                 int score, int groups, int top_groups, int group_top, int renorm, float scale,
                                 int32_t* ids, float* w, cudaStream_t s) {
  RouteArgs a{logits, bias,   ids,        w,         ldl,    scale,     T, k, score == MOEX_SCORE_SIGMOID,
              groups, top_groups, group_top, renorm, E / groups};
  // lanes a group: 32 over the groups' count rounded up to a power of two; at most 60 experts a lane (E <= 1024)
  a.lane_shift = 5;
  for (int g = 1; g < groups; g <<= 1) --a.lane_shift;
  const int lanes = 1 << a.lane_shift, per = (a.group_size + lanes - 1) / lanes;
  const uintptr_t bytes = type == MOEX_F32 ? 16 : 8;
  a.vec = a.group_size % 4 == 0 && ldl % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % bytes == 0;
  switch (type) {
    case MOEX_BF16: return cuda_status(route_launch<MOEX_BF16>(a, per, s));
    case MOEX_F16: return cuda_status(route_launch<MOEX_F16>(a, per, s));
    default: return cuda_status(route_launch<MOEX_F32>(a, per, s));
  }
}

}  // namespace moex
