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
  int T, E, k, sigmoid, groups, top_groups, group_top, renorm, group_size;
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

// One warp a token; lane l holds experts l + 32 i, i < PER (E <= 32 PER).
// Arg-max rounds take the largest key by redux.sync and the lowest index
// among the lanes that hold it.  FP32 throughout; expf and IEEE division.
template <int TYPE, int PER>
__global__ void __launch_bounds__(128) route_experts_kernel(const RouteArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (t >= a.T) return;
  constexpr uint32_t ALL = 0xffffffffu;
  const typename RowElem<TYPE>::T* row = static_cast<const typename RowElem<TYPE>::T*>(a.logits) + t * a.ldl;

  float s[PER];
  uint32_t open = 0;  // bit i: the expert exists and is not masked
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 32 * i;
    s[i] = e < a.E ? RowElem<TYPE>::get(row[e]) : -INFINITY;
    if (s[i] > -INFINITY) open |= 1u << i;  // false for NaN
    top = fmaxf(top, s[i]);                 // ignores NaN
  }
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = (open >> i) & 1u ? __fdiv_rn(1.f, 1.f + expf(-s[i])) : 0.f;
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(ALL, top, o));
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      // an infinite logit ties with the maximum: its exponent is 0, not inf - inf
      s[i] = (open >> i) & 1u ? expf(s[i] == top ? 0.f : s[i] - top) : 0.f;
      sum += s[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(ALL, sum, o);
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = sum > 0.f ? __fdiv_rn(s[i], sum) : 0.f;
  }
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 32 * i;
    const float b = a.bias && e < a.E ? a.bias[e] : 0.f;
    key[i] = e >= a.E ? KEY_NONE : (open >> i) & 1u ? rank_key(s[i] + b) : KEY_MASKED;
  }

  if (a.groups > 1) {
    // Lane g ends up with the key of group g: the sum of its best one or two
    // unmasked ranks.
    uint32_t gkey = KEY_NONE;
    for (int g = 0; g < a.groups; ++g) {
      const int lo = g * a.group_size, hi = lo + a.group_size;
      uint32_t b1 = KEY_NONE, b2 = KEY_NONE;  // this lane's best two of the group
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        const uint32_t v = e >= lo && e < hi ? key[i] : KEY_NONE;
        b2 = max(b2, min(b1, v));
        b1 = max(b1, v);
      }
      const uint32_t m1 = __reduce_max_sync(ALL, b1);
      uint32_t m = m1;
      if (m1 > KEY_MASKED) {
        float r = key_rank(m1);
        if (a.group_top == 2) {
          const uint32_t who = __ballot_sync(ALL, b1 == m1);
          const uint32_t m2 = __reduce_max_sync(ALL, lane == __ffs(who) - 1 ? b2 : b1);
          if (m2 > KEY_MASKED) r += key_rank(m2);
        }
        m = rank_key(r);
      }
      if (lane == g) gkey = m;
    }
    uint32_t keep = 0;
    for (int r = 0; r < a.top_groups; ++r) {
      const uint32_t m = __reduce_max_sync(ALL, gkey);
      const int g = __ffs(__ballot_sync(ALL, gkey == m)) - 1;
      keep |= 1u << g;
      if (lane == g) gkey = KEY_NONE;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 32 * i;
      if (e < a.E && !((keep >> (e / a.group_size)) & 1u)) key[i] = KEY_NONE;
    }
  }

  float my_w = 0.f;
  int my_id = 0;
  float total = 0.f;
  for (int r = 0; r < a.k; ++r) {
    uint32_t b = KEY_NONE;
    float bs = 0.f;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] > b) {  // ascending e: ties keep the lower index
        b = key[i];
        bs = s[i];
        be = lane + 32 * i;
      }
    const uint32_t m = __reduce_max_sync(ALL, b);
    const int e = static_cast<int>(__reduce_min_sync(ALL, b == m ? static_cast<uint32_t>(be) : 0x7fffffffu));
    const float we = __shfl_sync(ALL, bs, e & 31);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (e == lane + 32 * i) key[i] = KEY_NONE;
    total += we;
    if (lane == r) {
      my_id = e;
      my_w = we;
    }
  }
  if (lane < a.k) {
    if (a.renorm) my_w = total > 0.f ? __fdiv_rn(my_w, total) : 0.f;
    a.ids[t * a.k + lane] = my_id;
    a.w[t * a.k + lane] = my_w * a.scale;
  }
}

template <int TYPE>
static cudaError_t route_launch(const RouteArgs& a, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.T) + 3) / 4)), block(128);
  if (a.E <= 128) return launch_pdl(route_experts_kernel<TYPE, 4>, grid, block, 0, s, a);
  if (a.E <= 256) return launch_pdl(route_experts_kernel<TYPE, 8>, grid, block, 0, s, a);
  if (a.E <= 512) return launch_pdl(route_experts_kernel<TYPE, 16>, grid, block, 0, s, a);
  return launch_pdl(route_experts_kernel<TYPE, 32>, grid, block, 0, s, a);
}

moex_status launch_route_experts(const void* logits, int type, int64_t ldl, const float* bias, int T, int E, int k,
                                 int score, int groups, int top_groups, int group_top, int renorm, float scale,
                                 int32_t* ids, float* w, cudaStream_t s) {
  const RouteArgs a{logits, bias,   ids,        w,         ldl,    scale,     T, E, k, score == MOEX_SCORE_SIGMOID,
                    groups, top_groups, group_top, renorm, E / groups};
  switch (type) {
    case MOEX_BF16: return cuda_status(route_launch<MOEX_BF16>(a, s));
    case MOEX_F16: return cuda_status(route_launch<MOEX_F16>(a, s));
    default: return cuda_status(route_launch<MOEX_F32>(a, s));
  }
}

}  // namespace moex
