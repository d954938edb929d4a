// Residual addition and root-mean-square norm with FP32, 16-bit or q8_1
// output, and the values of q8_1 rows.
#include <cfloat>

#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace moex {

struct NormArgs {
  const void* x;
  const float* residual;  // or nullptr; may be sum
  const float* gamma;
  float* sum;             // or nullptr
  void* y;                // or nullptr
  int8_t* q;              // or nullptr
  float* ds;
  int64_t ldx, ldr, lds, ldy;
  float eps;
  int H;
};

// Sum over the CTA, the same value in every thread.
__device__ __forceinline__ float cta_sum(float v, float* part) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0) part[warp] = v;
  __syncthreads();
  v = lane < (blockDim.x >> 5) ? part[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One CTA a row, the row in registers: thread t holds the float4 at
// 4 * (t + i * threads), so the row is read once and written once, and a
// 32-value q8_1 block lies in eight neighbouring lanes (H % 32 == 0).
//   s = x + r;  y = s * rstd * gamma,  rstd = 1 / sqrt(mean(s^2) + eps)
// Sums are FP32 (a tree over threads); the q8_1 arithmetic is that of the
// library's quantiser (IEEE divisions, round half away from zero).
template <int XT, int YT, int CH>
__global__ void __launch_bounds__(1024) add_rms_norm_kernel(const NormArgs a) {
  __shared__ float part[2][32];
  const int n4 = a.H >> 2;
  const int64_t row = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  float4 v[CH];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < n4) {
      v[i] = load4<XT>(a.x, row * a.ldx + 4 * c);
      if (a.residual) {
        const float4 r = load4<MOEX_F32>(a.residual, row * a.ldr + 4 * c);
        v[i].x += r.x, v[i].y += r.y, v[i].z += r.z, v[i].w += r.w;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    ss += v[i].x * v[i].x + v[i].y * v[i].y + (v[i].z * v[i].z + v[i].w * v[i].w);
    if (a.sum && c < n4) store4<MOEX_F32>(a.sum, row * a.lds + 4 * c, v[i]);
  }
  ss = cta_sum(ss, part[0]);
  const int lane = threadIdx.x & 31;
  float rstd;
  if (ss <= FLT_MAX || isnan(ss)) {
    rstd = __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(ss, static_cast<float>(a.H)) + a.eps));
  } else {
    // The squares left FP32's range: once more on the row scaled by 2^-96.  Values are
    // then below 2^32, so 32768 squares fit; and one of the row's is above 2^56 here
    // (2^128 over 32768 squares), so the sum is above 2^-80.  The product with 1 / sqrt
    // is taken before the scaling, which is exact, so small values lose no bits.
    constexpr float DOWN = 1.2621774483536189e-29f;
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const float4 d = make_float4(v[i].x * DOWN, v[i].y * DOWN, v[i].z * DOWN, v[i].w * DOWN);
      ss += d.x * d.x + d.y * d.y + (d.z * d.z + d.w * d.w);
    }
    ss = cta_sum(ss, part[1]);
    rstd = __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(ss, static_cast<float>(a.H)) + a.eps * DOWN * DOWN));
#pragma unroll
    for (int i = 0; i < CH; ++i)
      v[i] = make_float4(v[i].x * rstd * DOWN, v[i].y * rstd * DOWN, v[i].z * rstd * DOWN, v[i].w * rstd * DOWN);
    rstd = 1.f;
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    const bool in = c < n4;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
      const float4 g = load4<MOEX_F32>(a.gamma, 4 * c);
      y = make_float4(v[i].x * rstd * g.x, v[i].y * rstd * g.y, v[i].z * rstd * g.z, v[i].w * rstd * g.w);
      if (a.y) store4<YT>(a.y, row * a.ldy + 4 * c, y);
    }
    if (a.q) {  // uniform over the CTA; lanes past the row take part in the shuffles
      float amax = fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w)));
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float d = __fdiv_rn(amax, 127.0f);
      const float f[4] = {y.x, y.y, y.z, y.w};
      int sum = 0;
      uint32_t packed = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // (a subnormal d may be a third too small, a value then up to 190 of it)
        const int qi = d > 0.f ? min(max(static_cast<int>(roundf(__fdiv_rn(f[j], d))), -127), 127) : 0;
        sum += qi;
        packed |= (static_cast<uint32_t>(qi) & 0xFFu) << (8 * j);
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (in) {
        reinterpret_cast<uint32_t*>(a.q)[row * n4 + c] = packed;
        if ((lane & 7) == 0)
          reinterpret_cast<float2*>(a.ds)[row * (a.H / QK) + (c >> 3)] =
              d > 0.f ? make_float2(d, __fmul_rn(d, static_cast<float>(sum))) : make_float2(0.f, 0.f);
      }
    }
  }
}

template <int XT, int YT>
static cudaError_t norm_launch(const NormArgs& a, int T, cudaStream_t s) {
  // Few rows: as many threads as there are float4s, up to 1024, for the shortest
  // way through a row.  Many rows: CTAs of at most 512 threads, so that an SM holds
  // several rows in different phases and loads while others reduce (8192 x 2560,
  // FP32 in and sum, BF16 out: 320 threads of two float4s 43.9 us, 640 of one
  // 46.6 us, 160 of four 47.8 us; 43.2 us at the copy rate).
  const int n4 = a.H >> 2, most = T > 2 * sm_count() ? 512 : 1024;
  int ch = 1;
  while (ch < 8 && (n4 + ch - 1) / ch > most) ch *= 2;
  const int threads = ((n4 + ch - 1) / ch + 31) / 32 * 32;
  switch (ch) {
    case 1: return launch_pdl(add_rms_norm_kernel<XT, YT, 1>, dim3(T), dim3(threads), 0, s, a);
    case 2: return launch_pdl(add_rms_norm_kernel<XT, YT, 2>, dim3(T), dim3(threads), 0, s, a);
    case 4: return launch_pdl(add_rms_norm_kernel<XT, YT, 4>, dim3(T), dim3(threads), 0, s, a);
    default: return launch_pdl(add_rms_norm_kernel<XT, YT, 8>, dim3(T), dim3(threads), 0, s, a);
  }
}

template <int XT>
static cudaError_t norm_launch_y(const NormArgs& a, int y_type, int T, cudaStream_t s) {
  switch (y_type) {
    case MOEX_BF16: return norm_launch<XT, MOEX_BF16>(a, T, s);
    case MOEX_F16: return norm_launch<XT, MOEX_F16>(a, T, s);
    default: return norm_launch<XT, MOEX_F32>(a, T, s);
  }
}

moex_status launch_add_rms_norm(const void* x, int x_type, int64_t ldx, const float* residual, int64_t ldr,
                                const float* gamma, float eps, int T, int64_t H, float* sum, int64_t lds, void* y,
                                int y_type, int64_t ldy, int8_t* q, float* ds, cudaStream_t s) {
  const NormArgs a{x, residual, gamma, sum, y, q, ds, ldx, ldr, lds, ldy, eps, static_cast<int>(H)};
  switch (x_type) {
    case MOEX_BF16: return cuda_status(norm_launch_y<MOEX_BF16>(a, y_type, T, s));
    case MOEX_F16: return cuda_status(norm_launch_y<MOEX_F16>(a, y_type, T, s));
    default: return cuda_status(norm_launch_y<MOEX_F32>(a, y_type, T, s));
  }
}

// ----------------------------------------------------------------- q8_1 values

// y = d * q, four values a thread (eight threads a block of 32).
template <int YT>
__global__ void __launch_bounds__(256) dequantize_q8_1_kernel(const int8_t* __restrict__ q,
                                                              const float* __restrict__ ds, int64_t n4, void* y) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (t >= n4) return;
  const char4 v = reinterpret_cast<const char4*>(q)[t];
  const float d = ds[2 * (t >> 3)];
  store4<YT>(y, 4 * t,
             make_float4(d * static_cast<float>(v.x), d * static_cast<float>(v.y), d * static_cast<float>(v.z),
                         d * static_cast<float>(v.w)));
}

moex_status launch_dequantize_q8_1(const int8_t* q, const float* ds, int T, int64_t K, void* y, int y_type,
                                   cudaStream_t s) {
  const int64_t n4 = static_cast<int64_t>(T) * K / 4;
  const dim3 grid(static_cast<unsigned>((n4 + 255) / 256));
  switch (y_type) {
    case MOEX_BF16:
      return cuda_status(launch_pdl(dequantize_q8_1_kernel<MOEX_BF16>, grid, dim3(256), 0, s, q, ds, n4, y));
    case MOEX_F16:
      return cuda_status(launch_pdl(dequantize_q8_1_kernel<MOEX_F16>, grid, dim3(256), 0, s, q, ds, n4, y));
    default: return cuda_status(launch_pdl(dequantize_q8_1_kernel<MOEX_F32>, grid, dim3(256), 0, s, q, ds, n4, y));
  }
}

}  // namespace moex
