// Rows of a block-quantized embedding table, scaled.
#include "common.cuh"
#include "internal.h"
#include "rows.cuh"

namespace moex {

// y = scale * (d * q): d * q is exact in FP32 (11 + 8 bits), then one product
// and the rounding to the output's type.  A thread takes a word of quants at a
// time: four values of Q8_0, or the eight of IQ4_NL whose nibbles share four
// bytes (values j and j + 16 of a block), so neighbouring lanes read and write
// whole lines; blockDim.y rows a CTA.  For many tokens the two dependent reads
// (id, row) and the instructions bound it (59% of the issue slots; 8192 rows of 2560,
// IQ4_NL to FP32: 19.3 to 19.7 us, 73% of the copy rate, where a kernel that only writes
// as many bytes takes 12.2; one value's conversion by an integer-to-float instruction and a
// 64-bit division a thread 30.3 us), for few the reads alone.
template <int FMT, int YT>
__global__ void __launch_bounds__(256) embed_kernel(const uint8_t* __restrict__ qs, const uint8_t* __restrict__ scales,
                                                    int64_t rows, int words, int64_t sc_row,
                                                    const int32_t* __restrict__ ids, int T, float scale, void* y,
                                                    int64_t ldy, uint32_t* status) {
  constexpr int WORDS = FMT == MOEX_Q8_0 ? 8 : 4;  // of a block
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (t >= T) return;
  const int64_t row = ids[t];
  const bool in = row >= 0 && row < rows;
  if (!in && threadIdx.x == 0) flag_status(status, DEV_BAD_TOKEN);
  const uint32_t* q = reinterpret_cast<const uint32_t*>(qs) + (in ? row * words : 0);
  const __half* d = reinterpret_cast<const __half*>(scales + (in ? row * sc_row : 0));
#pragma unroll 4
  for (int i = threadIdx.x; i < words; i += blockDim.x) {
    const int block = i / WORDS;
    const float k = in ? __half2float(d[block]) : 0.f;
    const uint32_t w = in ? q[i] : 0u;
    auto values = [&](uint32_t v, int at) {
      store4<YT>(y, t * ldy + at, make_float4(scale * (k * byte_value(v, 0)), scale * (k * byte_value(v, 1)),
                                              scale * (k * byte_value(v, 2)), scale * (k * byte_value(v, 3))));
    };
    if constexpr (FMT == MOEX_Q8_0) {
      values(w, 4 * i);
    } else {
      const int at = block * QK + 4 * (i % WORDS);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t v = (w >> (4 * half)) & 0x0F0F0F0Fu;
        v = (v | v >> 4) & 0x00FF00FFu;
        const uint32_t sel = (v | v >> 8) & 0xFFFFu;
        values(in ? iq4nl_lookup4(sel, sel ^ 0x8888u) : 0u, at + 16 * half);
      }
    }
  }
}

template <int FMT>
static cudaError_t embed_launch(const moex_qweight* W, const int32_t* ids, int T, float scale, void* y, int y_type,
                                int64_t ldy, uint32_t* status, cudaStream_t s) {
  const auto* qs = static_cast<const uint8_t*>(W->qs);
  const auto* sc = static_cast<const uint8_t*>(W->scales);
  const int words = static_cast<int>(W->K / QK) * (FMT == MOEX_Q8_0 ? 8 : 4);
  const int64_t sc_row = (W->K / QK * 2 + 15) / 16 * 16;
  // a row's threads: as many as it has words, up to 256; short rows share a CTA
  int x = 4;
  while (x < 256 && x < words) x *= 2;
  const dim3 block(x, 256 / x), grid((static_cast<unsigned>(T) + block.y - 1) / block.y);
  switch (y_type) {
    case MOEX_BF16:
      return launch_pdl(embed_kernel<FMT, MOEX_BF16>, grid, block, 0, s, qs, sc, W->rows, words, sc_row, ids, T, scale, y,
                        ldy, status);
    case MOEX_F16:
      return launch_pdl(embed_kernel<FMT, MOEX_F16>, grid, block, 0, s, qs, sc, W->rows, words, sc_row, ids, T, scale, y,
                        ldy, status);
    default:
      return launch_pdl(embed_kernel<FMT, MOEX_F32>, grid, block, 0, s, qs, sc, W->rows, words, sc_row, ids, T, scale, y,
                        ldy, status);
  }
}

moex_status launch_embed(const moex_qweight* W, const int32_t* ids, int T, float scale, void* y, int y_type,
                         int64_t ldy, cudaStream_t s) {
  uint32_t* status = device_status_ptr();
  if (!status) return MOEX_ECUDA;
  return cuda_status(W->fmt == MOEX_Q8_0 ? embed_launch<MOEX_Q8_0>(W, ids, T, scale, y, y_type, ldy, status, s)
                                         : embed_launch<MOEX_IQ4_NL>(W, ids, T, scale, y, y_type, ldy, status, s));
}

}  // namespace moex
