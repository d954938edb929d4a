// A sequence's tokens and length as the arrays of a batch give them, cut to what
// the batch can hold, whatever the arrays say.  Plain C++, so that the host can
// check it over the whole range of its arguments.
#pragma once

#ifdef __CUDACC__
#define MOEX_BOTH __host__ __device__ __forceinline__
#else
#define MOEX_BOTH inline
#endif

namespace moex {

// One sequence's new tokens and length: its tokens are first .. first + n - 1
// and token i has position ctx - n + i.
struct SeqView {
  int first, n, ctx;
  bool bad;  // something had to be cut
};

MOEX_BOTH int clip(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// lo, hi: the sequence's and the next one's first token; most: positions that
// the page table has.  Always 0 <= first, 0 <= n <= n_tokens - first and
// 0 <= ctx <= most.
MOEX_BOTH SeqView clip_seq(int lo, int hi, int ctx, int n_tokens, int most) {
  SeqView s;
  s.first = clip(lo, 0, n_tokens);
  s.n = clip(hi, s.first, n_tokens) - s.first;  // cut first: hi - first may leave 32 bits
  s.ctx = clip(ctx, 0, most);
  s.bad = s.first != lo || hi < lo || hi > n_tokens || s.ctx != ctx;
  return s;
}

}  // namespace moex
