// Tile sizes and launcher of the paged attention kernel over Q8_0 blocks.
#pragma once

#include <cuda_runtime.h>

#include "kv_q8.cuh"

namespace moex {

struct AttnArgs;

// Q8_DEAD: what starting a tile costs, in units (attn.cuh).  Measured, device time, 64 single tokens over contexts to
// 16384 / three to 100001 / drafts: 2 units 103.2 / 42.9 / 14.8 us, 3 98.7 / 42.2 / 15.1, 4 100.9 / 41.8 / 15.2,
// 6 100.9 / 41.4 / 15.8.
constexpr int Q8_WARPS = 4, Q8_DEAD = 3;
// Keys of a warp's step: 4 KB of keys and values with their scales, either way.
constexpr int q8_step(int D) { return D == 64 ? 32 : 16; }
// CTAs an SM, for tiles of 8 NT rows: as many as their registers allow without spilling much.  (Heads of 128, 8 rows: four
// instead of three, 128 registers in place of 168: 103.7 / 41.8 us for the batch and the long contexts, but one token
// over 1003 keys 7.5 us instead of 6.7.)
constexpr int q8_ctas(int D, int NT) { return D == 128 ? (NT == 1 ? 3 : 2) : NT == 1 ? 4 : 3; }

// The most CTAs of a cluster, and the most units of one of them, as far as the host knows (the page table's positions, not
// the lengths on the device): with more, ranges over all SMs and a second kernel that joins them are faster.  Measured, heads of 128, 8 key heads, ranges / clusters: one token over 1000 keys 9.4 / 6.7 us,
// 4000 keys 11.7 / 10.0, 8000 keys (16 units a CTA) 13.2 / 14.6, 16000 keys 18.3 / 24.5; 8 tokens over up to 1000 keys
// 10.9 / 8.6, 2000 keys 11.9 / 11.4, 4000 keys (16 units a CTA) 17.3 / 17.7; 16 tokens over 1000 keys 11.9 / 11.0.
constexpr int Q8_CLUSTER = 8, Q8_CLUSTER_STEPS = 8;

// CTAs of a launch and its workspace: their range starts, then two partial tiles each.
struct Q8Grid {
  bool cut;       // ranges may cut tiles
  int ctas, mt;   // mt: rows of a tile
  int cluster;    // CTAs of a tile's cluster; 0: ranges
  int row_tiles;  // tiles of rows of a sequence and key head that have a cluster of their own
  size_t plan_bytes, bytes;
};

// Clusters of `size` CTAs that run at a time.
int q8_clusters(int D, int mt, int size);

cudaError_t launch_attend_stream_q8(const AttnArgs& a, const ScaleView& sc, int q_type, int D, const Q8Grid& g,
                                    cudaStream_t s);

}  // namespace moex
