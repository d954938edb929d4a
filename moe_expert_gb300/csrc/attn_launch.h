// Tile sizes and launchers of the paged attention kernels.
#pragma once

#include <cuda_runtime.h>

namespace moex {

struct AttnArgs;

// DEAD: what starting a tile costs, in units (attn.cuh).  1 to 5 were measured: packed
// prompts 64.1 / 60.9 / 62.5 / 63.3 / 63.3 us, 64 single tokens 150.2 / 151.5 / 151.2 /
// 152.0 / 151.6 us.

// Few rows a key head: tiles of 16 rows, two CTAs an SM.
constexpr int STREAM_MT = 16, STREAM_DEAD = 2, STREAM_CTAS_PER_SM = 2;

// Many rows a key head: tiles of 256 rows, units of 128 keys, one CTA an SM.
constexpr int TILE_MT = 256, TILE_UK = 128, TILE_DEAD = 2;
// The hint (new tokens of the longest sequence x heads a key head) above which the
// large tiles are taken: with more rows than one small tile the streaming kernel
// reads every key once a tile.  Measured, 8 key heads, device time of a call,
// streaming / large tiles: heads of 128, 32 sequences of up to 5000 keys, 16 rows
// 38.7 / 62.1 us, 25 rows 55.5 / 63.9, 64 rows 98.9 / 63.6; 8 sequences of up to 500
// keys, 25 rows 13.9 / 15.3; heads of 64, 32 sequences of up to 5000 keys, 32 rows
// 34.0 / 50.3, 48 rows 45.5 / 49.7, 64 rows 56.6 / 50.1.  (The limit for heads of 128
// is from before the streaming kernel had its present registers, 25 rows 70.9 / 67.3:
// two small tiles would now be the faster choice.)
constexpr int TILE_MIN_ROWS = STREAM_MT, TILE_MIN_ROWS_64 = 3 * STREAM_MT;

cudaError_t launch_attend_stream(const AttnArgs& a, int type, int D, int ctas, cudaStream_t s);
cudaError_t launch_attend_tile(const AttnArgs& a, int type, int D, int ctas, cudaStream_t s);

}  // namespace moex
