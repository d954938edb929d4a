// Tile sizes and launchers of the paged attention kernels.
#pragma once

#include <cuda_runtime.h>

namespace moex {

struct AttnArgs;

// DEAD: what starting a tile costs, in units (attn.cuh).  1 to 5 were measured: packed
// prompts 62.6 / 59.7 / 61.4 / 62.0 / 62.0 us, 64 single tokens 153.7 / 152.3 / 153.5 /
// 154.7 / 155.6 us.

// Few rows a key head: tiles of 16 rows, two CTAs an SM.
constexpr int STREAM_MT = 16, STREAM_DEAD = 2, STREAM_CTAS_PER_SM = 2;

// Many rows a key head: tiles of 256 rows, units of 128 keys, one CTA an SM.
constexpr int TILE_MT = 256, TILE_UK = 128, TILE_DEAD = 2;
// The hint (new tokens of the longest sequence x heads a key head) above which the
// large tiles are taken: with more rows than one small tile the streaming kernel
// reads every key once a tile.  Measured, 8 key heads, device time of a call,
// streaming / large tiles: heads of 128, 32 sequences of up to 5000 keys, 16 rows
// 44.8 / 65.3 us, 25 rows 70.9 / 67.3, 64 rows 130 / 65; 8 sequences of up to 500
// keys, 25 rows 13.1 / 14.6; heads of 64, 32 sequences of up to 5000 keys, 32 rows
// 38.3 / 51.7, 48 rows 52.0 / 52.6, 64 rows 67.2 / 52.3.
constexpr int TILE_MIN_ROWS = STREAM_MT, TILE_MIN_ROWS_64 = 3 * STREAM_MT;

cudaError_t launch_attend_stream(const AttnArgs& a, int type, int D, int ctas, cudaStream_t s);
cudaError_t launch_attend_tile(const AttnArgs& a, int type, int D, int ctas, cudaStream_t s);

}  // namespace moex
