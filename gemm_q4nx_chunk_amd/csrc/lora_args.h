// Device-side arguments of the low-rank adapter kernels (one struct, passed by value).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q4nx {

constexpr int kLoraMaxJobs = 8;
constexpr int kLoraMaxRank = 256;
constexpr int kLoraMaxAdapters = 4096;   // the route kernel counts rows per adapter in LDS
constexpr int kLoraMaxRows = 4096;       // activation rows of one call
constexpr int kLoraWaveRows = 64;        // up to here each wave finds its tile's rows itself, 16 at most
constexpr int kLoraShrinkWaves = 8;
constexpr int kLoraStepCols = 64;        // columns of x that a wave multiplies per step
constexpr int kLoraRankGroup = 64;       // ranks of one shrink workgroup
constexpr int kLoraMaxSplit = 8;         // parts of u that the expand adds, four loads at a time

struct LoraJob {
  const uint16_t* a;       // adapter e's A [rank][cols] at a + e * a_stride (elements)
  const uint16_t* b;       // adapter e's B [rows][rank] at b + e * b_stride
  int64_t a_stride, b_stride;
  const float* scale;      // [n_adapters]
  const int32_t* ranks;    // [n_adapters] or null (every adapter has `rank`)
  const float* base;       // [M][rows]
  float* y;                // [M][rows]; may be base
  float* u;                // workspace: [split][M][rank] partial A x
  int32_t rank, rows;
  int32_t wg_begin;        // expand: first workgroup (along grid y) of this job
  int32_t rg_begin;        // shrink: first rank group (along grid z) of this job
};

// A tile of rows of one adapter.
struct LoraTile {
  int32_t e;     // adapter, -1: rows without one
  int32_t cnt;   // rows; 0: no tile
};

struct LoraArgs {
  LoraJob job[kLoraMaxJobs];
  int32_t n_jobs, n_adapters;
  int32_t M, cols;
  int32_t tile_rows;       // 16 or 64
  int32_t more;            // not the call's first rows: the error bit stays set
  int32_t split;           // parts of the columns in the shrink
  int32_t n_range;         // outputs of one expand workgroup
  const uint16_t* x;       // [M][cols]
  const int32_t* ids;      // [M]
  uint32_t* hdr;           // [0]: bit 0 = an id outside [-1, n_adapters)
  int32_t* sorted;         // [max_tiles][tile_rows] each tile's rows (M > kLoraWaveRows)
  LoraTile* tiles;         // [max_tiles]
  int32_t max_tiles;       // grid x
};

// Rows of a tile: 16 where adapters have few rows each (1000 rows of 100
// adapters, rank 64, 4096 x 4096: 45 us, 62 with 64), or the rows are few and
// short, so that more workgroups pay more than each adapter read fewer times
// (512 rows of 4 adapters, rank 64, 4096 x 4096: 23.3 and 25.1 us; 1613 x 2304:
// 20.6 and 23.3; but 1052 x 11264, rank 16: 29.3 and 26.5).  Where the rows stop
// being few depends on the rank and the outputs as well, and 2^22 elements of x
// are on the low side of it: 1024 rows of 4 adapters, 4096 outputs, ranks 16 and
// 64, take 18.3 and 24.5 us with 16 at 5120 columns (21.1 and 28.5 with 64), 19.6
// and 27.0 at 9728 (22.1 and 30.4); 2048 rows 23.4 and 32.8 at 2560 columns (26.7
// and 33.8), 27.7 and 41.6 at 4096 (27.5 and 37.7).
inline int lora_tile_rows(int M, int n_adapters, int cols) {
  const int groups = M < n_adapters + 1 ? M : n_adapters + 1;
  if (M <= kLoraWaveRows || M <= 32 * groups) return 16;
  return M <= 2048 && (int64_t)M * cols <= 1 << 22 ? 16 : 64;
}

// Tiles of rows of one adapter (or of none): whole ones, and at most one short
// one per adapter.  Up to kLoraWaveRows rows, a workgroup per row instead unless
// that is twice as many.
inline int lora_max_tiles(int M, int n_adapters, int tile_rows) {
  const int groups = M < n_adapters + 1 ? M : n_adapters + 1;
  const int tiles = M / tile_rows + groups;
  if (M <= kLoraWaveRows) return 2 * tiles > M ? M : tiles;
  return (tiles + 7) / 8 * 8;   // eight at a time, one on each XCD
}

// Room for M rows or fewer, so that none of it shrinks as M grows: rows of u in
// all its parts (above kLoraWaveRows a split of s > 1 leaves s * M / 64 workgroups
// at most 256), places in the tiles, and tiles.
inline size_t lora_u_rows(int M) { return M < 2048 ? (size_t)kLoraMaxSplit * M : 16384; }
inline size_t lora_places(int M, int n_adapters) {
  return (size_t)M + 64 * ((size_t)(M < n_adapters + 1 ? M : n_adapters + 1) + 7);
}
inline size_t lora_tiles(int M, int n_adapters) {
  return (size_t)M / 16 + (M < n_adapters + 1 ? M : n_adapters + 1) + 7;
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t s);

}  // namespace q4nx
