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
  int32_t more;            // not the call's first rows: the error bit stays set
  int32_t split;           // parts of the columns in the shrink
  int32_t n_range;         // outputs of one expand workgroup
  const uint16_t* x;       // [M][cols]
  const int32_t* ids;      // [M]
  uint32_t* hdr;           // [0]: bit 0 = an id outside [-1, n_adapters)
  int32_t* sorted;         // [max_tiles][64] each tile's rows (M > kLoraWaveRows)
  LoraTile* tiles;         // [max_tiles]
  int32_t max_tiles;       // grid x
};

// Tiles of rows of one adapter (or of none): whole ones, and at most one short
// one per adapter.  Up to kLoraWaveRows rows, a workgroup per row instead unless
// that is twice as many.
inline int lora_max_tiles(int M, int n_adapters) {
  const int groups = M < n_adapters + 1 ? M : n_adapters + 1;
  if (M <= kLoraWaveRows) return 2 * (M / 16 + groups) <= M ? M / 16 + groups : M;
  return M / 64 + groups;
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t s);

}  // namespace q4nx
