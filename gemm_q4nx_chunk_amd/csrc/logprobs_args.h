// Device-side arguments of the log-probability kernels (one struct, passed by value).
#pragma once

#include <algorithm>

#include "q4nx_dev.h"

namespace q4nx {

constexpr int kLogprobMaxK = 32;       // alternatives of a row
constexpr int kLogprobMaxTok = 64;     // given tokens of a row
constexpr int kLogprobMaxN = 1 << 20;  // logits of a row
constexpr int kLogprobMaxParts = 256;  // parts of a row: four lists a lane in the join

struct LogprobArgs {
  const float* y;          // [M] rows of n logits, ldy apart
  int32_t n, ldy, M;
  int32_t k, n_tok;
  int32_t parts, part_n;   // parts of a row, logits of a part
  const int32_t* tokens;   // [M][n_tok]
  float* logp;             // [M][n_tok]
  float* entropy;          // [M] or null
  int32_t* top_ids;        // [M][k]
  float* top_logp;         // [M][k] or null
  f32x4* stats;            // [M][parts]: m, rest, sum e d, -
  uint64_t* keys;          // [M][parts][k], decreasing, 0 past the last
};

constexpr int kLogprobChunk = 2048;    // logits that a wave holds in registers at a time

constexpr int kLogprobMaxChunks = 32;  // chunks of a part

// Fewest parts of a row whose parts have kLogprobMaxChunks chunks at most.  A
// value in a part passes as many additions in its lane as a chunk has values
// there (32) and the part chunks, and its chunk's sum may be rescaled once for
// each chunk after it (1.5 roundings of 2^-23), where the row rises all along:
// 64 additions and 32 rescales keep a sum within 2^-23 (32 + 48) of its value
// whatever the batch.  (Measured with 16384 rows of 151936 level logits: log Z
// within 8e-7; with one running sum a lane over the whole row 3.1e-5, for each
// addition may err the same way.)
inline int logprob_min_parts(int n) {
  const int chunks = (n + kLogprobChunk - 1) / kLogprobChunk;
  return (chunks + kLogprobMaxChunks - 1) / kLogprobMaxChunks;
}

// Logits of a part.  Up to 2048 waves of 1024 logits: those, in one go (16 rows
// of 50001: 10.8 us, 12.8 with 2048 a wave).  Else whole chunks, as many as leave
// about 16384 waves (1000 rows of 151936: 114 us; with 8192 waves 117, with 4096
// 118), for a wave's first chunk costs the most, but no more than the sums allow.
inline int logprob_part_n(int n, int M) {
  if ((int64_t)M * ((n + 1023) / 1024) <= 2048 && n <= kLogprobMaxParts * 1024) return 1024;
  const int chunks = (n + kLogprobChunk - 1) / kLogprobChunk;
  int parts = std::max(16384 / M, logprob_min_parts(n));
  parts = parts > chunks ? chunks : parts;
  parts = parts > kLogprobMaxParts ? kLogprobMaxParts : parts;
  return (chunks + parts - 1) / parts * kLogprobChunk;
}

// Workspace: the parts' stats, then their keys, laid out for the most parts that
// M rows or fewer have (logprob_part_n), so that it does not shrink as M grows.
struct LogprobWsLayout {
  size_t stats, keys, total;
};
inline LogprobWsLayout logprob_ws_layout(int n, int M, int k) {
  const int most = std::min((n + 1023) / 1024, kLogprobMaxParts);
  const size_t units = std::min((size_t)M * most, std::max((size_t)M * logprob_min_parts(n), (size_t)16384));
  LogprobWsLayout l;
  l.stats = 0;
  l.keys = units * 16;
  l.total = (l.keys + units * k * 8 + 255) & ~(size_t)255;
  return l;
}

hipError_t launch_token_logprobs(const LogprobArgs& a, hipStream_t s);

}  // namespace q4nx
