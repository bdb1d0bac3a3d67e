// Arguments of the cache and mixing kernels (kvcache.hip, attention.hip,
// linattn.hip), filled on the host after every check (api.hip).
#pragma once

#include "q4nx_dev.h"

namespace q4nx {

// Bits of a call's flags.
constexpr uint32_t kFlagIndex = 1;    // a slot or page outside the cache
constexpr uint32_t kFlagLength = 2;   // lengths that do not fit (attention)
constexpr uint32_t kFlagDecay = 2;    // a decay above 0 (linear attention)
constexpr uint32_t kFlagRows = 4;     // row ranges that do not fit (linear attention)

__device__ __forceinline__ void set_flag(uint32_t* flags, uint32_t bit) {
  if (flags) atomicOr(flags, bit);
}

// N products of which each takes operands from LDS: read(n) gives them, mul(n, v)
// uses them.  G are read while the G before them are used; the scheduler, left
// alone, either reads each right before its product and waits, or reads them all
// and runs out of registers.
template <int G, int N, typename Read, typename Mul>
__device__ __forceinline__ void fed(Read read, Mul mul) {
  static_assert(N % G == 0, "whole groups");
  decltype(read(0)) v[2][G];
#pragma unroll
  for (int n = 0; n < G; ++n) v[0][n] = read(n);
#pragma unroll
  for (int g = 0; g < N / G; ++g) {
    if (g + 1 < N / G) {
#pragma unroll
      for (int n = 0; n < G; ++n) v[(g + 1) & 1][n] = read(G * g + G + n);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < G; ++n) mul(G * g + n, v[g & 1][n]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// ---------------------------------------------------------------------------
// the paged cache
// ---------------------------------------------------------------------------
struct KvCache {
  void* k;
  void* v;
  float* ks;       // scales, or null (bf16)
  float* vs;
  int32_t heads, dim, page_shift, n_pages;
};

// Element of (page, head, token of the page, dimension).  A key's eight
// dimensions and a dimension's eight tokens lie together: what one lane hands
// to a matrix instruction.
__device__ __forceinline__ size_t kv_page(const KvCache& c, int page, int head) {
  return (((size_t)page * c.heads + head) << c.page_shift) * c.dim;
}
__device__ __forceinline__ int k_place(int dim, int tok, int d) {
  return (tok >> 4) * 16 * dim + (d >> 3) * 128 + (tok & 15) * 8 + (d & 7);
}
__device__ __forceinline__ int v_place(int dim, int tok, int d) {
  return (tok >> 3) * 8 * dim + d * 8 + (tok & 7);
}

struct HeadRows {
  const void* p;
  int64_t ld;
  int32_t heads;
  int32_t bf16;
};

struct AppendArgs {
  KvCache c;
  HeadRows q, k, v;
  uint16_t* q_out;
  const float* inv_freq;   // null: nothing turns
  const int32_t* pos;
  const int32_t* slots;
  uint32_t* flags;
  int32_t M, rot, interleaved, tile;   // tile: rows of a workgroup
};
constexpr int kAppendTile = 8;
// Tiles of a whole eight begin where the first row's run of slots does, so that there may be one more.
inline int append_tiles(const AppendArgs& a) { return (a.M + a.tile - 1) / a.tile + (a.tile == kAppendTile ? 1 : 0); }
hipError_t launch_kv_append(const AppendArgs& a, int head_parts, hipStream_t s);

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
constexpr int kAttnUnit = 128;      // keys that parts are counted in
constexpr int kAttnMaxSeq = 1024;

// Rows of one kernel and what they attend to.
enum AttnSet : int {
  ATTN_ALL = 0,      // every sequence's rows, with the prefix before its own keys
  ATTN_OWN = 1,      // every sequence's rows with its own keys
  ATTN_PREFIX = 2,   // all rows as one, with the prefix
};

// What a set's kernel leaves for the join: from the third int on, each entry's
// first part and parts a row tile.
struct AttnParts {
  int32_t* plan;     // [2 + 2 * entries]
  float* o;          // [part][tile rows][dim], not divided by the sum
  float* ml;         // [part][tile rows][2]: maximum (log2), sum
  int32_t rows;      // of a tile
  int32_t set;       // AttnSet
  int32_t slots;     // workgroups that run at once
  int32_t shares;    // the shares of a batch of more tiles than half of them
};

struct AttnPair { AttnParts p[2]; };   // the sequences', the prefix's

struct AttnArgs {
  KvCache c;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* pages;
  const int32_t* prefix_pages;
  uint32_t* flags;
  int32_t n_seq, M, q_heads, group, pages_ld, prefix_len;
  float scale;       // times log2(e)
};

// Entries of a set.
inline int attn_entries(int set, int n_seq) { return set == ATTN_PREFIX ? 1 : n_seq; }
// Parts at most: each row tile's last part may be short, and the others make up the slots or shares.
inline int64_t attn_max_parts(const AttnParts& p, int n_seq, int64_t rows, int kv_heads) {
  return (rows / p.rows + attn_entries(p.set, n_seq)) * kv_heads + (p.slots > p.shares ? p.slots : p.shares);
}
// Tiles of own: 16, 32 or 128 rows; of the prefix: own's or 128 (rows = 0: no prefix, or with the sequences).
hipError_t launch_attn(const AttnArgs& a, const AttnParts& own, int own_grid, const AttnParts& pre, int pre_grid, hipStream_t s);
// own: the set of the sequences; prefix: of the prefix, or rows = 0
hipError_t launch_attn_join(const AttnArgs& a, const AttnParts& own, const AttnParts& prefix, hipStream_t s);

// ---------------------------------------------------------------------------
// linear attention
// ---------------------------------------------------------------------------
struct LinearArgs {
  const uint16_t *q, *k, *v;
  int64_t q_ld, k_ld, v_ld, decay_ld;
  const float* decay;
  const float* state;
  float* state_out;
  float* out;
  const int32_t* q_start;
  const int32_t* slots;
  const int32_t* fresh;
  uint32_t* flags;
  int32_t k_heads, v_heads, dk, dv, n_seq, n_slots, M;
  float scale;
  // prompts: rows of a segment (a multiple of 64), and, where a sequence may have several, in the workspace
  int32_t seg;
  int32_t* plan;       // [n_seq + 1] first segment of each sequence
  double* seg_decay;   // [segment][v_heads] sum of its decays, -Inf if one of them has exp 0
  float* seg_state;    // [segment][v_heads][dk][dv], or null: a sequence is one segment
};
hipError_t launch_linear_rows(const LinearArgs& a, hipStream_t s);
// items: segments at most
hipError_t launch_linear_chunks(const LinearArgs& a, int items, hipStream_t s);

}  // namespace q4nx
