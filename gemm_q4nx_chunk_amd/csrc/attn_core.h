// What the attention kernels share: which rows and keys a workgroup has.
#pragma once

#include "kv_args.h"

namespace q4nx {

// The cut of a set into parts, found by every workgroup from the lengths (they
// live on the device, so that a captured graph follows them).  Each entry (a
// sequence, or all rows for the prefix) has row tiles of `rows` rows and
// splits each tile's keys in the same number of parts, one part a key head.
struct AttnPlan {
  int32_t start[kAttnMaxSeq + 1];   // first row of each sequence: rising, in 0..M
  int32_t first[kAttnMaxSeq + 1];   // first part of each entry
  int32_t per;                      // units of keys in a part
  int64_t sums[4];                  // of the waves
};

struct AttnEntry {
  int32_t row0, rows;   // the first row of q, and rows times group
  int32_t own;          // own tokens (0 for the prefix)
  int32_t pre;          // tokens of the prefix that come before them
  int32_t causal;       // own tokens that the first row sees, less one (may be negative); unused for the prefix
  int32_t tiles, units; // row tiles; units of keys that the last tile sees at most
};

__device__ __forceinline__ int attn_units(int keys) { return (keys + kAttnUnit - 1) / kAttnUnit; }

__device__ __forceinline__ AttnEntry attn_entry(const AttnArgs& a, const int32_t* start, int set, int tile_rows, int e) {
  AttnEntry x;
  if (set == ATTN_PREFIX) {
    x.row0 = start[0];
    x.rows = (start[a.n_seq] - start[0]) * a.group;
    x.own = 0;
    x.pre = a.prefix_len;
    x.causal = 0;
  } else {
    const int n = start[e + 1] - start[e];
    x.row0 = start[e];
    x.rows = n * a.group;
    const int64_t most = (int64_t)a.pages_ld << a.c.page_shift;
    const int have = a.kv_len[e];
    x.own = max(0, (int)min((int64_t)have, most));
    x.pre = set == ATTN_ALL ? a.prefix_len : 0;
    x.causal = x.own - n;
  }
  x.tiles = (x.rows + tile_rows - 1) / tile_rows;
  x.units = attn_units(x.pre) + attn_units(x.own);
  return x;
}

// Units of keys in a part, so that parts = sum over tiles of ceil(units / per) <= tiles + target / heads.  Few tiles
// are cut so that all parts fit the GPU at once; where the tiles alone come near that, only what is longer than its
// share is cut, and parts follow one another.
__device__ __forceinline__ int attn_per(const AttnArgs& a, const AttnParts& p, int64_t work, int tiles) {
  const int64_t have = (int64_t)tiles * a.c.heads;
  const int64_t target = have <= p.slots / 2 ? p.slots - have : p.shares;
  const int64_t per = (work * a.c.heads + target - 1) / target;
  return (int)max((int64_t)1, min(per, (int64_t)1 << 30));
}

// Inclusive scan of v over the workgroup's 256 threads; every thread gets the total.
template <typename T, bool MAX>
__device__ __forceinline__ T scan256(T v, int64_t* sums, T& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const T o = __shfl_up(v, off);
    if (lane >= off) v = MAX ? max(v, o) : v + o;
  }
  __syncthreads();   // sums may still be read
  if (lane == 63) sums[wave] = v;
  __syncthreads();
  T before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const T s = (T)sums[i];
    if (i < wave) before = MAX ? max(before, s) : before + s;
    total = MAX ? max(total, s) : total + s;
  }
  return MAX ? max(v, before) : v + before;
}

// Fills the plan; returns the parts of one key head.  All 256 threads call it.
__device__ inline int attn_plan(const AttnArgs& a, const AttnParts& p, AttnPlan& s) {
  const int tid = threadIdx.x, n = a.n_seq;
  // row starts, kept rising and within the rows (starts are >= 0, so 0 is the scan's neutral value)
  {
    int carry = 0, total;
    for (int b = 0; b <= n; b += 256) {
      const int e = b + tid;
      const int raw = e <= n ? a.q_start[e] : 0, v = min(max(raw, 0), a.M);
      const int up = max(scan256<int, true>(v, s.sums, total), carry);
      if (e <= n) {
        s.start[e] = up;
        const bool bad_len = e < n && (a.kv_len[e] < 0 || a.kv_len[e] > (int64_t)a.pages_ld << a.c.page_shift);
        if (blockIdx.x == 0 && (raw != up || bad_len)) set_flag(a.flags, kFlagLength);
      }
      carry = max(carry, total);
    }
  }
  __syncthreads();
  const int entries = p.set == ATTN_PREFIX ? 1 : n;
  int64_t work = 0, total;
  int tiles = 0, all_tiles;
  for (int e = tid; e < entries; e += 256) {
    const AttnEntry x = attn_entry(a, s.start, p.set, p.rows, e);
    work += (int64_t)x.tiles * x.units;
    tiles += x.tiles;
  }
  scan256<int64_t, false>(work, s.sums, total);
  scan256<int, false>(tiles, s.sums, all_tiles);
  const int per = attn_per(a, p, total, all_tiles);
  int carry = 0;
  for (int b = 0; b < entries; b += 256) {
    const int e = b + tid;
    int parts = 0, split = 0;
    if (e < entries) {
      const AttnEntry x = attn_entry(a, s.start, p.set, p.rows, e);
      split = x.tiles ? max(1, (x.units + per - 1) / per) : 0;
      parts = x.tiles * split;
    }
    int all;
    const int up = scan256<int, false>(parts, s.sums, all) + carry;
    if (e < entries) {
      s.first[e] = up - parts;
      if (blockIdx.x == 0) {
        p.plan[2 + 2 * e] = up - parts;
        p.plan[2 + 2 * e + 1] = split;
      }
    }
    carry += all;
  }
  if (tid == 0) {
    s.first[entries] = carry;
    s.per = per;
  }
  __syncthreads();
  return carry;
}

// One part's place: its entry, that entry's first part and number of parts.
struct AttnPlace { int e, first, split; AttnEntry x; };

// A plan of up to 64 entries needs no LDS and no barrier: each wave holds it, an entry a lane.  (One token of 777:
// the kernel 9.7 us with the workgroup's scans, 7.6 us with these.)
struct AttnWavePlan { int start, end, own, units, tiles, split, first, total; };

__device__ __forceinline__ int wave_scan_max(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(v, off);
    if (lane >= off) v = max(v, o);
  }
  return v;
}

__device__ __forceinline__ AttnWavePlan attn_wave_plan(const AttnArgs& a, const AttnParts& p) {
  const int lane = threadIdx.x & 63, n = a.n_seq;   // at most 64
  AttnWavePlan w;
  const int raw0 = a.q_start[min(lane, n)], raw1 = a.q_start[min(lane + 1, n)], have = a.kv_len[min(lane, n - 1)];
  const int64_t most = (int64_t)a.pages_ld << a.c.page_shift;
  w.start = wave_scan_max(min(max(raw0, 0), a.M));
  w.end = max(w.start, min(max(raw1, 0), a.M));
  w.own = max(0, (int)min((int64_t)have, most));
  if (blockIdx.x == 0 && lane < n && (raw0 != w.start || raw1 != w.end || have != w.own)) set_flag(a.flags, kFlagLength);
  int rows = (w.end - w.start) * a.group;
  if (p.set == ATTN_PREFIX) {
    w.start = __shfl(w.start, 0);
    w.end = __shfl(w.end, n - 1);
    w.own = 0;
    rows = lane == 0 ? (w.end - w.start) * a.group : 0;
  }
  if (lane >= n) rows = 0;
  w.tiles = (rows + p.rows - 1) / p.rows;
  w.units = attn_units(p.set == ATTN_OWN ? 0 : a.prefix_len) + attn_units(w.own);
  int64_t work = (int64_t)w.tiles * w.units;
  int tiles = w.tiles;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    work += __shfl_xor(work, off);
    tiles += __shfl_xor(tiles, off);
  }
  const int per = attn_per(a, p, work, tiles);
  w.split = w.tiles ? max(1, (w.units + per - 1) / per) : 0;
  const int parts = w.tiles * w.split;
  int up = parts;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(up, off);
    if (lane >= off) up += o;
  }
  w.first = up - parts;
  w.total = __shfl(up, 63);
  if (blockIdx.x == 0 && threadIdx.x < (p.set == ATTN_PREFIX ? 1 : n)) {
    p.plan[2 + 2 * lane] = w.first;
    p.plan[3 + 2 * lane] = w.split;
  }
  return w;
}

__device__ __forceinline__ AttnPlace attn_wave_place(const AttnArgs& a, const AttnParts& p, const AttnWavePlan& w, int it) {
  const int lane = threadIdx.x & 63, entries = p.set == ATTN_PREFIX ? 1 : a.n_seq;
  AttnPlace r;
  r.e = __popcll(__ballot(lane < entries && w.first <= it)) - 1;
  const int start = __builtin_amdgcn_readlane(w.start, r.e), end = __builtin_amdgcn_readlane(w.end, r.e);
  r.first = __builtin_amdgcn_readlane(w.first, r.e);
  r.split = __builtin_amdgcn_readlane(w.split, r.e);
  r.x.row0 = start;
  r.x.rows = (end - start) * a.group;
  r.x.own = __builtin_amdgcn_readlane(w.own, r.e);
  r.x.pre = p.set == ATTN_OWN ? 0 : a.prefix_len;
  r.x.causal = r.x.own - (end - start);
  r.x.tiles = __builtin_amdgcn_readlane(w.tiles, r.e);
  r.x.units = __builtin_amdgcn_readlane(w.units, r.e);
  return r;
}

// The entry that a part of a key head belongs to: the last whose first part is
// at most `it` (entries without parts come to the one after them).
__device__ __forceinline__ int attn_find(const AttnPlan& s, int entries, int it) {
  const int lane = threadIdx.x & 63;
  int count = 0;
  for (int b = 0; b < entries; b += 64)
    count += __popcll(__ballot(b + lane < entries && s.first[b + lane] <= it));
  return count - 1;
}

__device__ __forceinline__ AttnPlace attn_place(const AttnArgs& a, const AttnParts& p, const AttnPlan& s, int it) {
  AttnPlace r;
  r.e = attn_find(s, p.set == ATTN_PREFIX ? 1 : a.n_seq, it);
  r.first = s.first[r.e];
  r.x = attn_entry(a, s.start, p.set, p.rows, r.e);
  r.split = max(1, (r.x.units + s.per - 1) / s.per);
  return r;
}

// Where a page's keys and values of one head begin, in elements; false for a
// page outside the cache (page 0 is given then).
__device__ __forceinline__ bool attn_page(const KvCache& c, uint32_t* flags, int page, int head, size_t& at) {
  const bool ok = (uint32_t)page < (uint32_t)c.n_pages;
  if (!ok) set_flag(flags, kFlagIndex);
  at = kv_page(c, ok ? page : 0, head);
  return ok;
}

__device__ __forceinline__ bf16x8 bf16x8_of(const float (&f)[8]) {
  bf16x8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = (__bf16)f[i];
  return r;
}

// Eight codes as bf16 (exact).
__device__ __forceinline__ bf16x8 bf16x8_of_codes(u32x2 w) {
  bf16x8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = (__bf16)(float)(int)(int8_t)(w[i >> 2] >> (8 * (i & 3)));
  return r;
}

// Which of the eight tokens behind `keep` count: the others' values become 0.
__device__ __forceinline__ bf16x8 keep_first(bf16x8 v, int keep) {
  u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t mask = (keep > 2 * i ? 0xFFFFu : 0u) | (keep > 2 * i + 1 ? 0xFFFF0000u : 0u);
    w[i] &= mask;
  }
  return __builtin_bit_cast(bf16x8, w);
}

// Infinities and NaNs become 0; returns whether there was one.
__device__ __forceinline__ bool drop_nonfinite(bf16x8& v) {
  u32x4 w = __builtin_bit_cast(u32x4, v);
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool lo = (w[i] & 0x7F80u) == 0x7F80u, hi = (w[i] & 0x7F800000u) == 0x7F800000u;
    any |= lo || hi;
    w[i] &= (lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u);
  }
  v = __builtin_bit_cast(bf16x8, w);
  return any;
}

}  // namespace q4nx
