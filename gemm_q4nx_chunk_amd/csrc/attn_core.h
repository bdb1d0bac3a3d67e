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
  int32_t own[kAttnMaxSeq];         // tokens of each sequence, within its pages
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

__device__ __forceinline__ AttnEntry attn_entry(const AttnArgs& a, const int32_t* start, const int32_t* own, int set, int tile_rows, int e) {
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
    x.own = own[e];
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

// Fills the plan; returns the parts of one key head.  All 256 threads call it; the set's first workgroup writes
// what the join needs.
__device__ inline int attn_plan_small(const AttnArgs& a, const AttnParts& p, AttnPlan& s, bool first);
__device__ inline int attn_plan(const AttnArgs& a, const AttnParts& p, AttnPlan& s, bool first) {
  if (a.n_seq <= 64) return attn_plan_small(a, p, s, first);
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
        bool bad = raw != up;
        if (e < n) {
          const int have = a.kv_len[e];
          s.own[e] = max(0, (int)min((int64_t)have, (int64_t)a.pages_ld << a.c.page_shift));
          bad |= have != s.own[e];
        }
        if (first && bad) set_flag(a.flags, kFlagLength);
      }
      carry = max(carry, total);
    }
  }
  __syncthreads();
  const int entries = p.set == ATTN_PREFIX ? 1 : n;
  int64_t work = 0, total;
  int tiles = 0, all_tiles;
  for (int e = tid; e < entries; e += 256) {
    const AttnEntry x = attn_entry(a, s.start, s.own, p.set, p.rows, e);
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
      const AttnEntry x = attn_entry(a, s.start, s.own, p.set, p.rows, e);
      split = x.tiles ? max(1, (x.units + per - 1) / per) : 0;
      parts = x.tiles * split;
    }
    int all;
    const int up = scan256<int, false>(parts, s.sums, all) + carry;
    if (e < entries) {
      s.first[e] = up - parts;
      if (first) {
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

__device__ __forceinline__ int wave_scan_max(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(v, off);
    if (lane >= off) v = max(v, o);
  }
  return v;
}

// A plan of up to 64 sequences is one wave's work, with one barrier (one token of 777: 6.9 us, 9 with the
// workgroup's scans).  Each wave forms it, the first writes it.
__device__ inline int attn_plan_small(const AttnArgs& a, const AttnParts& p, AttnPlan& s, bool first) {
  const int tid = threadIdx.x, lane = tid & 63, n = a.n_seq;   // at most 64
  const int raw0 = a.q_start[min(lane, n)], raw1 = a.q_start[min(lane + 1, n)], have = a.kv_len[min(lane, n - 1)];
  const int start = wave_scan_max(min(max(raw0, 0), a.M)), end = max(start, min(max(raw1, 0), a.M));
  const int own = max(0, (int)min((int64_t)have, (int64_t)a.pages_ld << a.c.page_shift));
  if (first && tid < n && (raw0 != start || raw1 != end || have != own)) set_flag(a.flags, kFlagLength);
  const int begin = __shfl(start, 0), last = __shfl(end, n - 1);
  const bool is_pre = p.set == ATTN_PREFIX;
  const int rows = is_pre ? (lane == 0 ? (last - begin) * a.group : 0) : lane < n ? (end - start) * a.group : 0;
  const int units = attn_units(p.set == ATTN_OWN ? 0 : a.prefix_len) + (is_pre ? 0 : attn_units(own));
  const int my_tiles = (rows + p.rows - 1) / p.rows;
  int64_t work = (int64_t)my_tiles * units;
  int tiles = my_tiles;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    work += __shfl_xor(work, off);
    tiles += __shfl_xor(tiles, off);
  }
  const int per = attn_per(a, p, work, tiles);
  const int split = my_tiles ? max(1, (units + per - 1) / per) : 0, parts = my_tiles * split;
  int up = parts;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(up, off);
    if (lane >= off) up += o;
  }
  if (tid < n) {
    s.start[lane] = start;
    s.first[lane] = up - parts;
    s.own[lane] = own;
    if (first && (!is_pre || lane == 0)) {
      p.plan[2 + 2 * lane] = up - parts;
      p.plan[3 + 2 * lane] = split;
    }
  }
  if (tid == 0) {
    s.start[n] = last;
    s.per = per;
  }
  const int total = __shfl(up, 63);
  if (tid == 0) s.first[is_pre ? 1 : n] = total;
  __syncthreads();
  return total;
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
  r.x = attn_entry(a, s.start, s.own, p.set, p.rows, r.e);
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

// The first `keep` of eight tokens' values; the others become 0.  (Here and below without truth values, of which
// there would be more than scalar registers.)
__device__ __forceinline__ bf16x8 keep_first(bf16x8 v, int keep) {
  u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] &= (uint32_t)((0xFFFFFFFFull << (16 * min(max(keep - 2 * i, 0), 2))) >> 32);
  return __builtin_bit_cast(bf16x8, w);
}

// Infinities and NaNs become 0; not 0 if there was one.
__device__ __forceinline__ uint32_t drop_nonfinite(bf16x8& v) {
  u32x4 w = __builtin_bit_cast(u32x4, v);
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t top = ((w[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;   // each half's highest bit
    any |= top;
    w[i] &= ~(top | (top - (top >> 15)));
  }
  v = __builtin_bit_cast(bf16x8, w);
  return any;
}

}  // namespace q4nx
