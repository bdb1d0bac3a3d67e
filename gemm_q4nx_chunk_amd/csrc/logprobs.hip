// Log probabilities over the head's logits: of given tokens, with the entropy
// and the k likeliest alternatives of each row.
//
// With m = max y and one of the maxima set apart,
//   rest = sum over the others of exp(y_i - m),   log Z = m + log1p(rest),
//   log p_i = (y_i - m) - log1p(rest),
//   H = -sum p log p = log1p(rest) - sum exp(d_i) d_i / (1 + rest),  d = y - m.
// Setting one maximum apart keeps the digits of a likely token: its log
// probability is -log1p(rest), where log(1 + rest) of the whole sum would lose
// what lies below 2^-24.
//
// Two launches.  k_logprob_part: a wave streams a part of a row through
// registers in chunks of 256 NQ logits, and keeps (m, rest, t = sum e d) against
// the wave's maximum so far, and the top k so far.  k_logprob_join: one wave a
// row adds the parts, each by f = exp(m_part - m): rest += (1 + rest_p) f
// (rest_p alone for one part that has m), t += f (t_p + (1 + rest_p)(m_part - m)).
//
// Top k of a wave: a threshold T that at least k values seen reach, and a
// gathering space in LDS that holds the index of every value seen above T and,
// of those equal to T, the first ones.  The first chunk's T comes from the 64
// lanes' own maxima: a value that k of them reach.  After that only the values
// above T are gathered (of random logits about as many in every chunk as in the
// first, for T stays until the space is full): each lane marks its hits in a
// word, a sum over the lanes below gives it its place.  A full space is cut down
// to its k largest, and T raised to the least of them.  At the end the gathered values
// are read again, as keys (topk.h's: larger value, then lower index), and
// ordered by counting, for each, how many are larger.  Should more values lie
// above T than the space holds, T is raised by bisection over the order of
// fp32 first.
//
// Many rows are bound by HBM with k <= 1: 1000 rows of 151936 logits, 608 MB, take
// 114 us (5.3 TB/s), 4096 rows 429 us (5.8); a large copy, which writes too,
// reaches 5.2, this library's longest weight streams 6.0 to 6.3.  Their top k
// costs more: 1000 rows 148 us with k = 20 and 170 with k = 32, 828 and 937 MB
// fetched instead of 616, for the gathered values are read again; 4096 rows 508
// with k = 20.  64 rows (39 MB, in the Infinity Cache) take 11.9 us a call with
// k = 0 and 17.7 with k = 20, the latency of one chunk a wave and of the join, and
// the top k; one row 9.4 us with k = 5, its two kernels 5.0 and 4.8.
#include <algorithm>

#include "logprobs_args.h"
#include "topk.h"

namespace q4nx {

namespace {

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));   // rows start at any 4 bytes

constexpr float kLog2e = 1.44269504088896341f;
constexpr int kGather = 256;   // keys above T that a wave can gather
constexpr int kRoom = kGather + kLogprobMaxK;   // with those equal to it

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// Reductions over the wave by DPP: within rows of 16 lanes, then across them;
// lane 63 ends with the result, which every lane gets as a scalar.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float old, float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(__float_as_uint(old), __float_as_uint(v), CTRL, ROWS, 0xF, false));
}
__device__ __forceinline__ float last_lane(float v) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp<0x111, 0xF>(v, v));   // row_shr 1, 2, 4, 8
  v = fmaxf(v, dpp<0x112, 0xF>(v, v));
  v = fmaxf(v, dpp<0x114, 0xF>(v, v));
  v = fmaxf(v, dpp<0x118, 0xF>(v, v));
  v = fmaxf(v, dpp<0x142, 0xA>(v, v));   // row_bcast 15 into rows 1 and 3
  v = fmaxf(v, dpp<0x143, 0xC>(v, v));   // row_bcast 31 into rows 2 and 3
  return last_lane(v);
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0x111, 0xF>(0.f, v);
  v += dpp<0x112, 0xF>(0.f, v);
  v += dpp<0x114, 0xF>(0.f, v);
  v += dpp<0x118, 0xF>(0.f, v);
  v += dpp<0x142, 0xA>(0.f, v);
  v += dpp<0x143, 0xC>(0.f, v);
  return last_lane(v);
}

__device__ __forceinline__ int lanes_below(uint64_t mask, int lane) {
  return __popcll(mask & ((1ull << lane) - 1ull));
}

// Order of fp32 as unsigned integers, without NaN: a < b iff ord(a) < ord(b),
// up to the two zeros, which callers compare as floats.
__device__ __forceinline__ uint32_t ord_of(float v) {
  const uint32_t b = __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float of_ord(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

__device__ __forceinline__ float wave_min(float v) { return -wave_max(-v); }

// Sum over the lanes below (row_shr and row_bcast as above), and over all.
__device__ __forceinline__ int sum_below(int v, int& all) {
  int s = v;
  s += __builtin_amdgcn_update_dpp(0, s, 0x111, 0xF, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x112, 0xF, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x114, 0xF, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x118, 0xF, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x142, 0xA, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x143, 0xC, 0xF, false);
  all = __builtin_amdgcn_readlane(s, 63);
  return s - v;
}

// How many may reach a bound that at least k have to reach.
__host__ __device__ __forceinline__ int reach(int k) { return k + k / 4 + 4; }

// A bound that at least k lanes' values reach (k <= 64) and, unless values are
// alike, at most reach(k): bisection over unsigned order between lo, which all
// reach, and top, the largest.
__device__ __forceinline__ uint32_t reached_by_k(uint32_t v, uint32_t lo, uint32_t top, int k) {
  uint32_t hi = top;
  if (__popcll(__ballot(v >= top)) >= k) return top;
  while (hi - lo > 1) {
    const uint32_t mid = lo + (hi - lo) / 2;
    const int c = __popcll(__ballot(v >= mid));
    if (c < k) hi = mid;
    else {
      lo = mid;
      if (c <= reach(k)) break;
    }
  }
  return lo;
}

// How many of the wave's values are above T.
template <int NQ>
__device__ __forceinline__ int count_above(const f32x4 (&v)[NQ], float T) {
  int c = 0;
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) c += __popcll(__ballot(v[q][i] > T));
  return c;
}

// Orders a wave's LDS writes before its reads that follow, and the other way
// round: a wave's LDS operations run in order, the compiler must keep them so.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// How many of the n keys at g (padded with zeros to a multiple of U) are larger than `key`.
template <int U>
__device__ __forceinline__ int larger_keys(const uint64_t* g, int n, uint64_t key) {
  int c = 0;
  for (int j = 0; j < n; j += U) {
#pragma unroll
    for (int i = 0; i < U; ++i) c += g[j + i] > key ? 1 : 0;
  }
  return c;
}

// A wave's gathering space: the indexes gathered, their keys when they are
// ordered, and the best of them when the space is cut down.
struct Gather {
  int32_t index[kRoom];
  uint64_t key[kRoom + 8];
  uint64_t best[kLogprobMaxK];
};

// The keys of the largest min(k, n) of the n values gathered, in decreasing
// order, to out (not in g.key).  The values are read again: all at once, and
// only here.  One piece of 64 at a time, so that few registers are held beside
// a chunk's.
template <int U>
__device__ __forceinline__ void select_k(Gather& g, const float* row, int n, int k, int lane, uint64_t* out) {
  wave_lds_fence();
#pragma unroll 1
  for (int e = lane; e < n; e += 64) g.key[e] = topk_key(row[g.index[e]], g.index[e]);
  if (lane < U) g.key[n + lane] = 0;
  wave_lds_fence();
#pragma unroll 1
  for (int e = lane; e - lane < n; e += 64) {
    const uint64_t mine = e < n ? g.key[e] : 0;
    const int at = larger_keys<U>(g.key, n, mine);
    if (mine != 0 && at < k) out[at] = mine;
  }
}

// The running state of a wave.
struct TopState {
  int n;     // gathered values
  float T;   // at least k values seen reach it; -inf before there are k
};

// Takes a chunk's values (value q, c of lane l has index i0 + 256 q + c, i0
// with 4 l in it) into the gathered ones.  lm: the lane's maximum, cm: the
// chunk's.
template <int NQ>
__device__ __forceinline__ void take_chunk(const f32x4 (&v)[NQ], float lm, float cm, int i0, const float* row, int k,
                                           int lane, Gather& g, TopState& st) {
  const bool fresh = st.T == neg_inf();   // fewer than k so far: this chunk's own bound
  float T = st.T;
  if (fresh) {
    if (k == 1) T = cm;
    else if (__popcll(__ballot(lm > neg_inf())) > reach(k))   // else T stays below them all
      T = of_ord(reached_by_k(ord_of(lm), std::max(ord_of(wave_min(lm)), ord_of(neg_inf())), ord_of(cm), k));
  }
  uint32_t hits;   // bit 4 NQ - 1 - (4 q + c): value q, c is above T
  int at, above;
  for (;;) {
    hits = 0;
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int c = 0; c < 4; ++c) hits = hits + hits + (v[q][c] > T ? 1u : 0u);
    at = st.n + sum_below(__popc(hits), above);
    if (st.n + above <= kGather) break;
    if (st.n > k) {   // make room
      select_k<4>(g, row, st.n, k, lane, g.best);
      wave_lds_fence();
      if (lane < k) g.index[lane] = (int32_t)~(uint32_t)g.best[lane];
      st.n = k;
      T = fmaxf(T, of_ord((uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(g.best[k - 1] >> 32))));
      continue;
    }
    // more above T than there is room for: raise it
    uint32_t lo = ord_of(T), hi = ord_of(cm);
    while (hi - lo > 1) {
      const uint32_t mid = lo + (hi - lo) / 2;
      const int c = count_above(v, of_ord(mid));
      if (c > kGather - k) lo = mid;
      else {
        hi = mid;
        if (c >= k) break;
      }
    }
    T = of_ord(hi);
  }
  while (__ballot(hits != 0)) {   // a value of each lane that has one, the first first
    if (hits != 0) {
      const int b = 31 - __clz(hits), i = 4 * NQ - 1 - b;
      g.index[at++] = i0 + 64 * (i & ~3) + (i & 3);
      hits ^= 1u << b;
    }
  }
  st.n += above;
  // fewer than k of this chunk above its own bound: those equal to it, the lowest indexes first
  if (T != st.T && T > neg_inf()) {
    int need = k - above;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      if (need <= 0) continue;
      uint64_t b[4];
      int before = 0, all = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        b[c] = __ballot(v[q][c] == T);
        before += lanes_below(b[c], lane);
        all += __popcll(b[c]);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (v[q][c] == T) {
          if (before < need) g.index[st.n + before] = i0 + 256 * q + c;
          ++before;
        }
      st.n += min(all, need);
      need -= all;
    }
  }
  st.T = T;
}

}  // namespace

// The chunk whose value q, c of lane l has index i0 + 256 q + c (4 l in i0), -inf
// from `end` on.  A group that crosses the end is read from the last four
// logits before it (in a row of fewer than four, the first again and again)
// and moved down.
template <int NQ>
__device__ __forceinline__ void load_chunk(const float* row, int end, int i0, bool whole, f32x4 (&v)[NQ]) {
  if (whole) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) v[q] = *reinterpret_cast<const f32x4u*>(row + i0 + 256 * q);
    return;
  }
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int i = i0 + 256 * q, from = min(i, end - 4);
    const int by = i - from;   // 0: as it lies; 4 and up: nothing left
    if (end >= 4) {
      v[q] = *reinterpret_cast<const f32x4u*>(row + from);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) v[q][c] = row[max(0, from + c)];
    }
    const float n = neg_inf();
    const f32x4 o = v[q];
    v[q][0] = by == 0 ? o[0] : by == 1 ? o[1] : by == 2 ? o[2] : by == 3 ? o[3] : n;
    v[q][1] = by == 0 ? o[1] : by == 1 ? o[2] : by == 2 ? o[3] : n;
    v[q][2] = by == 0 ? o[2] : by == 1 ? o[3] : n;
    v[q][3] = by == 0 ? o[3] : n;
  }
}

template <int NQ>
__global__ __launch_bounds__(256) void k_logprob_part(LogprobArgs a) {
  constexpr int kChunk = 256 * NQ;
  __shared__ Gather gath[4];
  // the wave's number as a scalar: rows, bounds and branches then are scalar too
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t unit = blockIdx.x * 4 + wave;
  if (unit >= (uint32_t)a.M * a.parts) return;   // no barrier below
  const int m_row = unit / (uint32_t)a.parts, part = unit - (uint32_t)m_row * a.parts;
  const float* row = a.y + (size_t)m_row * a.ldy;
  const int begin = part * a.part_n, end = min(a.n, begin + a.part_n);
  Gather& g = gath[wave];
  TopState st = {0, neg_inf()};
  float m = neg_inf(), rest = 0.f, t = 0.f;   // rest, t: this lane's share, but for the one maximum set apart
  for (int c0 = begin; c0 < end; c0 += kChunk) {
    f32x4 v[NQ];
    load_chunk<NQ>(row, end, c0 + 4 * lane, c0 + kChunk <= end, v);
    // NaNs are passed over: a maximum takes the other operand, comparisons are
    // false, and the clamp of d below turns them into nothing.
    float lm = neg_inf();
#pragma unroll
    for (int q = 0; q < NQ; ++q) lm = fmaxf(lm, fmaxf(fmaxf(v[q][0], v[q][1]), fmaxf(v[q][2], v[q][3])));
    const float cm = wave_max(lm);
    if (cm == neg_inf()) continue;   // nothing left in this chunk
    if (a.k > 0 && cm > st.T) take_chunk<NQ>(v, lm, cm, c0 + 4 * lane, row, a.k, lane, g, st);
    // exp(-200) is 0 in fp32: the clamp changes no sum and keeps -inf and NaN out of e * d
    float r_c = 0.f, t_c = 0.f;   // this chunk's rest and t: a sum of its own, so that no value passes more
                                  // additions than a chunk has values in a lane and a part has chunks
    if (cm >= m) {
      if (cm > m && m != neg_inf()) {   // the old maximum joins the rest
        const float d = fmaxf(m - cm, -200.f), f = __builtin_amdgcn_exp2f(d * kLog2e);
        rest += lane == 0 ? 1.f : 0.f;
        t = f * fmaf(rest, d, t);
        rest *= f;
      }
      int same = cm > m ? -1 : 0;   // values equal to the maximum, but for the one set apart
      m = cm;
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bool is = v[q][c] == m;
          same += __popcll(__ballot(is));
          const float d = fmaxf(v[q][c] - m, -200.f);
          const float e = is ? 0.f : __builtin_amdgcn_exp2f(d * kLog2e);
          r_c += e;
          t_c = fmaf(e, d, t_c);
          if (c == 3) __builtin_amdgcn_sched_barrier(0);
        }
      r_c += lane == 0 ? (float)same : 0.f;
    } else {
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float d = fmaxf(v[q][c] - m, -200.f);
          const float e = __builtin_amdgcn_exp2f(d * kLog2e);
          r_c += e;
          t_c = fmaf(e, d, t_c);
          if (c == 3) __builtin_amdgcn_sched_barrier(0);
        }
    }
    rest += r_c;
    t += t_c;
  }
  rest = wave_sum(rest);
  t = wave_sum(t);
  if (lane == 0) a.stats[unit] = f32x4{m, rest, t, 0.f};
  if (a.k > 0) {
    uint64_t* keys = a.keys + (size_t)unit * a.k;
    select_k<8>(g, row, st.n, a.k, lane, keys);
    if (lane >= st.n && lane < a.k) keys[lane] = 0;
  }
}

// Joins the parts of a row, one wave a row.  Lane l owns parts l, l + 64, ...
// (four at most).  The row's top k: T, a key that at least k known keys reach,
// is at most the row's k-th, so the keys of at least T are gathered from the
// parts' lists and ordered by counting.  The known keys, and what at most is
// gathered (the host sizes the LDS for it), when reach(k) of them reach T:
//   kLanes (64 parts and more): the lanes' best; the lanes' whole lists.  (A
//     list is in decreasing order: it ends at its first key below T.)
//   kAll (up to 512 keys): every one, eight a lane; those.
//   kFours: the first four of each list; those, and what follows the fours.
enum JoinKeys { kLanes, kAll, kFours };
constexpr int kFirst = 4;    // keys of a list loaded ahead
constexpr int kAllKeys = 8;  // keys a lane, where all are loaded
inline JoinKeys join_keys(int parts, int k) {
  return parts >= 64 ? kLanes : parts * k <= 64 * kAllKeys ? kAll : kFours;
}
inline int join_room(int parts, int k) {
  switch (join_keys(parts, k)) {
    case kAll: return std::min(parts * k, reach(k));
    case kLanes: return std::min(64, reach(k)) * ((parts + 63) / 64) * k;
    default: return reach(k) + reach(k) / kFirst * std::max(0, k - kFirst);
  }
}

template <JoinKeys KEYS>
__global__ __launch_bounds__(64) void k_logprob_join(LogprobArgs a) {
  constexpr bool all_at_once = KEYS == kAll, by_lane = KEYS == kLanes;
  extern __shared__ uint64_t g[];   // join_room keys and 4
  const int m_row = blockIdx.x, lane = threadIdx.x, k = a.k;
  const float* row = a.y + (size_t)m_row * a.ldy;
  const size_t u0 = (size_t)m_row * a.parts;
  // everything whose place is known, in flight at once
  const int tok = lane < a.n_tok ? a.tokens[(size_t)m_row * a.n_tok + lane] : -1;
  f32x4 s[4];
  uint64_t key[4][kFirst];   // all at once: key i of lane l at 64 i + l of the parts' keys; else key j of part l + 64 i
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int p = lane + 64 * i;
    s[i] = f32x4{neg_inf(), 0.f, 0.f, 0.f};
    if (p < a.parts) s[i] = a.stats[u0 + p];
#pragma unroll
    for (int j = 0; j < kFirst; ++j) {
      key[i][j] = 0;
      if constexpr (all_at_once) {
        const int e = 64 * (kFirst * i + j) + lane;
        if (i < kAllKeys / kFirst && e < a.parts * k) key[i][j] = a.keys[u0 * k + e];
      } else {
        if (p < a.parts && j < k) key[i][j] = a.keys[(u0 + p) * k + j];
      }
    }
  }
  const bool inside = tok >= 0 && tok < a.n;
  const float yt = inside ? row[tok] : 0.f;

  const float m = wave_max(fmaxf(fmaxf(s[0][0], s[1][0]), fmaxf(s[2][0], s[3][0])));
  const bool left = m != neg_inf();
  float rest = 0.f, t = 0.f;
  bool apart = false;   // one part with the row's maximum has been met (in part order within a lane, lanes in order)
  {
    bool has = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) has |= s[i][0] == m;
    const uint64_t b = __ballot(has);
    apart = b == 0 || lane != __builtin_ctzll(b);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (s[i][0] == neg_inf()) continue;
    const bool is = s[i][0] == m;
    const float d = is ? 0.f : fmaxf(s[i][0] - m, -200.f);
    const float f = __builtin_amdgcn_exp2f(d * kLog2e);
    const float one = is && !apart ? 0.f : 1.f;
    if (is) apart = true;
    rest += (one + s[i][1]) * f;
    t += f * fmaf(1.f + s[i][1], d, s[i][2]);
  }
  rest = wave_sum(rest);
  t = wave_sum(t);
  const float lz = log1pf(rest);
  auto logp_of = [&](float v) { return (v == m ? 0.f : v - m) - lz; };
  if (lane < a.n_tok) {
    float lp = __builtin_nanf("");
    if (left && inside) lp = yt == yt ? logp_of(yt) : neg_inf();
    a.logp[(size_t)m_row * a.n_tok + lane] = lp;
  }
  if (a.entropy && lane == 0) a.entropy[m_row] = left ? lz - t / (1.f + rest) : __builtin_nanf("");
  if (k == 0) return;

  const int lists = (a.parts + 63) / 64;
  uint64_t best = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < kFirst; ++j)
      if (j == 0 || all_at_once) best = key[i][j] > best ? key[i][j] : best;
  const uint64_t top = wave_max_u64(best);
  auto reached = [&](uint64_t at) -> int {
    if constexpr (by_lane) return __popcll(__ballot(best >= at));
    int c = 0;
#pragma unroll
    for (int i = 0; i < (all_at_once ? kAllKeys / kFirst : 1); ++i)
#pragma unroll
      for (int j = 0; j < kFirst; ++j) c += __popcll(__ballot(key[i][j] >= at));
    return c;
  };
  uint64_t T = k == 1 ? top : 1;   // 1: every key
  if (k > 1 && reached(1) > reach(k)) {
    for (uint64_t hi = top + 1; hi > T + 1;) {   // fewer than k reach hi
      const uint64_t mid = T + (hi - T) / 2;
      const int c = reached(mid);
      if (c < k) hi = mid;
      else {
        T = mid;
        if (c <= reach(k)) break;
      }
    }
  }
  int n = 0;
  auto add = [&](uint64_t v) {
    const bool in = v >= T && v != 0;
    const uint64_t b = __ballot(in);
    const int at = n + lanes_below(b, lane);
    if (in) g[at] = v;
    n += __popcll(b);
    return b;
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= (all_at_once ? kAllKeys / kFirst : lists)) continue;
    uint64_t b = 0;
#pragma unroll
    for (int j = 0; j < kFirst; ++j) b = add(key[i][j]);
    const uint64_t* list = a.keys + (u0 + min(lane + 64 * i, a.parts - 1)) * k;
    bool mine = key[i][kFirst - 1] != 0 && key[i][kFirst - 1] >= T;
    for (int j0 = kFirst; !all_at_once && b != 0 && j0 < k; j0 += kFirst) {
      uint64_t v[kFirst];
#pragma unroll
      for (int j = 0; j < kFirst; ++j) v[j] = mine && j0 + j < k ? list[j0 + j] : 0;
#pragma unroll
      for (int j = 0; j < kFirst; ++j) b = add(v[j]);
      mine = v[kFirst - 1] != 0 && v[kFirst - 1] >= T;
    }
  }
  if (lane < 4) g[n + lane] = 0;
  wave_lds_fence();
  const size_t o0 = (size_t)m_row * k;
  for (int e0 = 0; e0 < n; e0 += 64) {
    const uint64_t mine = e0 + lane < n ? g[e0 + lane] : 0;
    const int at = larger_keys<4>(g, n, mine);
    if (mine && at < k) {
      a.top_ids[o0 + at] = (int32_t)~(uint32_t)mine;
      if (a.top_logp) a.top_logp[o0 + at] = logp_of(of_ord((uint32_t)(mine >> 32)));
    }
  }
  if (lane >= n && lane < k) {
    a.top_ids[o0 + lane] = -1;
    if (a.top_logp) a.top_logp[o0 + lane] = __builtin_nanf("");
  }
}

hipError_t launch_token_logprobs(const LogprobArgs& a, hipStream_t s) {
  const int64_t units = (int64_t)a.M * a.parts;
  const dim3 grid((unsigned)((units + 3) / 4));
  if (a.part_n < kLogprobChunk)
    hipLaunchKernelGGL((k_logprob_part<4>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_logprob_part<kLogprobChunk / 256>), grid, dim3(256), 0, s, a);
  const size_t lds = (join_room(a.parts, a.k) + 4) * sizeof(uint64_t);
  switch (join_keys(a.parts, a.k)) {
    case kAll: hipLaunchKernelGGL((k_logprob_join<kAll>), dim3(a.M), dim3(64), lds, s, a); break;
    case kLanes: hipLaunchKernelGGL((k_logprob_join<kLanes>), dim3(a.M), dim3(64), lds, s, a); break;
    case kFours: hipLaunchKernelGGL((k_logprob_join<kFours>), dim3(a.M), dim3(64), lds, s, a); break;
  }
  return hipGetLastError();
}

}  // namespace q4nx
