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
// Two launches.  k_logprob_part: one wave takes a part of a row (64 * 4 * NQ
// logits) into registers, forms the part's (m, rest, sum e d) and its top k.
// k_logprob_join: one wave a row joins the parts: of two parts with
// m1 >= m2, f = exp(m2 - m1),
//   rest = rest1 + (1 + rest2) f,   t = t1 + f (t2 + (1 + rest2)(m2 - m1)).
//
// Top k of a part: T, the k-th largest of the 64 lanes' own maxima, is at most
// the k-th largest value, so the top k are among the values above T and, if
// fewer than k are, the first of those equal to T.  These few (about 1.3 k of
// random logits) are gathered by ballots and ordered by counting, for each,
// how many have a larger key.  The key is topk.h's: larger value, then lower
// index.  Should more values lie above T than the gathering space holds, T is
// raised by bisection over the order of fp32 first.
#include <algorithm>

#include "logprobs_args.h"
#include "topk.h"

namespace q4nx {

namespace {

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));   // rows start at any 4 bytes

constexpr float kLog2e = 1.44269504088896341f;
constexpr int kGather = 192;   // values above T that a part can gather

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  return v;
}
__device__ __forceinline__ float wave_min(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v = fminf(v, __shfl_xor(v, off));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
  return v;
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

// The k-th largest of the 64 lanes' values (k <= 64): the least value that
// fewer than k lanes exceed.
__device__ __forceinline__ float kth_of_lanes(float v, int k) {
  int above = 0;
#pragma unroll
  for (int j = 0; j < 64; ++j) {
    const float o = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), j));
    above += o > v ? 1 : 0;
  }
  return wave_min(above < k ? v : __builtin_inff());
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

}  // namespace

template <int NQ>
__global__ __launch_bounds__(256) void k_logprob_part(LogprobArgs a) {
  __shared__ uint64_t gath[4][kGather + kLogprobMaxK];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * 4 + wave;
  if (unit >= (int64_t)a.M * a.parts) return;   // whole waves; no barrier below
  const int m_row = (int)(unit / a.parts), part = (int)(unit - (int64_t)m_row * a.parts);
  const float* row = a.y + (size_t)m_row * a.ldy;
  const int i0 = part * (256 * NQ) + 4 * lane;   // index of v[q][c]: i0 + 256 q + c
  f32x4 v[NQ];
  if ((part + 1) * (256 * NQ) <= a.n) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) v[q] = *reinterpret_cast<const f32x4u*>(row + i0 + 256 * q);
  } else {
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int c = 0; c < 4; ++c) v[q][c] = i0 + 256 * q + c < a.n ? row[i0 + 256 * q + c] : neg_inf();
  }
  // NaNs are passed over: a maximum takes the other operand, comparisons are
  // false, and the clamp of d below turns them into nothing.
  float qm[NQ], lm = neg_inf();
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    qm[q] = fmaxf(fmaxf(v[q][0], v[q][1]), fmaxf(v[q][2], v[q][3]));
    lm = fmaxf(lm, qm[q]);
  }
  const float m = wave_max(lm);
  uint64_t* keys = a.keys + (size_t)unit * a.k;
  if (m == neg_inf()) {   // nothing left in this part
    if (lane == 0) a.stats[unit] = f32x4{m, 0.f, 0.f, 0.f};
    if (lane < a.k) keys[lane] = 0;
    return;
  }

  if (a.k > 0) {
    uint64_t* g = gath[wave];
    float T = kth_of_lanes(lm, a.k);
    int n_above;
    for (;;) {
      n_above = 0;
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        if (__ballot(qm[q] > T) == 0) continue;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint64_t b = __ballot(v[q][c] > T);
          const int at = n_above + lanes_below(b, lane);
          if (v[q][c] > T && at < kGather) g[at] = topk_key(v[q][c], i0 + 256 * q + c);
          n_above += __popcll(b);
        }
      }
      if (n_above <= kGather) break;
      // raise T: more than kGather values above lo, fewer than k above hi
      uint32_t lo = ord_of(T), hi = ord_of(m);
      while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const int c = count_above(v, of_ord(mid));
        if (c > kGather) lo = mid;
        else {
          hi = mid;
          if (c >= a.k) break;
        }
      }
      T = of_ord(hi);
    }
    // ties at T, the lowest indexes first
    int n_all = n_above;
    if (n_above < a.k && T > neg_inf()) {
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        if (n_all >= a.k) continue;
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
            if (n_all + before < a.k) g[n_all + before] = topk_key(v[q][c], i0 + 256 * q + c);
            ++before;
          }
        n_all = min(n_all + all, a.k);
      }
    }
    // The wave's own LDS writes and reads run in order; the fence keeps the
    // compiler from moving them.
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    for (int e0 = 0; e0 < n_all; e0 += 64) {
      const uint64_t mine = e0 + lane < n_all ? g[e0 + lane] : 0;
      int above = 0;
      for (int j = 0; j < n_all; ++j) above += g[j] > mine ? 1 : 0;
      if (mine && above < a.k) keys[above] = mine;
    }
    if (lane >= n_all && lane < a.k) keys[lane] = 0;
  }

  float rest = 0.f, t = 0.f;
  int n_max = 0;   // values equal to m: all but one of them count 1 in rest, and 0 in t
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const bool has_max = __ballot(qm[q] == m) != 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      // exp(-200) is 0 in fp32: the clamp changes no sum and keeps -inf and NaN out of e * d
      const float d = fmaxf(v[q][c] - m, -200.f);
      float e = __builtin_amdgcn_exp2f(d * kLog2e);
      if (has_max) {
        n_max += __popcll(__ballot(v[q][c] == m));
        e = v[q][c] == m ? 0.f : e;
      }
      rest += e;
      t = fmaf(e, d, t);
    }
  }
  rest = wave_sum(rest) + (float)(n_max - 1);
  t = wave_sum(t);
  if (lane == 0) a.stats[unit] = f32x4{m, rest, t, 0.f};
}

// Joins the parts of a row, one wave a row.  The top k of the row: lane l owns
// the lists of parts l, l + 64, ...; T, the k-th largest of the lanes' best
// keys, is at most the row's k-th key, and at most k lanes reach it, so at most
// k * k keys of each of their lists have to be gathered (kLogprobLists lists a
// lane at most: the host sizes the LDS for it) and ordered by counting.
__global__ __launch_bounds__(64) void k_logprob_join(LogprobArgs a) {
  extern __shared__ uint64_t g[];
  const int m_row = blockIdx.x, lane = threadIdx.x;
  const float* row = a.y + (size_t)m_row * a.ldy;
  const size_t u0 = (size_t)m_row * a.parts;
  float m = neg_inf(), rest = 0.f, t = 0.f;
  auto join = [&](float m2, float rest2, float t2) {
    if (m2 == neg_inf()) return;
    if (m == neg_inf()) { m = m2; rest = rest2; t = t2; return; }
    const bool up = m2 > m;
    const float d = fmaxf(up ? m - m2 : m2 - m, -200.f);   // of equal maxima (also +inf) 0
    const float dd = m == m2 ? 0.f : d;
    const float f = __builtin_amdgcn_exp2f(dd * kLog2e);
    const float rl = up ? rest : rest2, tl = up ? t : t2;      // the lower part
    const float rh = up ? rest2 : rest, th = up ? t2 : t;
    rest = rh + (1.f + rl) * f;
    t = th + f * (tl + (1.f + rl) * dd);
    m = up ? m2 : m;
  };
  uint64_t best = 0;
  for (int p = lane; p < a.parts; p += 64) {
    const f32x4 s = a.stats[u0 + p];
    join(s[0], s[1], s[2]);
    if (a.k > 0) {
      const uint64_t h = a.keys[(u0 + p) * a.k];
      best = h > best ? h : best;
    }
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    // both lanes of a pair join the lower lane's side first, so they end with the same bits
    const float om = __shfl_xor(m, off), orr = __shfl_xor(rest, off), ot = __shfl_xor(t, off);
    if (lane & off) {
      const float m2 = m, r2 = rest, t2 = t;
      m = om; rest = orr; t = ot;
      join(m2, r2, t2);
    } else {
      join(om, orr, ot);
    }
  }
  const bool left = m != neg_inf();
  const float lz = log1pf(rest);
  auto logp_of = [&](float v) { return (v == m ? 0.f : v - m) - lz; };
  for (int c = lane; c < a.n_tok; c += 64) {
    const int tok = a.tokens[(size_t)m_row * a.n_tok + c];
    float lp = __builtin_nanf("");
    if (left && tok >= 0 && tok < a.n) {
      const float v = row[tok];
      lp = v == v ? logp_of(v) : neg_inf();
    }
    a.logp[(size_t)m_row * a.n_tok + c] = lp;
  }
  if (a.entropy && lane == 0) a.entropy[m_row] = left ? lz - t / (1.f + rest) : __builtin_nanf("");
  if (a.k == 0) return;

  int above = 0;
#pragma unroll 16
  for (int j = 0; j < 64; ++j) {
    const uint64_t o = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(best >> 32), j) << 32) |
                       (uint32_t)__builtin_amdgcn_readlane((uint32_t)best, j);
    above += o > best ? 1 : 0;
  }
  uint64_t T = above < a.k ? best : ~0ull;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint64_t o = __shfl_xor(T, off);
    T = o < T ? o : T;
  }
  int n_all = 0;
  for (int p0 = 0; p0 < a.parts; p0 += 64) {
    const uint64_t* list = a.keys + (u0 + min(p0 + lane, a.parts - 1)) * a.k;
    const bool own = p0 + lane < a.parts && best >= T;
    for (int s = 0; s < a.k; ++s) {
      const uint64_t key = own ? list[s] : 0;
      const uint64_t b = __ballot(key != 0 && key >= T);
      if (b == 0) break;
      if (key != 0 && key >= T) g[n_all + lanes_below(b, lane)] = key;
      n_all += __popcll(b);
    }
  }
  __syncthreads();
  const size_t o0 = (size_t)m_row * a.k;
  for (int e0 = 0; e0 < n_all; e0 += 64) {
    const uint64_t mine = e0 + lane < n_all ? g[e0 + lane] : 0;
    int larger = 0;
    for (int j = 0; j < n_all; ++j) larger += g[j] > mine ? 1 : 0;
    if (mine && larger < a.k) {
      a.top_ids[o0 + larger] = (int32_t)~(uint32_t)mine;
      if (a.top_logp) a.top_logp[o0 + larger] = logp_of(of_ord((uint32_t)(mine >> 32)));
    }
  }
  if (lane >= n_all && lane < a.k) {
    a.top_ids[o0 + lane] = -1;
    if (a.top_logp) a.top_logp[o0 + lane] = __builtin_nanf("");
  }
}

hipError_t launch_token_logprobs(const LogprobArgs& a, hipStream_t s) {
  const int64_t units = (int64_t)a.M * a.parts;
  const dim3 grid((unsigned)((units + 3) / 4));
  if (a.part_n == 1024)
    hipLaunchKernelGGL((k_logprob_part<4>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_logprob_part<16>), grid, dim3(256), 0, s, a);
  const size_t lds = (size_t)std::min(a.k, 64) * ((a.parts + 63) / 64) * a.k * sizeof(uint64_t);
  hipLaunchKernelGGL(k_logprob_join, dim3(a.M), dim3(64), lds, s, a);
  return hipGetLastError();
}

}  // namespace q4nx
