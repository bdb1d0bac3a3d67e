// Attention over the paged cache, and the join of its parts.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(z_j - max z),  z_j = scale log2(e) q.k_j
//
// Both products run transposed, S^T = K Q^T and O^T = V^T P^T, on matrix
// instructions of 16 x 16: a lane then holds scores of one row only (its
// column), so that the running maximum and the rescaling need no exchange but
// one over the four lanes of a column, and P^T is already in the order in which
// the second product takes it.  Which key stands in which line of S^T is free:
// lines are dealt so that a lane's eight scores belong to eight neighbouring
// tokens, which is what one 16-byte piece of the cache's values holds.  So K and
// V go from memory to the matrix cores as they lie, in whole lines.
#include <algorithm>
#include <type_traits>

#include "attn_core.h"

namespace q4nx {

namespace {

constexpr float kNegInf = -__builtin_huge_valf();

typedef __attribute__((address_space(3))) void lds_void;

// Eight elements of the cache, as they come.
template <bool I8>
struct Raw {
  u32x4 w;
  __device__ __forceinline__ void load(const void* p, size_t at) { w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + at); }
  __device__ __forceinline__ bf16x8 get() const { return __builtin_bit_cast(bf16x8, w); }
  // the first `n` of the eight, and, if `finite`, no infinity or NaN; whether there was one
  __device__ __forceinline__ uint32_t keep(int n, bool finite) {
    bf16x8 v = keep_first(get(), n);
    const uint32_t odd = finite ? drop_nonfinite(v) : 0u;
    w = __builtin_bit_cast(u32x4, v);
    return odd;
  }
};
template <>
struct Raw<true> {
  u32x2 w;
  __device__ __forceinline__ void load(const void* p, size_t at) { w = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(p) + at); }
  __device__ __forceinline__ bf16x8 get() const { return bf16x8_of_codes(w); }
  __device__ __forceinline__ uint32_t keep(int, bool) { return 0u; }
};

// x - y of an x that has been rounded: a product is not taken into a fused multiply-add.
__device__ __forceinline__ float rounded_less(float x, float y) {
#pragma clang fp contract(off)
  return x - y;
}

// Four dimensions of a row and head, from d.  A sum of 0 is that of a row that
// sees nothing (any other has its largest term, 1, or a NaN).
__device__ __forceinline__ void write_row(const AttnArgs& a, size_t row, int D, int d, f32x4 o, float m, float l) {
  const bool none = l == 0.f;
  const float inv = none ? 0.f : 1.f / l;
  uint32_t w[2];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    bf16x2 v;
    v[0] = (__bf16)(o[2 * n] * inv);
    v[1] = (__bf16)(o[2 * n + 1] * inv);
    w[n] = __builtin_bit_cast(uint32_t, v);
  }
  *reinterpret_cast<u32x2*>(a.out + row * D + d) = u32x2{w[0], w[1]};
  if (a.lse && d == 0) a.lse[row] = none ? kNegInf : m * 0.6931471805599453f + logf(l);
}

}  // namespace

// Few rows (16 or 32 a tile): a sequence's one row, or a window's, with the query
// heads of one key head.  The workgroup's four waves take 32 keys each of a unit
// of 128, with maxima, sums and outputs of their own that are joined at the end,
// so that a unit's K and V are read once, straight into registers.  The next
// keys are asked for as soon as the products have taken the last ones, the next
// values likewise: 16 KB a wave are always on the way.  Bound by memory, so that
// the softmax's numerators can enter in two bf16 parts, which hold 16 bits.
// (32 heads of 128: one token of 1000, 8192, 32768: 11.4, 16.0, 32.5 us a call, 4.1
// TB/s at the last; 64 tokens of 2000: 66 us, 5.0 TB/s; over 8 bits 42, where turning
// codes to bf16 holds it back.)
template <int D, bool I8, int RB>
__device__ __forceinline__ void attn_few(const AttnArgs& a, const AttnParts& p, int block, int blocks, AttnPlan& plan, uint8_t* lds) {
  constexpr int kRows = 16 * RB, NS = D / 32, NJ = D / 16, kLd = D + 4;
  __shared__ float s_m[4][kRows], s_l[4][kRows];
  float* const s_o = reinterpret_cast<float*>(lds);   // [4][16][kLd]
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, c = lane & 15, g = lane >> 4;
  const int KH = a.c.heads, ps = a.c.page_shift;
  const int total = attn_plan(a, p, plan, block == 0);
  for (int idx = block; idx < total * KH; idx += blocks) {
    const int head = idx % KH, it = idx / KH;
    const AttnPlace at = attn_place(a, p, plan, it);
    const AttnEntry& x = at.x;
    const int local = it - at.first, part = local % at.split, rt = local / at.split;
    // the lane's rows
    int r[RB], lim_own[RB];
    auto seen = [&](int row) { return min(max(x.causal + row / a.group + 1, 0), x.own); };
    bf16x8 qf[RB][NS];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      r[b] = min(rt * kRows + 16 * b + c, x.rows - 1);
      lim_own[b] = seen(r[b]);
      const uint16_t* qp = a.q + ((size_t)(x.row0 + r[b] / a.group) * a.q_heads + head * a.group + r[b] % a.group) * D + 8 * g;
#pragma unroll
      for (int s = 0; s < NS; ++s) qf[b][s] = *reinterpret_cast<const bf16x8*>(qp + 32 * s);
    }
    const int lim_first = seen(rt * kRows), lim_last = seen(min(rt * kRows + kRows, x.rows) - 1);
    const int pre_units = attn_units(x.pre), units = pre_units + attn_units(lim_last);
    const int per = (units + at.split - 1) / at.split, u0 = part * per, u1 = min(units, u0 + per);
    const int32_t* own_pages = p.set == ATTN_PREFIX ? nullptr : a.pages + (size_t)at.e * a.pages_ld;

    f32x4 acc[RB][NJ];
    float m_run[RB], l_run[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[b][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      m_run[b] = kNegInf;
      l_run[b] = 0.f;
    }

    // 32 keys: the 16 of each half may lie in pages of their own
    struct Keys {
      int key0, have;        // keys from `have` on are no row's
      bool pre, ok0, ok1;
      size_t at0, at1;       // first elements of the halves' pages, and the tokens there
      int t0, t1;
    };
    auto next_unit = [&](int u) {   // the wave's next unit with keys, from u on
      if (u < pre_units && u * kAttnUnit + 32 * wave >= x.pre) u = pre_units;
      return u < u1 && (u < pre_units || (u - pre_units) * kAttnUnit + 32 * wave < lim_last) ? u : u1;
    };
    // The pages of a unit's halves are asked for ahead of the keys of the unit before: loads come back in order, and a
    // page that is waited for would be waited for behind all keys and values on the way.
    struct Pages { int p0, p1; };
    auto ask_pages = [&](int u) {
      const bool pre = u < pre_units;
      const int key0 = (pre ? u : u - pre_units) * kAttnUnit + 32 * wave, last = (pre ? x.pre : lim_last) - 1;
      const int32_t* table = pre ? a.prefix_pages : own_pages;
      return Pages{table[key0 >> ps], table[min(key0 + 16, last) >> ps]};
    };
    auto keys_of = [&](int u, const Pages& g) {
      Keys k;
      k.pre = u < pre_units;
      k.key0 = (k.pre ? u : u - pre_units) * kAttnUnit + 32 * wave;
      k.have = k.pre ? x.pre : lim_last;
      k.ok0 = attn_page(a.c, a.flags, __builtin_amdgcn_readfirstlane(g.p0), head, k.at0);
      k.ok1 = attn_page(a.c, a.flags, __builtin_amdgcn_readfirstlane(g.p1), head, k.at1);
      if (k.key0 + 16 >= k.have) {   // a half of no keys reads what is there of the first one's page
        k.ok1 = false;
        k.at1 = k.at0;
      }
      k.t0 = k.key0 & ((1 << ps) - 1);
      k.t1 = (k.key0 + 16) & ((1 << ps) - 1);
      return k;
    };
    Raw<I8> kf[2 * NS], vf[NJ];
    f32x4 ks[I8 ? 2 : 1], vs[I8 ? 2 : 1];
    auto scales = [&](const float* from, const Keys& k, f32x4* to) {
      const float* f = from + (g & 2 ? k.at1 / D + k.t1 : k.at0 / D + k.t0) + (g & 1) * 8;
      to[0] = *reinterpret_cast<const f32x4*>(f);
      to[1] = *reinterpret_cast<const f32x4*>(f + 4);
    };
    // line c of block b holds token 8 (c / 4) + 4 b + c % 4, in half c / 8
    auto ask_keys = [&](const Keys& k) {
      const size_t from = (c & 8 ? k.at1 + (size_t)k.t1 * D : k.at0 + (size_t)k.t0 * D) + g * 128 + ((8 * (c >> 2) + (c & 3)) & 15) * 8;
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int b = 0; b < 2; ++b) kf[2 * s + b].load(a.c.k, from + s * 512 + b * 32);
      if constexpr (I8) scales(a.c.ks, k, ks);
    };
    auto ask_values = [&](const Keys& k) {
      const size_t from = (g & 2 ? k.at1 + (size_t)k.t1 * D : k.at0 + (size_t)k.t0 * D) + (size_t)(g & 1) * 8 * D + c * 8;
#pragma unroll
      for (int j = 0; j < NJ; ++j) vf[j].load(a.c.v, from + j * 128);
      if constexpr (I8) scales(a.c.vs, k, vs);
    };

    // what follows the last unit is the last again: no load stands under a branch
    auto after = [&](int u) {
      const int n = next_unit(u + 1);
      return n < u1 ? n : u;
    };
    int u = next_unit(u0);
    if (u < u1) {
      Keys cur = keys_of(u, ask_pages(u));
      int un = after(u);
      Pages pages = ask_pages(un);
      __builtin_amdgcn_sched_barrier(0);   // in the loop's order, or the loop waits for values before its first product
      ask_keys(cur);
      __builtin_amdgcn_sched_barrier(0);
      ask_values(cur);
      __builtin_amdgcn_sched_barrier(0);
      for (bool more = true; more;) {   // in here, or the compiler sees a way to it past the loads and waits for all
        f32x4 st[RB][2];
#pragma unroll
        for (int b = 0; b < RB; ++b) st[b][0] = st[b][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const bf16x8 k8 = kf[2 * s + n].get();
#pragma unroll
            for (int b = 0; b < RB; ++b) st[b][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k8, qf[b][s], st[b][n], 0, 0, 0);
          }
        float z[RB][8];
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            z[b][n] = st[b][n >> 2][n & 3];
            if constexpr (I8) z[b][n] *= ks[n >> 2][n & 3];   // first: q times codes may be 127 times what q k is
            z[b][n] *= a.scale;
          }
        __builtin_amdgcn_sched_barrier(0);
        const Keys nxt = keys_of(un, pages);
        const int uf = after(un);
        pages = ask_pages(uf);
        ask_keys(nxt);
        __builtin_amdgcn_sched_barrier(0);
        const int mine = cur.key0 + 8 * g;   // the lane's first key
        const bool ok = g & 2 ? cur.ok1 : cur.ok0;
        const bool masked = cur.key0 + 32 > (cur.pre ? x.pre : lim_first) || !cur.ok0 || !cur.ok1;
        if (masked) {
#pragma unroll
          for (int b = 0; b < RB; ++b) {
            const int lim = ok ? (cur.pre ? x.pre : lim_own[b]) - mine : 0;
#pragma unroll
            for (int n = 0; n < 8; ++n)
              if (n >= lim) z[b][n] = kNegInf;
          }
        }
        bf16x8 hi[RB], lo[RB];
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          float top = z[b][0];
#pragma unroll
          for (int n = 1; n < 8; ++n) top = fmaxf(top, z[b][n]);
          top = fmaxf(top, __shfl_xor(top, 16));
          top = fmaxf(top, __shfl_xor(top, 32));
          if (__ballot(top > m_run[b] + 8.f)) {   // as below, in many rows
            const float m_new = fmaxf(m_run[b], top);
            const float alpha = __builtin_amdgcn_exp2f(m_run[b] - (m_new == kNegInf ? 0.f : m_new));
            m_run[b] = m_new;
            l_run[b] *= alpha;
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[b][j] *= alpha;
          }
          const float base = m_run[b] == kNegInf ? 0.f : m_run[b];
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            float e = __builtin_amdgcn_exp2f(rounded_less(z[b][n], base));
            l_run[b] += e;
            if constexpr (I8) e = z[b][n] == kNegInf ? 0.f : e * vs[n >> 2][n & 3];
            hi[b][n] = (__bf16)e;
            lo[b][n] = (__bf16)(e - (float)hi[b][n]);
          }
        }
        uint32_t odd = 0;
        if (!I8 && masked) {
          // values behind the tokens may be anything: 0 instead.  An infinity or NaN that only some of the rows
          // see is kept out of the product, which has a 0 for the others, and added to those rows.
          const int there = ok ? cur.have - mine : 0;
          const bool some = !cur.pre && lim_first < lim_last;
#pragma unroll
          for (int j = 0; j < NJ; ++j) odd |= vf[j].keep(there, some);
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const bf16x8 v8 = vf[j].get();
#pragma unroll
          for (int b = 0; b < RB; ++b) {
            acc[b][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v8, lo[b], acc[b][j], 0, 0, 0);
            acc[b][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v8, hi[b], acc[b][j], 0, 0, 0);
          }
        }
        if (!I8 && __ballot(odd != 0)) {
          for (int n = 0; n < 32 && cur.key0 + n < cur.have; ++n) {
            const bool half = n & 16;
            if (!(half ? cur.ok1 : cur.ok0)) continue;
            const uint16_t* vp = static_cast<const uint16_t*>(a.c.v) + (half ? cur.at1 : cur.at0);
            const int tok = half ? cur.t1 + (n & 15) : cur.t0 + n;
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
              for (int d = 0; d < 4; ++d) {
                const float v = bf16lo(vp[v_place(D, tok, 16 * j + 4 * g + d)]);
#pragma unroll
                for (int b = 0; b < RB; ++b)
                  if (!(fabsf(v) <= __FLT_MAX__) && cur.key0 + n < lim_own[b]) acc[b][j][d] += v;
                if (d == 3) __builtin_amdgcn_sched_barrier(0);   // or all are read at once, and spill others
              }
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        ask_values(nxt);
        cur = nxt;
        more = un != u;
        u = un;
        un = uf;
      }
    }
    // the four waves' parts become one
    const bool whole = at.split == 1 && p.set == ATTN_ALL;
    const size_t slot = (size_t)it * KH + head;
    __syncthreads();   // the item before has been read
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      l_run[b] += __shfl_xor(l_run[b], 16);
      l_run[b] += __shfl_xor(l_run[b], 32);
      if (g == 0) s_m[wave][16 * b + c] = m_run[b];
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      float m_all = s_m[0][16 * b + c];
#pragma unroll
      for (int w = 1; w < 4; ++w) m_all = fmaxf(m_all, s_m[w][16 * b + c]);
      const float f = m_all == kNegInf ? 0.f : __builtin_amdgcn_exp2f(m_run[b] - m_all);
      if (g == 0) s_l[wave][16 * b + c] = l_run[b] * f;
      if (b > 0) __syncthreads();   // the block before has been read
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        *reinterpret_cast<f32x4*>(&s_o[(wave * 16 + c) * kLd + 16 * j + 4 * g]) = acc[b][j] * f;
      __syncthreads();
      for (int q4 = tid; q4 < 16 * (D / 4); q4 += 256) {
        const int row = q4 / (D / 4), d = 4 * (q4 % (D / 4)), tr = 16 * b + row, rr = rt * kRows + tr;
        if (rr >= x.rows) continue;
        f32x4 o = *reinterpret_cast<const f32x4*>(&s_o[row * kLd + d]);
        float l = s_l[0][tr], m = s_m[0][tr];
#pragma unroll
        for (int w = 1; w < 4; ++w) {
          o += *reinterpret_cast<const f32x4*>(&s_o[(w * 16 + row) * kLd + d]);
          l += s_l[w][tr];
          m = fmaxf(m, s_m[w][tr]);
        }
        if (whole) {
          write_row(a, (size_t)(x.row0 + rr / a.group) * a.q_heads + head * a.group + rr % a.group, D, d, o, m, l);
        } else {
          *reinterpret_cast<f32x4*>(p.o + (slot * kRows + tr) * D + d) = o;
          if (d == 0) {
            p.ml[(slot * kRows + tr) * 2] = m;
            p.ml[(slot * kRows + tr) * 2 + 1] = l;
          }
        }
      }
    }
  }
}

// Many rows (128 a tile): prompts, and the shared prefix of a batch.  Each wave
// has 32 rows, in matrix instructions of 32 x 32; the four share a tile of 64
// keys that goes from memory straight to LDS, in the order in which it lies,
// while the tile before it is worked on.  Lines of S^T are dealt as above, so
// that a lane's scores of 16 keys are eight neighbouring tokens': P never
// leaves its registers.
//
// The maximum that scores are taken against is raised only when a row's grows
// by 2^8: numerators up to 2^8 lose nothing in bf16 or in the fp32 sums, and the
// outputs are rescaled a few times a row instead of once a tile.
//
// Numerators enter the second product as one bf16 part, half a step of 2^-8 each: of the outputs' own size they are
// off by 0.0023 in all, 0.0017 of it the outputs' rounding.  Two parts take a third product for every two (2048 tokens
// over 8192: 425 us for 322, 64 wide 256 for 196, 256 wide 447 for 365).  With TWO they do: rows of few-row sequences
// over a prefix, which have two over their own keys, so that a request's bits do not go by how many others are behind
// the prefix (64 tokens behind 16384: 59 us for 52; 64 of 2000 behind 8192: the same).
//
// Bound by the matrix cores (44 % busy) and the softmax between them: 4096 tokens
// over 16384 of 32 heads of 128 run at 960 TFLOP/s, where a large library product
// reaches 1235; 2048 over 8192 at 750 (64 wide: 610, 256 wide: 660).  Eight waves of
// 256 rows, half of them at the products while the others are at the softmax, with
// a barrier at each change, were slower (319 us for 300, 64 wide 232 for 193): the
// barriers and what is done between them cost more than the overlap gave, which two
// workgroups a CU find by themselves.
template <int D, bool I8, bool TWO>
__device__ __forceinline__ void attn_many(const AttnArgs& a, const AttnParts& p, int block, int blocks, AttnPlan& plan, uint8_t* lds) {
  constexpr int kRows = 128, KT = 64, NQ = D / 16, NB = KT / 32, NO = D / 32, kBlocks = KT / 16, kTiles = kAttnUnit / KT;
  static_assert(kBlocks == 4, "a block of K and of V for each wave");
  constexpr int kTile = KT * D;   // elements of K or V
  __shared__ __align__(16) int32_t s_valid[2][4];     // tokens that count of each 16
  __shared__ int32_t s_odd;
  __shared__ __align__(16) float s_ks[I8 ? 2 : 1][I8 ? KT : 4], s_vs[I8 ? 2 : 1][I8 ? KT : 4];
  uint16_t* const s_kv = reinterpret_cast<uint16_t*>(lds);   // [2][K | V]
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, c = lane & 31, hh = lane >> 5;
  const int KH = a.c.heads, ps = a.c.page_shift;
  const int total = attn_plan(a, p, plan, block == 0);
  // -Inf of a key that is not seen stays -Inf under any scale
  const float scale = a.scale == 0.f ? 1e-45f : fabsf(a.scale);
  const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
  // where the lane's operands lie in a tile
  const int line = 16 * ((c >> 3) >> 1) + 8 * ((c >> 2) & 1) + 4 * ((c >> 3) & 1) + (c & 3);
  const int k_at = (line >> 4) * 16 * D + hh * 128 + (line & 15) * 8, v_at = hh * 8 * D + c * 8;
  for (int idx = block; idx < total * KH; idx += blocks) {
    const int head = idx % KH, nth = idx / KH;
    const AttnPlace at = attn_place(a, p, plan, nth);
    const AttnEntry& x = at.x;
    const int split = at.split, e = at.e;
    const int local = x.tiles * split - 1 - (nth - at.first);   // the last tiles see most keys: first
    const int part = local % split, rt = local / split, it = at.first + local;
    const int r0 = rt * kRows + 32 * wave;
    const bool has_rows = r0 < x.rows;
    const int r = min(r0 + c, x.rows - 1);
    const int i = r / a.group, h = head * a.group + r % a.group;
    auto seen = [&](int row) { return min(max(x.causal + row / a.group + 1, 0), x.own); };
    const int lim_own = seen(r), lim_first = seen(min(r0, x.rows - 1)), lim_wave = seen(min(r0 + 31, x.rows - 1));
    const int lim_tile = seen(rt * kRows), lim_last = seen(min(rt * kRows + kRows, x.rows) - 1);
    const int pre_units = attn_units(x.pre), units = pre_units + attn_units(lim_last);
    const int per = (units + split - 1) / split, u0 = part * per, u1 = min(units, u0 + per);
    // tiles: [0, pre_end) of the prefix, [own_begin, own_end) of the sequence's own
    const int pre_end = (x.pre + KT - 1) / KT, own_begin = pre_units * kTiles, own_end = own_begin + (lim_last + KT - 1) / KT;
    const int t_end = min(u1 * kTiles, own_end);
    auto skip = [&](int t) { return t >= pre_end && t < own_begin ? own_begin : t; };
    const int32_t* own_pages = p.set == ATTN_PREFIX ? nullptr : a.pages + (size_t)e * a.pages_ld;

    bf16x8 qf[NQ];
    const uint16_t* qp = a.q + ((size_t)(x.row0 + i) * a.q_heads + h) * D + 8 * hh;
#pragma unroll
    for (int s = 0; s < NQ; ++s) {
      u32x4 w = *reinterpret_cast<const u32x4*>(qp + 16 * s);
      w ^= u32x4{flip, flip, flip, flip};
      qf[s] = __builtin_bit_cast(bf16x8, w);
    }
    f32x16 acc[NO];
#pragma unroll
    for (int o = 0; o < NO; ++o)
#pragma unroll
      for (int n = 0; n < 16; ++n) acc[o][n] = 0.f;
    float m_run = kNegInf, l_run = 0.f;

    // A tile's loading: wave w has 16-token block w of K and of V.
    // 8-bit tiles go through registers, 16 bytes of codes at a time, and become bf16 on the way.
    constexpr int kRaw = I8 ? KT * D / 16 / 256 : 1;
    u32x4 raw_k[kRaw], raw_v[kRaw];
    float raw_scale = 0.f;
    // the 16-token block of the wave's n-th piece, and of the lane's scale (8 bits)
    auto block_of = [&](int n) { return I8 ? (wave * 64 + 256 * n) / D : wave; };
    const int scale_block = tid % KT / 16;
    auto page_of = [&](int t, int blk) {   // 0 where nothing is to be loaded
      const bool pre = t < own_begin;
      const int key = (pre ? t : t - own_begin) * KT + 16 * blk, have = pre ? x.pre : lim_last;
      return t < t_end && key < have ? (pre ? a.prefix_pages : own_pages)[key >> ps] : 0;
    };
    // pages: of the wave's pieces, asked for a tile ahead, as the loads that need them would wait for them
    struct Pages { int piece[kRaw], scale; };
    auto ask_pages = [&](int t) {
      Pages g;
#pragma unroll
      for (int n = 0; n < kRaw; ++n) g.piece[n] = page_of(t, block_of(n));
      g.scale = I8 ? page_of(t, scale_block) : 0;
      return g;
    };
    auto issue = [&](int t, int buf, const Pages& g) {
      const bool pre = t < own_begin;
      const int key0 = (pre ? t : t - own_begin) * KT, have = pre ? x.pre : lim_last;
      if constexpr (I8) {
#pragma unroll
        for (int n = 0; n < kRaw; ++n) {
          const int page = __builtin_amdgcn_readfirstlane(g.piece[n]), key = key0 + 16 * block_of(n);
          const size_t base = kv_page(a.c, (uint32_t)page < (uint32_t)a.c.n_pages ? page : 0, head) +
                              (size_t)(key & ((1 << ps) - 1)) * D + ((tid + 256 * n) % D) * 16;
          raw_k[n] = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(a.c.k) + base);
          raw_v[n] = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(a.c.v) + base);
        }
        if (tid < 2 * KT) {
          const int tok = tid % KT, key = key0 + tok;
          const bool ok = (uint32_t)g.scale < (uint32_t)a.c.n_pages;
          if (!ok) set_flag(a.flags, kFlagIndex);
          raw_scale = (tid < KT ? a.c.ks : a.c.vs)[(((size_t)(ok ? g.scale : 0) * KH + head) << ps) + (key & ((1 << ps) - 1))];
          if (tid < KT && (tok & 15) == 0) s_valid[buf][tok >> 4] = ok ? min(max(have - key, 0), 16) : 0;
        }
      } else {
        const int blk = block_of(0), key = key0 + 16 * blk, page = __builtin_amdgcn_readfirstlane(g.piece[0]);
        const bool ok = (uint32_t)page < (uint32_t)a.c.n_pages;
        if (!ok) set_flag(a.flags, kFlagIndex);
        if (lane == 0) s_valid[buf][blk] = ok ? min(max(have - key, 0), 16) : 0;
        if (key < have) {
          const size_t at = kv_page(a.c, ok ? page : 0, head) + (size_t)(key & ((1 << ps) - 1)) * D + lane * 8;
          uint16_t* to = s_kv + buf * 2 * kTile + blk * 16 * D;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint16_t* from = static_cast<const uint16_t*>(kv ? a.c.v : a.c.k) + at;
#pragma unroll
            for (int n = 0; n < D / 32; ++n)
              __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(from + 512 * n),
                                               (lds_void*)(to + kv * kTile + 512 * n), 16, 0, 0);
          }
        }
      }
    };
    auto finish = [&](int buf) {
      if constexpr (I8) {
#pragma unroll
        for (int n = 0; n < kRaw; ++n) {
          uint16_t* to = s_kv + buf * 2 * kTile + (tid + 256 * n) * 16;
          *reinterpret_cast<bf16x8*>(to) = bf16x8_of_codes(u32x2{raw_k[n].x, raw_k[n].y});
          *reinterpret_cast<bf16x8*>(to + 8) = bf16x8_of_codes(u32x2{raw_k[n].z, raw_k[n].w});
          *reinterpret_cast<bf16x8*>(to + kTile) = bf16x8_of_codes(u32x2{raw_v[n].x, raw_v[n].y});
          *reinterpret_cast<bf16x8*>(to + kTile + 8) = bf16x8_of_codes(u32x2{raw_v[n].z, raw_v[n].w});
        }
        if (tid < 2 * KT) (tid < KT ? s_ks : s_vs)[buf][tid % KT] = raw_scale;
      }
    };

    int t = skip(u0 * kTiles);
    __syncthreads();   // the item before is done with LDS
    if (t < t_end) {
      issue(t, 0, ask_pages(t));
      finish(0);
    }
    int next = skip(t + 1);
    Pages pages = ask_pages(next);
    for (int buf = 0; t < t_end; buf ^= 1) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      const int after = skip(next + 1);
      if (next < t_end) {
        issue(next, buf ^ 1, pages);
        pages = ask_pages(after);
      }
      const bool pre = t < own_begin;
      const int key0 = (pre ? t : t - own_begin) * KT;
      int valid[kBlocks], least = 16;
#pragma unroll
      for (int n = 0; n < kBlocks; ++n) {
        valid[n] = __builtin_amdgcn_readfirstlane(s_valid[buf][n]);
        least = min(least, valid[n]);
      }
      // A tile that some rows do not see whole: values behind the tokens may be anything, and an infinity or NaN of
      // a token would reach the rows that do not see it, as a product with 0.  Both become 0 here, and the rows
      // that do see it get it below.
      bool odd = false;
      if (!I8 && (least < 16 || (!pre && key0 + KT > lim_tile))) {
        if (tid == 0) s_odd = 0;
        __syncthreads();
        uint32_t any = 0;
#pragma unroll
        for (int n = 0; n < kTile / 8 / 256; ++n) {
          const int grp = (tid + 256 * n) / D;
          bf16x8* at = reinterpret_cast<bf16x8*>(s_kv + buf * 2 * kTile + kTile) + tid + 256 * n;
          bf16x8 v = keep_first(*at, s_valid[buf][grp >> 1] - 8 * (grp & 1));
          any |= drop_nonfinite(v);
          *at = v;
        }
        if (any) s_odd = 1;
        __syncthreads();
        odd = __builtin_amdgcn_readfirstlane(s_odd) != 0;
      }
      if (has_rows && (pre || key0 < lim_wave)) {
        const uint16_t* sk = s_kv + buf * 2 * kTile + k_at;
        const uint16_t* sv = s_kv + buf * 2 * kTile + kTile + v_at;
        f32x16 st[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int n = 0; n < 16; ++n) st[b][n] = 0.f;
        fed<D == 64 ? 2 : 4, NQ * NB>([&](int n) { return *reinterpret_cast<const bf16x8*>(sk + (n % NB) * 32 * D + (n / NB) * 256); },
                     [&](int n, bf16x8 k) {
                       st[n % NB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, qf[n / NB], st[n % NB], 0, 0, 0);
                     });
        if constexpr (I8) {
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int n = 0; n < 16; ++n) st[b][n] *= s_ks[buf][32 * b + 16 * (n >> 3) + 8 * hh + (n & 7)];
        }
        const bool masked = least < 16 || (!pre && key0 + KT > lim_first);
        if (masked) {
          const int lim = (pre ? x.pre : lim_own) - key0 - 8 * hh;
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int n = 0; n < 16; ++n)
              if ((n & 7) >= min(lim - 32 * b - 16 * (n >> 3), valid[2 * b + (n >> 3)] - 8 * hh)) st[b][n] = kNegInf;
        }
        float top = st[0][0];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int n = 0; n < 16; ++n) top = fmaxf(top, st[b][n]);
        top = fmaxf(top, __shfl_xor(top, 32)) * scale;
        if (__ballot(top > m_run + 8.f)) {
          const float m_new = fmaxf(m_run, top);
          const float alpha = __builtin_amdgcn_exp2f(m_run - (m_new == kNegInf ? 0.f : m_new));
          m_run = m_new;
          l_run *= alpha;
#pragma unroll
          for (int o = 0; o < NO; ++o)
#pragma unroll
            for (int n = 0; n < 16; ++n) acc[o][n] *= alpha;
        }
        const float base = m_run == kNegInf ? 0.f : m_run;
        // Below 2^24 the product that is not rounded before the subtraction is within 1/2 of the one that base was
        // rounded from, which both sums have alike.  Beyond, numerators would leave fp32: scores are rounded first, as
        // base was, so that the largest one's exponent is 0.
        const bool far = __ballot(fabsf(base) > 16777216.f) != 0;
        if (far) {
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int n = 0; n < 16; ++n) st[b][n] = rounded_less(st[b][n] * scale, base);
        }
        const float by = far ? 1.f : scale, less = far ? 0.f : base;
        float sum = 0.f;
        bf16x8 pf[NB][2], pl[TWO ? NB : 1][2];
        auto enter = [&](int b, int n, float w) {
          const __bf16 hi = (__bf16)w;
          pf[b][n >> 3][n & 7] = hi;
          if constexpr (TWO) pl[b][n >> 3][n & 7] = (__bf16)(w - (float)hi);
        };
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            const float e2 = __builtin_amdgcn_exp2f(fmaf(st[b][n], by, -less));
            sum += e2;
            if constexpr (I8) st[b][n] = e2;
            else enter(b, n, e2);
          }
          __builtin_amdgcn_sched_barrier(0);   // or the values' reads come ahead of all this, and registers spill
        }
        if constexpr (I8) {
          // a token that a row does not see may have any scale
          auto weigh = [&](auto some) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int n = 0; n < 16; ++n) {
                const float v = st[b][n] * s_vs[buf][32 * b + 16 * (n >> 3) + 8 * hh + (n & 7)];
                enter(b, n, some && st[b][n] == 0.f ? 0.f : v);
              }
          };
          if (masked) weigh(std::true_type{});
          else weigh(std::false_type{});
        }
        l_run += sum;
        fed<D == 64 ? 2 : 4, NB * 2 * NO>(
            [&](int n) { return *reinterpret_cast<const bf16x8*>(sv + (n / NO) * 2 * 8 * D + (n % NO) * 256); },
            [&](int n, bf16x8 v) {
              if constexpr (TWO)
                acc[n % NO] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, pl[n / NO / 2][n / NO % 2], acc[n % NO], 0, 0, 0);
              acc[n % NO] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, pf[n / NO / 2][n / NO % 2], acc[n % NO], 0, 0, 0);
            });
        if (odd) {
          int h4 = 4 * hh;
          asm volatile("" : "+v"(h4));   // or the places below are formed ahead of the loops, and spilled
          for (int n = 0; n < KT; ++n) {
            if ((n & 15) >= s_valid[buf][n >> 4]) continue;
            const int key = key0 + n;
            const uint16_t* vp = static_cast<const uint16_t*>(a.c.v) +
                                 kv_page(a.c, (pre ? a.prefix_pages : own_pages)[key >> ps], head);   // a page of the cache
            const bool mine = key < (pre ? x.pre : lim_own);
#pragma unroll
            for (int o = 0; o < NO; ++o)
#pragma unroll
              for (int d = 0; d < 16; ++d) {
                const float v = bf16lo(vp[v_place(D, key & ((1 << ps) - 1), 32 * o + 8 * (d >> 2) + h4 + (d & 3))]);
                if (!(fabsf(v) <= __FLT_MAX__) && mine) acc[o][d] += v;
                if ((d & 3) == 3) __builtin_amdgcn_sched_barrier(0);   // or all are read at once, and spill others
              }
          }
        }
      }
      if (next < t_end) finish(buf ^ 1);
      t = next;
      next = after;
    }
    l_run += __shfl_xor(l_run, 32);
    int mine = r0 + c;
    asm volatile("" : "+v"(mine));   // the row's place is formed again here, not kept over the tiles
    const int rr = mine;
    if (rr < x.rows) {
      const bool whole = split == 1 && p.set == ATTN_ALL;
      const size_t slot = ((size_t)it * KH + head) * kRows + 32 * wave + c;
      const size_t row = (size_t)(x.row0 + rr / a.group) * a.q_heads + head * a.group + rr % a.group;
#pragma unroll
      for (int o = 0; o < NO; ++o)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const f32x4 v = {acc[o][4 * n], acc[o][4 * n + 1], acc[o][4 * n + 2], acc[o][4 * n + 3]};
          const int d = 32 * o + 8 * n + 4 * hh;
          if (whole) write_row(a, row, D, d, v, m_run, l_run);
          else *reinterpret_cast<f32x4*>(p.o + slot * D + d) = v;
        }
      if (!whole && hh == 0) {
        p.ml[slot * 2] = m_run;
        p.ml[slot * 2 + 1] = l_run;
      }
    }
  }
}

constexpr int attn_lds(int dim, int rows) { return rows == 128 ? 2 * 2 * 64 * dim * 2 : 4 * 16 * (dim + 4) * 4; }

// Workgroups a CU that the registers are cut for.  (Three of 16 rows at 128 dimensions: 8 bits 46 us for 52, 64
// tokens of 2000; bf16 spills, 72 for 64.  256 dimensions take all registers, and bf16 tiles of 32 rows spill 76 to 104
// bytes a lane even so: 16 windows of 8 rows and 4000 tokens, 16 heads over 4, 44 us, of 4 rows in tiles of 16, which do
// not, 42.  64 dimensions of few rows beside a prefix's two parts spill 12 bytes, over 8 bits 76; two workgroups for
// three: 64 tokens of 2000 behind 4096 45 us for 41, over 8 bits 45 for 40, but of 300 behind 16384 48 for 47 and 53 for 65.)
constexpr int attn_occupancy(int dim, bool i8, int rows) {
  return dim == 256 ? 1 : dim == 64 ? (rows == 32 ? 2 : 3) : i8 && rows == 16 ? 3 : 2;
}

template <int D, bool I8, int ROWS, bool TWO = false>
__device__ __forceinline__ void attn_rows(const AttnArgs& a, const AttnParts& p, int block, int blocks, AttnPlan& plan, uint8_t* lds) {
  if constexpr (ROWS == 128) attn_many<D, I8, TWO>(a, p, block, blocks, plan, lds);
  else attn_few<D, I8, ROWS / 16>(a, p, block, blocks, plan, lds);
}

template <int D, bool I8, int ROWS>
__global__ __launch_bounds__(256, attn_occupancy(D, I8, ROWS)) void k_attn(AttnArgs a, AttnParts p) {
  __shared__ AttnPlan plan;
  extern __shared__ __align__(16) uint8_t lds[];
  attn_rows<D, I8, ROWS>(a, p, blockIdx.x, gridDim.x, plan, lds);
}

// Several sequences behind a prefix, in one launch: pre_grid workgroups have the
// prefix's parts (tiles of PRE rows), the others the sequences' (OWN rows).  Side
// by side, the prefix's products fill the matrix cores while the sequences' keys
// and values stream (16 windows over 8 bits: 45 us, one after the other 71; 64
// tokens behind 8192: 92 for 109.  Since then the few rows' loop has become faster:
// 41 and 89, of which this kernel has 35 and 75, 4.9 TB/s).
template <int D, bool I8, int OWN, int PRE>
__global__ __launch_bounds__(256, attn_occupancy(D, I8, OWN > PRE ? OWN : PRE)) void k_attn_shared(AttnArgs a, AttnPair sets, int pre_grid) {
  __shared__ AttnPlan plan;
  extern __shared__ __align__(16) uint8_t lds[];
  const bool is_pre = (int)blockIdx.x < pre_grid;
  const int block = is_pre ? blockIdx.x : blockIdx.x - pre_grid, blocks = is_pre ? pre_grid : gridDim.x - pre_grid;
  if constexpr (OWN == PRE) attn_rows<D, I8, OWN>(a, sets.p[is_pre], block, blocks, plan, lds);
  else if (is_pre) attn_rows<D, I8, PRE, true>(a, sets.p[1], block, blocks, plan, lds);
  else attn_rows<D, I8, OWN>(a, sets.p[0], block, blocks, plan, lds);
}

// The parts of one row and head, joined in order.  D / 4 lanes have four
// dimensions each of a head; with GROUPS > 1 so many of them share the head's
// parts (few rows, many parts), else a workgroup has several heads of its row.
template <int D, int GROUPS>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, AttnParts own, AttnParts pre) {
  constexpr int L = D / 4, kHeads = 256 / L / GROUPS;
  __shared__ float s_o[GROUPS > 1 ? GROUPS : 1][D + 4];
  __shared__ float s_l[GROUPS];
  const int m = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
  // the row's sequence; starts that fall count as the largest before them
  int seq = -1, begin = 0, row0 = 0;
  {
    int up = 0, before = 0;
    for (int b = 0; b <= a.n_seq; b += 64) {
      const int e = b + lane;
      const int v = max(wave_scan_max(e <= a.n_seq ? min(max(a.q_start[e], 0), a.M) : 0), up);
      if (b == 0) row0 = __shfl(v, 0);
      const int n = __popcll(__ballot(e <= a.n_seq && v <= m));
      if (n) begin = __shfl(v, n - 1);
      before += n;
      up = __shfl(v, 63);
      if (n < 64) break;
    }
    seq = before - 1;
  }
  if (seq < 0 || seq >= a.n_seq) return;   // no sequence's row
  const int i = m - begin, KH = a.c.heads;
  const int split = own.plan[2 + 2 * seq + 1], first = own.plan[2 + 2 * seq];
  const int pre_split = pre.rows ? pre.plan[3] : 0, parts = split + pre_split;
  if (!pre.rows && split == 1) return;     // written by its only part
  const int grp = GROUPS > 1 ? tid / L : 0, l0 = tid % L, d = 4 * l0;
  const int h = GROUPS > 1 ? blockIdx.y : blockIdx.y * kHeads + tid / L;
  if (GROUPS == 1 && h >= a.q_heads) return;
  const int head = h / a.group, r = i * a.group + h % a.group, rt = r / own.rows;
  const size_t slot0 = ((size_t)(first + rt * split) * KH + head) * own.rows + r % own.rows, step = (size_t)KH * own.rows;
  const int rp = (m - row0) * a.group + h % a.group;
  const size_t pslot0 = pre.rows ? ((size_t)(rp / pre.rows * pre_split) * KH + head) * pre.rows + rp % pre.rows : 0;
  const size_t pstep = (size_t)KH * pre.rows;
  auto ml_of = [&](int s) { return s < pre_split ? pre.ml + 2 * (pslot0 + s * pstep) : own.ml + 2 * (slot0 + (s - pre_split) * step); };
  auto o_of = [&](int s) {
    return *reinterpret_cast<const f32x4*>(s < pre_split ? pre.o + (pslot0 + s * pstep) * D + d : own.o + (slot0 + (s - pre_split) * step) * D + d);
  };
  constexpr int kSeen = GROUPS > 1 ? 64 : L;   // lanes that look for the maximum together
  float top = kNegInf;
  for (int s = lane % kSeen; s < parts; s += kSeen) top = fmaxf(top, ml_of(s)[0]);
#pragma unroll
  for (int off = kSeen / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
  const float base = top == kNegInf ? 0.f : top;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  float l = 0.f;
  int s = grp;
  for (; s + 3 * GROUPS < parts; s += 4 * GROUPS) {   // four parts on the way at once
    f32x4 v[4];
    float f[4], w[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float* ml = ml_of(s + n * GROUPS);
      f[n] = ml[0];
      w[n] = ml[1];
      v[n] = o_of(s + n * GROUPS);
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      f[n] = __builtin_amdgcn_exp2f(f[n] - base);
      l += f[n] * w[n];
      o += f[n] * v[n];
    }
  }
  for (; s < parts; s += GROUPS) {
    const float* ml = ml_of(s);
    const f32x4 v = o_of(s);
    const float f = __builtin_amdgcn_exp2f(ml[0] - base);
    l += f * ml[1];
    o += f * v;
  }
  if constexpr (GROUPS > 1) {
    *reinterpret_cast<f32x4*>(&s_o[grp][d]) = o;
    if (l0 == 0) s_l[grp] = l;
    __syncthreads();
    if (grp > 0) return;
#pragma unroll
    for (int w = 1; w < GROUPS; ++w) {
      o += *reinterpret_cast<const f32x4*>(&s_o[w][d]);
      l += s_l[w];
    }
  }
  write_row(a, (size_t)m * a.q_heads + h, D, d, o, top, l);
}

template <int D, bool I8>
static void launch_attn_of(const AttnArgs& a, const AttnParts& own, int own_grid, const AttnParts& pre, int pre_grid, hipStream_t s) {
#define Q4NX_ONE(ROWS) hipLaunchKernelGGL((k_attn<D, I8, ROWS>), dim3(own_grid), dim3(256), attn_lds(D, ROWS), s, a, own)
#define Q4NX_SHARED(OWN, PRE)                                                                    \
  hipLaunchKernelGGL((k_attn_shared<D, I8, OWN, PRE>), dim3(pre_grid + own_grid), dim3(256),     \
                     std::max(attn_lds(D, OWN), attn_lds(D, PRE)), s, a, (AttnPair{{own, pre}}), pre_grid)
  if (pre.rows == 0) {
    if (own.rows == 128) Q4NX_ONE(128);
    else if (own.rows == 32) Q4NX_ONE(32);
    else Q4NX_ONE(16);
  } else if (own.rows == 128) Q4NX_SHARED(128, 128);
  else if (own.rows == 32 && pre.rows == 32) Q4NX_SHARED(32, 32);
  else if (own.rows == 32) Q4NX_SHARED(32, 128);
  else if (pre.rows == 16) Q4NX_SHARED(16, 16);
  else Q4NX_SHARED(16, 128);
#undef Q4NX_ONE
#undef Q4NX_SHARED
}

hipError_t launch_attn(const AttnArgs& a, const AttnParts& own, int own_grid, const AttnParts& pre, int pre_grid, hipStream_t s) {
#define Q4NX_ATTN(D)                                                    \
  if (a.c.ks) launch_attn_of<D, true>(a, own, own_grid, pre, pre_grid, s); \
  else launch_attn_of<D, false>(a, own, own_grid, pre, pre_grid, s)
  if (a.c.dim == 64) { Q4NX_ATTN(64); }
  else if (a.c.dim == 128) { Q4NX_ATTN(128); }
  else { Q4NX_ATTN(256); }
#undef Q4NX_ATTN
  return hipGetLastError();
}

hipError_t launch_attn_join(const AttnArgs& a, const AttnParts& own, const AttnParts& prefix, hipStream_t s) {
  // from about 64 rows of 32 heads on the heads alone fill the GPU (64 rows of 26 parts: 8.3 us); under it a head's
  // parts are shared out (16 windows of 28 heads: 7.9 us; a call is the same within 1 us with the border at 1024)
#define Q4NX_JOIN(D)                                                                                                     \
  if ((int64_t)a.M * a.q_heads < 2048)                                                                                   \
    hipLaunchKernelGGL((k_attn_join<D, 1024 / D>), dim3(a.M, a.q_heads), dim3(256), 0, s, a, own, prefix);               \
  else                                                                                                                   \
    hipLaunchKernelGGL((k_attn_join<D, 1>), dim3(a.M, (a.q_heads + 1024 / D - 1) / (1024 / D)), dim3(256), 0, s, a, own, \
                       prefix)
  if (a.c.dim == 64) { Q4NX_JOIN(64); }
  else if (a.c.dim == 128) { Q4NX_JOIN(128); }
  else { Q4NX_JOIN(256); }
#undef Q4NX_JOIN
  return hipGetLastError();
}

}  // namespace q4nx
