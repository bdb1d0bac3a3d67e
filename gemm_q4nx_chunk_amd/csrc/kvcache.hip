// Rotation by position and append to the paged cache.
//
//   t = pos * inv_freq[i];  (a, b) -> (a cos t - b sin t, b cos t + a sin t)
//
// A workgroup has one token or eight and a part of their heads: it forms the
// angles of its tokens once (in fp64, which holds pos * inv_freq to 53 bits: all
// of them for positions below 2^29, and what is lost of others is far below a
// bf16's step), keeps them in LDS, and turns every head with them.  A lane has two pieces of eight values, so
// that both sides of a pair and what the cache holds together are one lane's.
// Each value is read once and written once.  Bound by memory where there are many
// rows (4096 of 32 + 8 heads of 128, fp32: 30 us, 5.1 TB/s; bf16 26 us, 4.1 TB/s), by
// the launch and a few latencies where there are few (3.5 us).  Over 8 bits the fp64
// turns and codes make it 36 us (from bf16 rows, 2.5 TB/s).
//
// Eight tokens whose slots are a run (a prompt's; the tiles begin where the first
// row's run of eight does) have their values exchanged through LDS and stored
// sixteen bytes at a time; others' values go to their places one by one.
//
// bf16 values are rounded from fp32.  8-bit codes are formed in fp64 from the
// turned fp64 values: a code next to a rounding border depends on nothing that
// the formula does not say.
//
// Of rows with one slot the last is stored: each workgroup looks its tokens'
// slots up among the later rows, so that no two workgroups write one place.
#include <type_traits>

#include "kv_args.h"

namespace q4nx {

namespace {

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u32x4u __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

template <typename T>
struct Turn { T c, s; };

// To fp32: the angle less whole turns in fp64 (2 pi in two parts, so that nothing of a turn's digits is lost), then
// the fp32 functions: what is left, below pi, is off by 2^-23 at most, a bf16's half step by 2^-8 of the value.
__device__ __forceinline__ void turn_of(double angle, Turn<float>& t) {
  const double turns = rint(angle * 0.15915494309189535);
  const double rest = fma(-turns, 2.4492935982947064e-16, fma(-turns, 6.283185307179586, angle));
  sincosf((float)rest, &t.s, &t.c);
}
__device__ __forceinline__ void turn_of(double angle, Turn<double>& t) { sincos(angle, &t.s, &t.c); }

__device__ __forceinline__ float mul_add(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ double mul_add(double a, double b, double c) { return fma(a, b, c); }

}  // namespace

// I8: the cache's type; T: what values are turned in; TM: tokens of a workgroup.  (All eight waves a SIMD for many rows
// of bf16: 16384 rows 122 us for 133 with seven; 8 bits need their registers, 51 for 35 us at 4096 rows with fewer.)
template <int D, bool I8, typename T, int TM>
__global__ __launch_bounds__(256, !I8 && TM == 8 ? 8 : 1) void k_kv_append(AppendArgs a) {
  constexpr int L = D / 16;            // lanes of a head: 4, 8 or 16
  constexpr int kItems = 256 / L;      // heads at a time
  typedef typename std::conditional<I8, uint8_t, uint16_t>::type Elem;
  extern __shared__ __align__(16) uint8_t lds[];
  Turn<T>* turn = reinterpret_cast<Turn<T>*>(lds);   // [TM][rot / 2]
  __shared__ int s_slot[TM], s_dead[TM];
  __shared__ __align__(16) Elem s_v[TM == 8 ? kItems : 1][TM == 8 ? D + 8 : 1];
  const int tid = threadIdx.x;
  const int off = TM == 8 ? max(a.slots[0], 0) & 7 : 0;
  const int m0 = max((int)blockIdx.x * TM - off, 0), rows = min((int)(blockIdx.x + 1) * TM - off, a.M) - m0;
  if (rows <= 0) return;
  const int half = a.inv_freq ? a.rot / 2 : 0;
  for (int i = tid; i < rows * half; i += 256) {
    const int t = i / half, p = i - t * half;
    turn_of((double)a.pos[m0 + t] * (double)a.inv_freq[p], turn[i]);
  }
  if (tid < rows) {
    int slot = a.slots[m0 + tid];
    if (slot < -1 || slot >= (int64_t)a.c.n_pages << a.c.page_shift) {
      if (blockIdx.y == 0) set_flag(a.flags, kFlagIndex);
      slot = -1;
    }
    s_slot[tid] = slot;
    s_dead[tid] = 0;
  }
  __syncthreads();
  // a later row with one of these slots; most are out of their range
  int lo = 0x7FFFFFFF, hi = -1;
#pragma unroll
  for (int t = 0; t < TM; ++t)
    if (t < rows && s_slot[t] >= 0) {
      lo = min(lo, s_slot[t]);
      hi = max(hi, s_slot[t]);
    }
  for (int j = m0 + 1 + tid; j < a.M; j += 256) {
    const int slot = a.slots[j];
    if (slot >= lo && slot <= hi)
      for (int t = 0; t < rows; ++t)
        if (slot == s_slot[t] && m0 + t < j) s_dead[t] = 1;   // every writer writes the same
  }
  __syncthreads();

  // A head's 16 values of a lane: piece e0 of eight and piece e1.
  const int qh = a.q.p ? a.q.heads : 0, KH = a.c.heads;
  auto place = [&](int t) { return kv_page(a.c, s_slot[t] >> a.c.page_shift, 0); };
  // 8 bits: a head's scale over its lanes, and the lane's codes
  auto codes_of = [&](const T (&y)[16], float& scale, uint32_t (&w)[4]) {
    T top = 0;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      top = fmax(top, fabs(y[i]));
      nan |= y[i] != y[i];
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
      top = fmax(top, __shfl_xor(top, o));
      nan |= __shfl_xor((int)nan, o) != 0;
    }
    scale = nan ? __builtin_nanf("") : (float)(top / (T)127);
    const bool plain = scale > 0.f && scale <= __FLT_MAX__;
    // A product with the reciprocal is the quotient but for its last bits of 53: it rounds to the same code unless it
    // lies next to a half step, where the quotient itself decides.
    const T inv = plain ? (T)1 / (T)scale : 0;
    bool border = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = 0u;
    auto put = [&](int i, T quotient) {
      const int code = plain ? (int)fmin(fmax(rint(quotient), (T)-127), (T)127) : 0;
      w[i >> 2] |= (uint32_t)(code & 255) << (8 * (i & 3));
    };
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const T quotient = y[i] * inv;
      border |= fabs(quotient - rint(quotient)) > (T)0.499999999;
      put(i, quotient);
    }
    if (border) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = 0u;
#pragma unroll
      for (int i = 0; i < 16; ++i) put(i, y[i] / (T)scale);
    }
  };
  auto load16 = [&](const HeadRows& src, int64_t row, int e0, int e1, T (&y)[16]) {
    if (src.bf16) {
      const uint16_t* p = static_cast<const uint16_t*>(src.p) + row;
      const u32x4u w[2] = {*reinterpret_cast<const u32x4u*>(p + 8 * e0), *reinterpret_cast<const u32x4u*>(p + 8 * e1)};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[2 * i] = bf16lo(w[i >> 2][i & 3]);
        y[2 * i + 1] = bf16hi(w[i >> 2][i & 3]);
      }
    } else {
      const float* p = static_cast<const float*>(src.p) + row;
      f32x4u x[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) x[n] = *reinterpret_cast<const f32x4u*>(p + 8 * (n < 2 ? e0 : e1) + 4 * (n & 1));
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = x[i >> 2][i & 3];
    }
  };

  // q and k.  8 bits: a head's lanes side by side, to find its largest value; else eight tokens side by side, whose
  // pieces lie together in the cache.
  for (int it = blockIdx.y * 256 + tid; it < rows * (qh + KH) * L; it += gridDim.y * 256) {
    int l, t, h;
    if (I8 || TM == 1) {
      l = it % L;
      const int u = it / L;
      t = u % rows;
      h = u / rows;
    } else {
      t = it % rows;
      const int u = it / rows;
      l = u % L;
      h = u / L;
    }
    const int m = m0 + t;
    const bool is_q = h < qh;
    const HeadRows& src = is_q ? a.q : a.k;
    const int head = is_q ? h : h - qh;
    const bool kept = s_slot[t] >= 0 && !s_dead[t];
    int e0 = 2 * l, e1 = 2 * l + 1;
    if (!a.interleaved && 8 * l < half) {
      e0 = l;
      e1 = l + half / 8;
    }
    T y[16];
    load16(src, (int64_t)m * src.ld + (int64_t)head * D, e0, e1, y);
    if (!a.interleaved) {
      if (8 * l < half) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const Turn<T> w = turn[t * half + 8 * l + i];
          const T p = y[i], r = y[8 + i];
          y[i] = mul_add(p, w.c, -r * w.s);
          y[8 + i] = mul_add(r, w.c, p * w.s);
        }
      }
    } else if (8 * l < half) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const Turn<T> w = turn[t * half + 8 * l + i];
        const T p = y[2 * i], r = y[2 * i + 1];
        y[2 * i] = mul_add(p, w.c, -r * w.s);
        y[2 * i + 1] = mul_add(r, w.c, p * w.s);
      }
    }
    u32x4 w[2];
#pragma unroll
    for (int n = 0; n < 8; ++n) w[n >> 2][n & 3] = bf16_pair((float)y[2 * n], (float)y[2 * n + 1]);
    if (is_q) {
      uint16_t* o = a.q_out + ((size_t)m * qh + head) * D;
      *reinterpret_cast<u32x4*>(o + 8 * e0) = w[0];
      *reinterpret_cast<u32x4*>(o + 8 * e1) = w[1];
    }
    if constexpr (I8) {
      float scale;
      uint32_t c[4];
      codes_of(y, scale, c);   // of q's heads too: the lanes stay together
      if (!is_q && kept) {
        const int tok = s_slot[t] & ((1 << a.c.page_shift) - 1);
        uint8_t* o = static_cast<uint8_t*>(a.c.k) + place(t) + ((size_t)head << a.c.page_shift) * D;
        *reinterpret_cast<u32x2*>(o + k_place(D, tok, 8 * e0)) = u32x2{c[0], c[1]};
        *reinterpret_cast<u32x2*>(o + k_place(D, tok, 8 * e1)) = u32x2{c[2], c[3]};
        if (l == 0) a.c.ks[place(t) / D + ((size_t)head << a.c.page_shift) + tok] = scale;
      }
    } else if (!is_q && kept) {
      const int tok = s_slot[t] & ((1 << a.c.page_shift) - 1);
      uint16_t* o = static_cast<uint16_t*>(a.c.k) + place(t) + ((size_t)head << a.c.page_shift) * D;
      *reinterpret_cast<u32x4*>(o + k_place(D, tok, 8 * e0)) = w[0];
      *reinterpret_cast<u32x4*>(o + k_place(D, tok, 8 * e1)) = w[1];
    }
  }

  // v: a head's lanes side by side, then its tokens
  bool run = TM == 8 && rows == 8 && s_slot[0] >= 0 && (s_slot[0] & 7) == 0;
  if constexpr (TM == 8)
    for (int t = 0; t < 8 && run; ++t) run = s_slot[t] == s_slot[0] + t && !s_dead[t];
  const int items = rows * KH * L;
  for (int base = blockIdx.y * 256; base < items; base += gridDim.y * 256) {
    const int it = base + tid, l = it % L, u = it / L, t = u % rows, head = u / rows;
    const bool mine = it < items;
    T y[16];
    if (mine) load16(a.v, (int64_t)(m0 + t) * a.v.ld + (int64_t)head * D, 2 * l, 2 * l + 1, y);
    else
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = 0;
    const bool kept = mine && s_slot[t] >= 0 && !s_dead[t];
    const int tok = kept ? s_slot[t] & ((1 << a.c.page_shift) - 1) : 0;
    Elem e[16];
    if constexpr (I8) {
      float scale;
      uint32_t c[4];
      codes_of(y, scale, c);
#pragma unroll
      for (int i = 0; i < 16; ++i) e[i] = (uint8_t)(c[i >> 2] >> (8 * (i & 3)));
      if (kept && l == 0) a.c.vs[place(t) / D + ((size_t)head << a.c.page_shift) + tok] = scale;
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) e[i] = __builtin_bit_cast(uint16_t, (__bf16)(float)y[i]);
    }
    if (TM == 8 && run) {   // the same in the whole workgroup
#pragma unroll
      for (int i = 0; i < 16; ++i) s_v[tid / L][16 * l + i] = e[i];
      __syncthreads();
      // 8 tokens of a dimension, 256 / L / 8 heads at a time
      const int head0 = base / L / 8;
      for (int n = tid; n < kItems / 8 * D; n += 256) {
        const int hl = n / D, d = n % D;
        if (head0 + hl < KH) {
          const size_t at = place(0) + ((size_t)(head0 + hl) << a.c.page_shift) * D +
                            v_place(D, s_slot[0] & ((1 << a.c.page_shift) - 1), d);
          Elem x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = s_v[8 * hl + i][d];
          if constexpr (I8) {
            *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.c.v) + at) = __builtin_bit_cast(u32x2, x);
          } else {
            *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.c.v) + at) = __builtin_bit_cast(u32x4, x);
          }
        }
      }
      __syncthreads();
    } else if (kept) {
      Elem* o = static_cast<Elem*>(a.c.v) + place(t) + ((size_t)head << a.c.page_shift) * D;
#pragma unroll
      for (int i = 0; i < 16; ++i) o[v_place(D, tok, 16 * l + i)] = e[i];
    }
  }
}

hipError_t launch_kv_append(const AppendArgs& a, int head_parts, hipStream_t s) {
  const dim3 grid(append_tiles(a), head_parts);
  const bool i8 = a.c.ks != nullptr;
  const size_t lds = a.inv_freq ? (size_t)a.tile * (a.rot / 2) * (i8 ? 16 : 8) : 0;
#define Q4NX_APPEND(D, I8, T)                                                                                            \
  if (a.tile == kAppendTile) hipLaunchKernelGGL((k_kv_append<D, I8, T, kAppendTile>), grid, dim3(256), lds, s, a);       \
  else hipLaunchKernelGGL((k_kv_append<D, I8, T, 1>), grid, dim3(256), lds, s, a)
#define Q4NX_APPEND_D(D)                    \
  if (i8) { Q4NX_APPEND(D, true, double); } \
  else { Q4NX_APPEND(D, false, float); }
  if (a.c.dim == 64) { Q4NX_APPEND_D(64) }
  else if (a.c.dim == 128) { Q4NX_APPEND_D(128) }
  else { Q4NX_APPEND_D(256) }
#undef Q4NX_APPEND_D
#undef Q4NX_APPEND
  return hipGetLastError();
}

}  // namespace q4nx
