// Rotation by position and append to the paged cache.
//
//   t = pos * inv_freq[i];  (a, b) -> (a cos t - b sin t, b cos t + a sin t)
//
// A workgroup has a few tokens and a part of their heads: it forms the angles
// of its tokens once (fp64: pos * inv_freq is exact there, and the sine and
// cosine reduce it without losing a far position's digits), keeps them in LDS,
// and turns every head with them.  D/8 neighbouring lanes hold a head, eight
// values each, so that an 8-bit head's largest value is a few lane exchanges
// away.  Each value is read once and written once.
//
// bf16 values are rounded from fp32.  8-bit codes are formed in fp64 from the
// turned fp64 values: a code next to a rounding border depends on nothing that
// the formula does not say.
//
// Of rows with one slot the last is stored: each workgroup looks its tokens'
// slots up among the later rows, so that no two workgroups write one place.
#include "kv_args.h"

namespace q4nx {

namespace {

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u32x2u __attribute__((ext_vector_type(2), aligned(2)));

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// Four neighbouring values of a row.
__device__ __forceinline__ f32x4 load4(const HeadRows& h, int64_t at) {
  if (h.bf16) {
    const u32x2u w = *reinterpret_cast<const u32x2u*>(static_cast<const uint16_t*>(h.p) + at);
    return f32x4{bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y)};
  }
  return *reinterpret_cast<const f32x4u*>(static_cast<const float*>(h.p) + at);
}

template <typename T>
struct Turn { T c, s; };

__device__ __forceinline__ void turn_of(double angle, Turn<float>& t) {
  double s, c;
  sincos(angle, &s, &c);
  t = {(float)c, (float)s};
}
__device__ __forceinline__ void turn_of(double angle, Turn<double>& t) { sincos(angle, &t.s, &t.c); }

__device__ __forceinline__ float mul_add(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ double mul_add(double a, double b, double c) { return fma(a, b, c); }

}  // namespace

// I8: the cache's type; T: what values are turned in.
template <int D, bool I8, typename T>
__global__ __launch_bounds__(256) void k_kv_append(AppendArgs a) {
  constexpr int L = D / 8;             // lanes of a head
  constexpr int kItems = 256 / L;      // heads at a time
  extern __shared__ __align__(16) uint8_t lds[];
  Turn<T>* turn = reinterpret_cast<Turn<T>*>(lds);   // [tile][rot / 2]
  __shared__ int s_slot[kAppendTile];
  __shared__ int s_dead[kAppendTile];
  const int tid = threadIdx.x, m0 = blockIdx.x * a.tile, rows = min(a.tile, a.M - m0);
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
  for (int j = m0 + 1 + tid; j < a.M; j += 256) {
    const int slot = a.slots[j];
    for (int t = 0; t < rows; ++t)
      if (slot == s_slot[t] && m0 + t < j) s_dead[t] = 1;   // every writer writes the same
  }
  __syncthreads();

  const int qh = a.q.p ? a.q.heads : 0, heads = qh + 2 * a.c.heads;
  const int l = tid % L;
  for (int it = blockIdx.y * kItems + tid / L; it < rows * heads; it += gridDim.y * kItems) {
    const int t = it / heads, h = it - t * heads, m = m0 + t;
    const bool is_q = h < qh, is_v = h >= qh + a.c.heads;
    const HeadRows& src = is_q ? a.q : is_v ? a.v : a.k;
    const int head = is_q ? h : is_v ? h - qh - a.c.heads : h - qh;
    if (!is_q && (s_slot[t] < 0 || s_dead[t])) continue;   // the same in a head's lanes
    const int64_t row = (int64_t)m * src.ld + (int64_t)head * D;
    // the lane's values: four from d0 and four from d1
    const bool turns = !is_v && 4 * l < half;
    const int d0 = turns && !a.interleaved ? 4 * l : 8 * l;
    const int d1 = turns && !a.interleaved ? half + 4 * l : 8 * l + 4;
    const f32x4 x0 = load4(src, row + d0), x1 = load4(src, row + d1);
    T y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = x0[i];
      y[4 + i] = x1[i];
    }
    if (turns) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Turn<T> w = turn[t * half + 4 * l + i];
        if (a.interleaved) {
          const T p = y[2 * i], r = y[2 * i + 1];
          y[2 * i] = mul_add(p, w.c, -r * w.s);
          y[2 * i + 1] = mul_add(r, w.c, p * w.s);
        } else {
          const T p = y[i], r = y[4 + i];
          y[i] = mul_add(p, w.c, -r * w.s);
          y[4 + i] = mul_add(r, w.c, p * w.s);
        }
      }
    }
    if (is_q) {
      uint16_t* o = a.q_out + ((size_t)m * qh + head) * D;
      *reinterpret_cast<u32x2*>(o + d0) = u32x2{bf16_pair((float)y[0], (float)y[1]), bf16_pair((float)y[2], (float)y[3])};
      *reinterpret_cast<u32x2*>(o + d1) = u32x2{bf16_pair((float)y[4], (float)y[5]), bf16_pair((float)y[6], (float)y[7])};
      continue;
    }
    const int page = s_slot[t] >> a.c.page_shift, tok = s_slot[t] & ((1 << a.c.page_shift) - 1);
    const size_t base = kv_page(a.c, page, head);
    if constexpr (I8) {
      T top = 0;
      bool nan = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        top = fmax(top, fabs(y[i]));
        nan |= y[i] != y[i];
      }
#pragma unroll
      for (int off = 1; off < L; off <<= 1) {
        top = fmax(top, __shfl_xor(top, off));
        nan |= __shfl_xor((int)nan, off) != 0;
      }
      const float scale = nan ? __builtin_nanf("") : (float)(top / (T)127);
      const bool plain = scale > 0.f && scale <= __FLT_MAX__;
      uint32_t w[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int code = plain ? (int)fmin(fmax(rint(y[i] / (T)scale), (T)-127), (T)127) : 0;
        w[i >> 2] |= (uint32_t)(code & 255) << (8 * (i & 3));
      }
      if (is_v) {
        uint8_t* o = static_cast<uint8_t*>(a.c.v) + base;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[v_place(D, tok, 8 * l + i)] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
      } else {
        uint8_t* o = static_cast<uint8_t*>(a.c.k) + base;
        *reinterpret_cast<uint32_t*>(o + k_place(D, tok, d0)) = w[0];
        *reinterpret_cast<uint32_t*>(o + k_place(D, tok, d1)) = w[1];
      }
      if (l == 0) (is_v ? a.c.vs : a.c.ks)[(((size_t)page * a.c.heads + head) << a.c.page_shift) + tok] = scale;
    } else {
      const uint32_t w[4] = {bf16_pair((float)y[0], (float)y[1]), bf16_pair((float)y[2], (float)y[3]),
                             bf16_pair((float)y[4], (float)y[5]), bf16_pair((float)y[6], (float)y[7])};
      if (is_v) {
        uint16_t* o = static_cast<uint16_t*>(a.c.v) + base;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[v_place(D, tok, 8 * l + i)] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
      } else {
        uint16_t* o = static_cast<uint16_t*>(a.c.k) + base;
        *reinterpret_cast<u32x2*>(o + k_place(D, tok, d0)) = u32x2{w[0], w[1]};
        *reinterpret_cast<u32x2*>(o + k_place(D, tok, d1)) = u32x2{w[2], w[3]};
      }
    }
  }
}

hipError_t launch_kv_append(const AppendArgs& a, int head_parts, hipStream_t s) {
  const dim3 grid((a.M + a.tile - 1) / a.tile, head_parts);
  const bool i8 = a.c.ks != nullptr;
  const size_t lds = a.inv_freq ? (size_t)a.tile * (a.rot / 2) * (i8 ? 16 : 8) : 0;
#define Q4NX_APPEND(D)                                                                            \
  if (i8) hipLaunchKernelGGL((k_kv_append<D, true, double>), grid, dim3(256), lds, s, a);         \
  else hipLaunchKernelGGL((k_kv_append<D, false, float>), grid, dim3(256), lds, s, a)
  if (a.c.dim == 64) { Q4NX_APPEND(64); }
  else if (a.c.dim == 128) { Q4NX_APPEND(128); }
  else { Q4NX_APPEND(256); }
#undef Q4NX_APPEND
  return hipGetLastError();
}

}  // namespace q4nx
