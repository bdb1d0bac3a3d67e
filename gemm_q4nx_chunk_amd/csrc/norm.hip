// Residual addition and RMS norm between two projections.
//
//   s = y + r,  x = bf16(s * 1 / sqrt(mean(s^2) + eps) * w)
//
// y is what a GEMV wrote (fp32), r the residual stream (fp32), w the norm's
// bf16 weights (the q4nx model file of the NPU engine page, "From a GGUF",
// keeps its norms in bf16) and x the bf16 activations that the next GEMV,
// router or adapter reads.  One pass: a row's values stay in registers between
// the sum of squares and the scaling, so each input is read once and each
// output written once.  The sum of squares is fp32 in a fixed order (a
// thread's values in column order, an xor tree over the lanes, then the waves
// in order); each x is rounded once, from fp32, which is what the projections
// take.
//
// A row whose squares leave fp32 (their mean with eps overflows, or lies so low
// that a square below 2^-126 may count) is summed again from the registers,
// scaled by a power of two that puts the larger of its maximum and sqrt(eps)
// just below 1:
//   x = t / sqrt(mean(t^2) + 4^-e eps) * w,  t = 2^-e s.
// A square below 2^-126 counts for at most 2^-30 of a mean of 2^-96 and up, so
// that other rows, with any usual eps all that do not overflow, need no second
// sum.
//
// Bound by HBM for many rows and by two memory latencies (load, reduce, store)
// for few.
#include "q4nx_dev.h"

namespace q4nx {

namespace {

// Rows start at any multiple of 4 (fp32) or 2 bytes (bf16): D may be odd.
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u32x2u __attribute__((ext_vector_type(2), aligned(2)));

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

constexpr float kLowMean = 0x1p-96f;

// Sum (or maximum) of a value over the row's threads, in every one of them.
template <int WAVES, bool MAX>
__device__ __forceinline__ float over_row(float v, float* part, int wave, int lane) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    const float o = __shfl_xor(v, off);
    v = MAX ? fmaxf(v, o) : v + o;
  }
  if constexpr (WAVES > 1) {
    if (lane == 0) part[wave] = v;
    __syncthreads();
    v = 0.f;   // maxima are of magnitudes
#pragma unroll
    for (int i = 0; i < WAVES; ++i) v = MAX ? fmaxf(v, part[i]) : v + part[i];
  }
  return v;
}

// Sum of the squares of pre * s, pre a power of two.
template <int NV>
__device__ __forceinline__ float squares(const f32x4 (&s)[NV], float pre) {
  float sum = 0.f;
#pragma unroll
  for (int g = 0; g < NV; ++g)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = fmaf(pre * s[g][i], pre * s[g][i], sum);
  return sum;
}

}  // namespace

// WAVES waves share a row (one workgroup), or, for WAVES == 0, each of the
// workgroup's four waves has a row of its own.  A thread holds NV groups of
// four neighbouring columns, group g at column 4 * (g * threads + thread).
template <int WAVES, int NV>
__global__ __launch_bounds__(WAVES ? 64 * WAVES : 256) void k_add_rmsnorm(
    const float* y, const float* r, const uint16_t* __restrict__ w, int M, int D, float eps, float* r_out,
    uint16_t* x) {
  constexpr int kThreads = WAVES ? 64 * WAVES : 64;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t = WAVES ? threadIdx.x : lane;
  const int m = WAVES ? blockIdx.x : blockIdx.x * 4 + wave;
  if (m >= M) return;   // whole waves, and only where no barrier follows (WAVES == 0)
  const size_t row = (size_t)m * D;
  f32x4 s[NV];
  u32x2 wv[NV];
#pragma unroll
  for (int g = 0; g < NV; ++g) {
    const int c = 4 * (g * kThreads + t);
    s[g] = f32x4{0.f, 0.f, 0.f, 0.f};
    wv[g] = u32x2{0u, 0u};
    if (c + 3 < D) {
      s[g] = *reinterpret_cast<const f32x4u*>(r + row + c);
      wv[g] = *reinterpret_cast<const u32x2u*>(w + c);
      if (y) s[g] += *reinterpret_cast<const f32x4u*>(y + row + c);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c + i < D) {
          s[g][i] = r[row + c + i] + (y ? y[row + c + i] : 0.f);
          wv[g][i >> 1] |= (uint32_t)w[c + i] << (16 * (i & 1));
        }
    }
  }
  __shared__ float part[WAVES > 1 ? WAVES : 1];
  const float mean = over_row<WAVES, false>(squares(s, 1.f), part, wave, lane) / (float)D + eps;
  float inv = 1.f / sqrtf(mean);
  auto write = [&](float pre) {
#pragma unroll
    for (int g = 0; g < NV; ++g) {
      const int c = 4 * (g * kThreads + t);
      const f32x4 v = s[g];
      const u32x2 o = {bf16_pair(v[0] * pre * inv * bf16lo(wv[g].x), v[1] * pre * inv * bf16hi(wv[g].x)),
                       bf16_pair(v[2] * pre * inv * bf16lo(wv[g].y), v[3] * pre * inv * bf16hi(wv[g].y))};
      if (c + 3 < D) {
        if (r_out) *reinterpret_cast<f32x4u*>(r_out + row + c) = v;
        *reinterpret_cast<u32x2u*>(x + row + c) = o;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + i < D) {
            if (r_out) r_out[row + c + i] = v[i];
            x[row + c + i] = (uint16_t)(o[i >> 1] >> (16 * (i & 1)));
          }
      }
    }
  };
  if (__builtin_expect(!(mean >= kLowMean && mean <= __FLT_MAX__), 0)) {   // the same in all of the row's threads
    if constexpr (WAVES > 1) __syncthreads();                               // part is read above
    float top = 0.f, pre = 1.f;                                             // pre: 2^-e
#pragma unroll
    for (int g = 0; g < NV; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(s[g][i]));
    top = over_row<WAVES, true>(top, part, wave, lane);
    // rows of an infinity, of a NaN (the mean is one) and of zeros stay with what they have
    if (top > 0.f && top <= __FLT_MAX__ && mean == mean) {
      // 2^126 at most, which takes 2^-149 to 2^-23
      pre = ldexpf(1.f, -max(__builtin_amdgcn_frexp_expf(fmaxf(top, sqrtf(eps))), -126));
      if constexpr (WAVES > 1) __syncthreads();
      inv = 1.f / sqrtf(over_row<WAVES, false>(squares(s, pre), part, wave, lane) / (float)D + eps * pre * pre);
    }
    write(pre);
    return;
  }
  write(1.f);
}

hipError_t launch_add_rmsnorm(const float* y, const float* r, const uint16_t* w, int M, int D, float eps,
                              float* r_out, uint16_t* x, hipStream_t s) {
#define Q4NX_NORM(WAVES, NV)                                                                                  \
  hipLaunchKernelGGL((k_add_rmsnorm<WAVES, NV>), dim3(WAVES ? M : (M + 3) / 4), dim3(WAVES ? 64 * WAVES : 256), \
                     0, s, y, r, w, M, D, eps, r_out, x)
  if (D <= 256) Q4NX_NORM(0, 1);
  else if (D <= 512) Q4NX_NORM(0, 2);
  else if (D <= 1024) Q4NX_NORM(4, 1);
  else if (D <= 2048) Q4NX_NORM(4, 2);
  else if (D <= 4096) Q4NX_NORM(4, 4);
  else if (D <= 8192) Q4NX_NORM(8, 4);
  else if (D <= 16384) Q4NX_NORM(16, 4);
  else Q4NX_NORM(16, 8);
#undef Q4NX_NORM
  return hipGetLastError();
}

}  // namespace q4nx
