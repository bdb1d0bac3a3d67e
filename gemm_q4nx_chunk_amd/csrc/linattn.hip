// Linear attention with a decay for each head.
//
//   S_t = exp(d_t) S_{t-1} + k_t v_t^T,   out_t = scale q_t^T S_t
#include <algorithm>

#include "kv_args.h"

namespace q4nx {

namespace {

struct LinearSeq {
  int32_t row0, rows;
  int32_t slot;    // -1: none
  bool fresh;      // begins with zeros
};

// Sequence s of the call.  Starts that fall count as the largest before them; a
// slot that an earlier sequence with rows has is none.  All of the workgroup's
// threads call it; `mem` is LDS of their own.
__device__ inline LinearSeq linear_seq(const LinearArgs& a, int s, int32_t* mem, bool flags) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (tid == 0) {
    mem[0] = 0;   // the largest start up to s
    mem[1] = 0;   // and up to s + 1
    mem[2] = 0;   // the slot is taken
  }
  __syncthreads();
  int up = 0;
  for (int e = tid; e <= s; e += blockDim.x) {
    const int raw = a.q_start[e];
    up = max(up, min(max(raw, 0), a.M));
  }
  if (up) atomicMax(&mem[0], up);
  __syncthreads();
  const int row0 = mem[0], raw1 = a.q_start[s + 1], row1 = max(row0, min(max(raw1, 0), a.M));
  const int raw0 = a.q_start[s];
  const int raw_slot = a.slots[s];
  bool bad = raw_slot < -1 || raw_slot >= a.n_slots;
  if (raw_slot >= 0) {
    // an earlier one with rows: its start rises to the next one's
    for (int e = tid; e < s; e += blockDim.x)
      if (a.slots[e] == raw_slot) {
        int before = 0;
        for (int i = 0; i <= e; ++i) before = max(before, min(max(a.q_start[i], 0), a.M));
        if (min(max(a.q_start[e + 1], 0), a.M) > before) mem[2] = 1;
      }
  }
  __syncthreads();
  bad |= mem[2] != 0;
  LinearSeq x;
  x.row0 = row0;
  x.rows = row1 - row0;
  x.slot = bad ? -1 : raw_slot;
  x.fresh = x.slot < 0 || (a.fresh && a.fresh[s]);
  if (flags && tid == 0) {
    if (bad && x.rows) set_flag(a.flags, kFlagIndex);
    if (raw0 != row0 || raw1 != row1) set_flag(a.flags, kFlagRows);
  }
  return x;
}

// exp of a decay; one above 0 or NaN counts as 0.
__device__ __forceinline__ float decay_of(const LinearArgs& a, int64_t row, int h, bool& bad) {
  const float d = a.decay[row * a.decay_ld + h];
  if (d <= 0.f) return d;
  bad = true;
  return 0.f;
}

}  // namespace

// The recurrence, row by row: CW columns of a head's state stay in a
// workgroup's registers (a thread has RP lines of four columns), so that for
// one row the state is read once and written once.  Bound by memory.
template <int DK, int DV, int CW>
__global__ __launch_bounds__(256) void k_linear_rows(LinearArgs a) {
  constexpr int LC = CW / 4, RG = 256 / LC, RP = DK / RG;
  __shared__ int32_t s_seq[4];
  __shared__ float s_q[DK], s_k[DK];
  __shared__ f32x4 s_o[RG][LC];
  const int tid = threadIdx.x, lc = tid % LC, rg = tid / LC;
  constexpr int kParts = DV / CW;
  const int part = blockIdx.x % kParts, h = blockIdx.x / kParts, sq = blockIdx.y;
  const LinearSeq x = linear_seq(a, sq, s_seq, blockIdx.x == 0);
  if (x.rows == 0) return;
  const int kh = h / (a.v_heads / a.k_heads), col = part * CW + 4 * lc;
  const size_t at = ((size_t)max(x.slot, 0) * a.v_heads + h) * DK * DV + (size_t)rg * RP * DV + col;
  f32x4 S[RP];
#pragma unroll
  for (int i = 0; i < RP; ++i)
    S[i] = x.fresh ? f32x4{0.f, 0.f, 0.f, 0.f} : *reinterpret_cast<const f32x4*>(a.state + at + (size_t)i * DV);
  bool bad = false;
  for (int t = 0; t < x.rows; ++t) {
    const int64_t row = x.row0 + t;
    if (tid < DK) {
      s_q[tid] = bf16lo(a.q[row * a.q_ld + kh * DK + tid]) * a.scale;
      s_k[tid] = bf16lo(a.k[row * a.k_ld + kh * DK + tid]);
    }
    const u32x2 vw = *reinterpret_cast<const u32x2*>(a.v + row * a.v_ld + h * DV + col);
    const f32x4 v = {bf16lo(vw.x), bf16hi(vw.x), bf16lo(vw.y), bf16hi(vw.y)};
    const float f = expf(decay_of(a, row, h, bad));
    __syncthreads();
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < RP; ++i) {
      const float kk = s_k[rg * RP + i], qq = s_q[rg * RP + i];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        // a state that is forgotten is gone, whatever it was
        S[i][n] = fmaf(kk, v[n], f == 0.f ? 0.f : f * S[i][n]);
        o[n] = fmaf(qq, S[i][n], o[n]);
      }
    }
    s_o[rg][lc] = o;
    __syncthreads();
    if (tid < CW) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < RG; ++w) sum += s_o[w][tid >> 2][tid & 3];
      a.out[((size_t)row * a.v_heads + h) * DV + part * CW + tid] = sum;
    }
    __syncthreads();
  }
  if (bad && tid == 0) set_flag(a.flags, kFlagDecay);
  if (x.slot >= 0)
#pragma unroll
    for (int i = 0; i < RP; ++i) *reinterpret_cast<f32x4*>(a.state_out + at + (size_t)i * DV) = S[i];
}

// ---------------------------------------------------------------------------
// prompts: chunks of 64 rows on the matrix cores
// ---------------------------------------------------------------------------
// With G_i the sum of a chunk's decays up to row i (fp64) and S the state before it:
//   out_i = scale (exp(G_i) q_i S + sum_{j <= i} exp(G_i - G_j) (q_i.k_j) v_j)
//   S' = exp(G_last) S + sum_j k_j (exp(G_last - G_j) v_j)^T
// Each wave has 32 columns of the state, all of its lines, in accumulators of
// 32 x 32; K's lines are dealt so that a lane's accumulators are eight
// neighbouring lines of its column, which is how the state enters q S as an
// operand.  q, k and v are exact in bf16; what meets them (the state, the
// weights of the rows, the decayed values) is cut into three bf16 parts that
// hold its 24 bits, so that no product loses to bf16.
//
// A long sequence is cut into segments: one launch forms each segment's own
// contribution to the state, a second carries the states over the segments, and
// a third runs the segments from their states.
namespace {

constexpr int kChunk = 64;

// bf16 parts of x: x = hi + mid + lo to 2^-24 (x below 2^127).
struct Parts { bf16x8 p[3]; };
__device__ __forceinline__ Parts parts_of(const float (&x)[8]) {
  Parts r;
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const __bf16 hi = (__bf16)x[n];
    const float r1 = x[n] - (float)hi;
    const __bf16 mid = (__bf16)r1;
    r.p[0][n] = hi;
    r.p[1][n] = mid;
    r.p[2][n] = (__bf16)(r1 - (float)mid);
  }
  return r;
}

// The line of a 32-line operand that lane c holds: accumulators 8 t + n of half
// h are then lines 16 t + 8 h + n.
__device__ __forceinline__ int dealt(int c) { return 16 * (c >> 4) + 8 * ((c >> 2) & 1) + 4 * ((c >> 3) & 1) + (c & 3); }

__device__ __forceinline__ bool huge(uint32_t bits) { return (bits & 0x7F800000u) >= 0x7F000000u; }
__device__ __forceinline__ bool nonfinite2(uint32_t w) {
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// Exclusive sums of the sequences' segments: first[s] for s in 0..n_seq, in LDS.
__device__ inline void linear_plan(const LinearArgs& a, int32_t* first, int32_t* start) {
  const int tid = threadIdx.x, lane = tid & 63;
  if (tid < 64) {   // one wave: 64 sequences at a time
    int up = 0, sum = 0;
    for (int b = 0; b <= a.n_seq; b += 64) {
      const int e = b + lane;
      int v = e <= a.n_seq ? min(max(a.q_start[e], 0), a.M) : 0;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(v, off);
        if (lane >= off) v = max(v, o);
      }
      v = max(v, up);
      if (e <= a.n_seq) start[e] = v;
      up = __shfl(v, 63);
    }
    for (int b = 0; b < a.n_seq; b += 64) {
      const int e = b + lane;
      const int segs = e < a.n_seq ? (start[e + 1] - start[e] + a.seg - 1) / a.seg : 0;
      int v = segs;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(v, off);
        if (lane >= off) v += o;
      }
      if (e < a.n_seq) first[e] = sum + v - segs;
      sum += __shfl(v, 63);
    }
    if (lane == 0) first[a.n_seq] = sum;
  }
  __syncthreads();
}

}  // namespace

template <int DK, int DV, bool OUT>
__global__ __launch_bounds__(2 * DV, 2) void k_linear_chunks(LinearArgs a) {
  constexpr int kThreads = 2 * DV, kWaves = DV / 32, NT = DK / 32;
  // elements: q [DK/8][64][8] | k likewise, then the rows' weights [3][8][64][8] | k^T [8][DK][8] | v^T [8][DV][8]
  constexpr int kQ = 0, kK = OUT ? kChunk * DK : 0, kA = OUT ? (kChunk * DK > 3 * kChunk * kChunk ? kChunk * DK : 3 * kChunk * kChunk) : 0;
  constexpr int kKT = kK + kA, kVT = kKT + kChunk * DK;
  extern __shared__ __align__(16) uint16_t lds[];
  __shared__ double s_G[kChunk];
  __shared__ float s_d[kChunk];
  __shared__ int32_t s_seq[4];
  __shared__ int s_odd[2];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, c = lane & 31, hh = lane >> 5;
  const int h = blockIdx.x % a.v_heads, item = blockIdx.x / a.v_heads, kh = h / (a.v_heads / a.k_heads);
  int seq, seg;
  {
    int32_t* first = reinterpret_cast<int32_t*>(lds);
    linear_plan(a, first, first + kAttnMaxSeq + 1);
    if (!OUT && blockIdx.x == 0)
      for (int e = tid; e <= a.n_seq; e += kThreads) a.plan[e] = first[e];
    if (item >= first[a.n_seq]) return;
    int count = 0;
    for (int b = 0; b < a.n_seq; b += 64) count += __popcll(__ballot(b + lane < a.n_seq && first[b + lane] <= item));
    seq = count - 1;
    seg = item - first[seq];
    if (!OUT && seg == first[seq + 1] - first[seq] - 1) return;   // what the last one adds, it adds itself
    __syncthreads();
  }
  const LinearSeq x = linear_seq(a, seq, s_seq, OUT && h == 0 && seg == 0);
  const int row0 = x.row0 + seg * a.seg, rows = min(a.seg, x.rows - seg * a.seg);
  const size_t state_size = (size_t)DK * DV;
  // the lane's column and first line of its accumulators
  const int col = 32 * wave + c, line0 = 8 * hh;
  f32x16 S[NT];
  {
    const float* from = nullptr;
    if (OUT) {
      if (seg > 0) from = a.seg_state + ((size_t)(item - 1) * a.v_heads + h) * state_size;
      else if (!x.fresh) from = a.state + ((size_t)x.slot * a.v_heads + h) * state_size;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int n = 0; n < 16; ++n) S[t][n] = from ? from[(size_t)(32 * t + 16 * (n >> 3) + line0 + (n & 7)) * DV + col] : 0.f;
  }
  auto state_odd = [&]() {
    bool odd = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int n = 0; n < 16; ++n) odd |= huge(__float_as_uint(S[t][n]));
    return odd;
  };
  double G_all = 0.0;
  bool bad = false;
  if (tid < 2) s_odd[tid] = 0;
  __syncthreads();
  for (int r0 = 0, turn = 0; r0 < rows; r0 += kChunk, turn ^= 1) {
    const int n_rows = min(kChunk, rows - r0);
    const int64_t g0 = row0 + r0;
    bool odd = state_odd();
    // operands to LDS; rows behind the last are zeros
    if constexpr (OUT) {
      for (int u = tid; u < kChunk * DK / 8; u += kThreads) {
        const int r = (u & 15) | ((u >> 6) / (DK / 32) << 4), ch = ((u >> 4) & 3) + 4 * ((u >> 6) % (DK / 32));
        u32x4 w = {0u, 0u, 0u, 0u}, y = w;
        if (r < n_rows) {
          w = *reinterpret_cast<const u32x4*>(a.q + (g0 + r) * a.q_ld + kh * DK + 8 * ch);
          y = *reinterpret_cast<const u32x4*>(a.k + (g0 + r) * a.k_ld + kh * DK + 8 * ch);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) odd |= nonfinite2(w[n]);
        *reinterpret_cast<u32x4*>(lds + kQ + (ch * kChunk + r) * 8) = w;
        *reinterpret_cast<u32x4*>(lds + kK + (ch * kChunk + r) * 8) = y;
      }
    }
    auto transpose = [&](const uint16_t* src, int64_t ld, int width, int at) {
      for (int u = tid; u < 8 * width / 2; u += kThreads) {
        const int d = 2 * (u % (width / 2)), r = 8 * (u / (width / 2));
        uint32_t w[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) w[n] = r + n < n_rows ? *reinterpret_cast<const uint32_t*>(src + (g0 + r + n) * ld + d) : 0u;
        u32x4 lo, hi;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          odd |= nonfinite2(w[2 * n]) || nonfinite2(w[2 * n + 1]);
          lo[n] = __builtin_amdgcn_perm(w[2 * n + 1], w[2 * n], 0x05040100u);
          hi[n] = __builtin_amdgcn_perm(w[2 * n + 1], w[2 * n], 0x07060302u);
        }
        uint16_t* to = lds + at + ((r >> 3) * width + d) * 8;
        *reinterpret_cast<u32x4*>(to) = lo;
        *reinterpret_cast<u32x4*>(to + 8) = hi;
      }
    };
    transpose(a.k + kh * DK, a.k_ld, DK, kKT);
    transpose(a.v + h * DV, a.v_ld, DV, kVT);
    if (wave == kWaves - 1) {
      const float d = lane < n_rows ? decay_of(a, g0 + lane, h, bad) : 0.f;
      s_d[lane] = d;
      double G = (double)fmaxf(d, -1e5f);   // exp of less is 0 in fp32, and sums of these stay exact to 2^-30
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const double o = __shfl_up(G, off);
        if (lane >= off) G += o;
      }
      s_G[lane] = G;
    }
    if (odd) s_odd[turn] = 1;
    __syncthreads();
    const bool slow = s_odd[turn] != 0;
    if (tid == 0) s_odd[turn ^ 1] = 0;
    const double G_last = s_G[kChunk - 1];
    G_all += G_last;
    if (slow) {
      // an infinity or NaN: row by row, so that it reaches what the recurrence lets it reach
      for (int t = 0; t < n_rows; ++t) {
        const float f = expf(s_d[t]);
        const float v = bf16lo(lds[kVT + ((t >> 3) * DV + col) * 8 + (t & 7)]);
        float o = 0.f;
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            const int line = 32 * b + 16 * (n >> 3) + line0 + (n & 7);
            const float kk = bf16lo(lds[kKT + ((t >> 3) * DK + line) * 8 + (t & 7)]);
            S[b][n] = fmaf(kk, v, f == 0.f ? 0.f : f * S[b][n]);
            if constexpr (OUT) o = fmaf(bf16lo(lds[kQ + ((line >> 3) * kChunk + t) * 8 + (line & 7)]), S[b][n], o);
          }
        if constexpr (OUT) {
          o += __shfl_xor(o, 32);
          if (hh == 0) a.out[((size_t)(g0 + t) * a.v_heads + h) * DV + col] = o * a.scale;
        }
      }
      __syncthreads();
      continue;
    }
    if constexpr (OUT) {
      // the rows' weights: tiles (0,0), (1,0) and (1,1) of (row tile, key tile), transposed: a lane has one row
      constexpr int kMine = (3 + kWaves - 1) / kWaves;
      f32x16 w[kMine];
#pragma unroll
      for (int m = 0; m < kMine; ++m) {
        const int tile = wave + m * kWaves, ti = tile > 0, tj = tile > 1;
        if (tile < 3) {
#pragma unroll
          for (int n = 0; n < 16; ++n) w[m][n] = 0.f;
#pragma unroll
          for (int s = 0; s < DK / 16; ++s)
            w[m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                *reinterpret_cast<const bf16x8*>(lds + kK + ((2 * s + hh) * kChunk + 32 * tj + dealt(c)) * 8),
                *reinterpret_cast<const bf16x8*>(lds + kQ + ((2 * s + hh) * kChunk + 32 * ti + c) * 8), w[m], 0, 0, 0);
          const int row = 32 * ti + c;
          const double Gi = s_G[row];
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            const int j = 32 * tj + 16 * (n >> 3) + line0 + (n & 7);
            w[m][n] = j <= row ? w[m][n] * expf((float)(Gi - s_G[j])) : 0.f;
          }
        }
      }
      __syncthreads();   // k's rows are done with
#pragma unroll
      for (int m = 0; m < kMine; ++m) {
        const int tile = wave + m * kWaves, ti = tile > 0, tj = tile > 1;
        if (tile < 3)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            float f[8];
#pragma unroll
            for (int n = 0; n < 8; ++n) f[n] = w[m][8 * t + n];
            const Parts q3 = parts_of(f);
#pragma unroll
            for (int i = 0; i < 3; ++i)
              *reinterpret_cast<bf16x8*>(lds + kK + i * kChunk * kChunk + ((4 * tj + 2 * t + hh) * kChunk + 32 * ti + c) * 8) = q3.p[i];
          }
      }
      // q S, scaled by each row's decay since the chunk's beginning
      f32x16 o[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < 16; ++n) o[i][n] = 0.f;
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float f[8];
#pragma unroll
          for (int n = 0; n < 8; ++n) f[n] = S[b][8 * t + n];
          const Parts s3 = parts_of(f);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const bf16x8 q8 = *reinterpret_cast<const bf16x8*>(lds + kQ + ((4 * b + 2 * t + hh) * kChunk + 32 * i + c) * 8);
#pragma unroll
            for (int k = 2; k >= 0; --k) o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q8, s3.p[k], o[i], 0, 0, 0);
          }
        }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < 16; ++n) o[i][n] *= expf((float)s_G[32 * i + 8 * (n >> 2) + 4 * hh + (n & 3)]);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int s = 0; s < 2 + 2 * i; ++s) {
          const bf16x8 v8 = *reinterpret_cast<const bf16x8*>(lds + kVT + ((2 * s + hh) * DV + col) * 8);
#pragma unroll
          for (int k = 2; k >= 0; --k)
            o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                *reinterpret_cast<const bf16x8*>(lds + kK + k * kChunk * kChunk + ((2 * s + hh) * kChunk + 32 * i + c) * 8), v8, o[i], 0, 0, 0);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          const int row = 32 * i + 8 * (n >> 2) + 4 * hh + (n & 3);
          if (row < n_rows) a.out[((size_t)(g0 + row) * a.v_heads + h) * DV + col] = o[i][n] * a.scale;
        }
    }
    // the state
    const float f_all = expf((float)G_last);
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
      for (int n = 0; n < 16; ++n) S[b][n] *= f_all;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const bf16x8 v8 = *reinterpret_cast<const bf16x8*>(lds + kVT + ((2 * s + hh) * DV + col) * 8);
      float f[8];
#pragma unroll
      for (int n = 0; n < 8; ++n) f[n] = (float)v8[n] * expf((float)(G_last - s_G[16 * s + 8 * hh + n]));
      const Parts v3 = parts_of(f);
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        const bf16x8 k8 = *reinterpret_cast<const bf16x8*>(lds + kKT + ((2 * s + hh) * DK + 32 * b + dealt(c)) * 8);
#pragma unroll
        for (int k = 2; k >= 0; --k) S[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k8, v3.p[k], S[b], 0, 0, 0);
      }
    }
    __syncthreads();   // the operands are done with
  }
  if (bad) set_flag(a.flags, kFlagDecay);
  float* to = nullptr;
  if constexpr (OUT) {
    if (row0 + rows == x.row0 + x.rows && x.slot >= 0) to = a.state_out + ((size_t)x.slot * a.v_heads + h) * state_size;
  } else {
    to = a.seg_state + ((size_t)item * a.v_heads + h) * state_size;
    if (tid == 0) a.seg_decay[(size_t)item * a.v_heads + h] = G_all;
  }
  if (to)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int n = 0; n < 16; ++n) to[(size_t)(32 * t + 16 * (n >> 3) + line0 + (n & 7)) * DV + col] = S[t][n];
}

// The states that a sequence's segments begin with: what segment s left becomes
// what segment s + 1 begins with.
template <int DK, int DV>
__global__ __launch_bounds__(256) void k_linear_carry(LinearArgs a) {
  __shared__ int32_t s_seq[4];
  constexpr int kParts = DK * DV / 1024;
  const int part = blockIdx.x % kParts, h = blockIdx.x / kParts, seq = blockIdx.y;
  const int first = a.plan[seq], segs = a.plan[seq + 1] - first;
  if (segs < 2) return;
  const LinearSeq x = linear_seq(a, seq, s_seq, false);
  const size_t at = (size_t)part * 1024 + 4 * threadIdx.x, size = (size_t)DK * DV;
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  if (!x.fresh) S = *reinterpret_cast<const f32x4*>(a.state + ((size_t)x.slot * a.v_heads + h) * size + at);
  for (int s = 0; s + 1 < segs; ++s) {
    const size_t i = (size_t)(first + s) * a.v_heads + h;
    const float f = expf((float)a.seg_decay[i]);
    float* p = a.seg_state + i * size + at;
    const f32x4 u = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
    for (int n = 0; n < 4; ++n) S[n] = (f == 0.f ? 0.f : f * S[n]) + u[n];
    *reinterpret_cast<f32x4*>(p) = S;
  }
}

hipError_t launch_linear_chunks(const LinearArgs& a, int items, hipStream_t s) {
#define Q4NX_CHUNKS(DK, DV)                                                                                          \
  {                                                                                                                  \
    constexpr int kA = 64 * DK > 3 * 64 * 64 ? 64 * DK : 3 * 64 * 64;                                                \
    constexpr int kState = 2 * 64 * (DK + DV), kOut = 2 * (64 * DK + kA) + kState;                                   \
    if (a.seg_state) {                                                                                               \
      hipLaunchKernelGGL((k_linear_chunks<DK, DV, false>), dim3(items * a.v_heads), dim3(2 * DV), kState, s, a);     \
      hipLaunchKernelGGL((k_linear_carry<DK, DV>), dim3(a.v_heads * (DK * DV / 1024), a.n_seq), dim3(256), 0, s, a); \
    }                                                                                                                \
    hipLaunchKernelGGL((k_linear_chunks<DK, DV, true>), dim3(items * a.v_heads), dim3(2 * DV), kOut, s, a);          \
  }
  if (a.dk == 64 && a.dv == 64) Q4NX_CHUNKS(64, 64)
  else if (a.dk == 64) Q4NX_CHUNKS(64, 128)
  else if (a.dv == 64) Q4NX_CHUNKS(128, 64)
  else Q4NX_CHUNKS(128, 128)
#undef Q4NX_CHUNKS
  return hipGetLastError();
}

hipError_t launch_linear_rows(const LinearArgs& a, hipStream_t s) {
  // 32 columns a workgroup while whole heads would leave CUs empty
  const bool few = (int64_t)a.n_seq * a.v_heads < 512;
#define Q4NX_ROWS(DK, DV)                                                                                            \
  if (few) hipLaunchKernelGGL((k_linear_rows<DK, DV, 32>), dim3(a.v_heads * (DV / 32), a.n_seq), dim3(256), 0, s, a); \
  else hipLaunchKernelGGL((k_linear_rows<DK, DV, DV>), dim3(a.v_heads, a.n_seq), dim3(256), 0, s, a)
  if (a.dk == 64 && a.dv == 64) { Q4NX_ROWS(64, 64); }
  else if (a.dk == 64) { Q4NX_ROWS(64, 128); }
  else if (a.dv == 64) { Q4NX_ROWS(128, 64); }
  else { Q4NX_ROWS(128, 128); }
#undef Q4NX_ROWS
  return hipGetLastError();
}

}  // namespace q4nx
