// Linear attention with a decay for each head.
//
//   S_t = exp(d_t) S_{t-1} + k_t v_t^T,   out_t = scale q_t^T S_t
#include <algorithm>
#include <type_traits>

#include "kv_args.h"

namespace q4nx {

namespace {

struct LinearSeq {
  int32_t row0, rows;
  int32_t slot;    // -1: none
  bool fresh;      // begins with zeros
};

// Sequence s of the call, whose rows are start..end (kept rising, within the rows).  A slot that an earlier
// sequence with rows has is none.  All of the workgroup's threads call it; `taken` is LDS of their own.
__device__ inline LinearSeq linear_seq(const LinearArgs& a, int s, int start, int end, int32_t* taken, bool flags) {
  const int tid = threadIdx.x;
  if (tid == 0) *taken = 0;
  const int raw_slot = a.slots[s], fresh = a.fresh ? a.fresh[s] : 0, raw0 = a.q_start[s], raw1 = a.q_start[s + 1];
  __syncthreads();
  if (raw_slot >= 0 && s > 0) {
    for (int e = tid; e < s; e += blockDim.x)
      if (a.slots[e] == raw_slot) {
        int before = 0;   // rows: its start rises to the next one's
        for (int i = 0; i <= e; ++i) before = max(before, min(max(a.q_start[i], 0), a.M));
        if (min(max(a.q_start[e + 1], 0), a.M) > before) *taken = 1;
      }
    __syncthreads();
  }
  const bool bad = raw_slot < -1 || raw_slot >= a.n_slots || *taken;
  LinearSeq x;
  x.row0 = start;
  x.rows = end - start;
  x.slot = bad ? -1 : raw_slot;
  x.fresh = x.slot < 0 || fresh;
  if (flags && tid == 0) {
    if (bad && x.rows) set_flag(a.flags, kFlagIndex);
    if (raw0 != start || raw1 != end) set_flag(a.flags, kFlagRows);
  }
  return x;
}

// The largest of the first n + 1 row starts, each within the rows: where sequence n begins.  One wave at least.
__device__ inline int linear_start(const LinearArgs& a, int n) {
  const int lane = threadIdx.x & 63;
  int up = 0;
  for (int e = lane; e <= n; e += 64) up = max(up, min(max(a.q_start[e], 0), a.M));
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) up = max(up, __shfl_xor(up, off));
  return up;
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
// one row the state is read once and written once.  Bound by memory (64 sequences
// of one row, 32 heads of 128 x 128: 45 us, 270 MB at 5.9 TB/s).
template <int DK, int DV, int CW>
__global__ __launch_bounds__(256) void k_linear_rows(LinearArgs a) {
  constexpr int LC = CW / 4, RG = 256 / LC, RP = DK / RG;
  __shared__ int32_t s_taken;
  __shared__ float s_q[DK], s_k[DK];
  __shared__ f32x4 s_o[RG][LC];
  const int tid = threadIdx.x, lc = tid % LC, rg = tid / LC;
  constexpr int kParts = DV / CW;
  const int part = blockIdx.x % kParts, h = blockIdx.x / kParts, sq = blockIdx.y;
  const int start = linear_start(a, sq), end = max(start, min(max(a.q_start[sq + 1], 0), a.M));
  const LinearSeq x = linear_seq(a, sq, start, end, &s_taken, blockIdx.x == 0);
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
//
// 4096 rows of 32 heads of 128 x 128: 28, 12 and 55 us in the three launches.  The
// second moves its 67 MB at the rate of a copy; the others are bound by the cutting
// into parts and the latency between a chunk's steps (matrix cores 22 and 29 % busy,
// 2.9 and 3.2 TB/s).
namespace {

constexpr int kChunk = 64;

typedef __attribute__((address_space(3))) void lds_void;

// bf16 parts of x, its first, second and third eight bits: x = hi + mid + lo.  (Cut, not rounded, so that no part
// of a finite x overflows.)
struct Parts { bf16x8 p[3]; };
__device__ __forceinline__ Parts parts_of(const float (&x)[8]) {
  Parts r;
  u32x4 w[3];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    uint32_t b[3][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float v = x[2 * n + i];
      b[0][i] = __float_as_uint(v);
      const float r1 = v - __uint_as_float(b[0][i] & 0xFFFF0000u);
      b[1][i] = __float_as_uint(r1);
      b[2][i] = __float_as_uint(r1 - __uint_as_float(b[1][i] & 0xFFFF0000u));
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) w[k][n] = __builtin_amdgcn_perm(b[k][1], b[k][0], 0x07060302u);   // upper halves
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) r.p[k] = __builtin_bit_cast(bf16x8, w[k]);
  return r;
}

// The line of a 32-line operand that lane c holds: accumulators 8 t + n of half
// h are then lines 16 t + 8 h + n.
__device__ __forceinline__ int dealt(int c) { return 16 * (c >> 4) + 8 * ((c >> 2) & 1) + 4 * ((c >> 3) & 1) + (c & 3); }

__device__ __forceinline__ bf16x8 ld8(const uint16_t* p) { return *reinterpret_cast<const bf16x8*>(p); }

// The highest bit of each half that holds an infinity or NaN (and other bits).
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; }

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
__global__ __launch_bounds__(2 * DV, DV == 64 ? 1 : 2) void k_linear_chunks(LinearArgs a) {
  constexpr int kThreads = 2 * DV, kWaves = DV / 32, NT = DK / 32;
  // elements: q [64][DK/8][8] | k likewise, then the rows' weights [3][8][64][8] | k^T [8][DK][8] | v^T [8][DV][8].
  // Piece p of row r of q and k lies at p ^ turned(r), so that 16 rows' pieces of one column are 16 different
  // places of the banks.
  auto turned = [](int r) { return DK == 128 ? r & 15 : (r >> 1) & 7; };
  constexpr int kQ = 0, kK = OUT ? kChunk * DK : 0, kA = OUT ? (kChunk * DK > 3 * kChunk * kChunk ? kChunk * DK : 3 * kChunk * kChunk) : 0;
  constexpr int kKT = kK + kA, kVT = kKT + kChunk * DK;
  extern __shared__ __align__(16) uint16_t lds[];
  __shared__ double s_G[kChunk];
  __shared__ float s_d[kChunk], s_since[kChunk];
  __shared__ __align__(16) float s_left[kChunk];
  __shared__ int32_t s_taken;
  __shared__ int s_odd[2];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, c = lane & 31, hh = lane >> 5;
  // neighbouring heads, which share q and k, on one XCD (workgroups go round the eight)
  const int item = blockIdx.x / a.v_heads, nth = blockIdx.x % a.v_heads;
  const int h = a.v_heads % 8 ? nth : (nth & 7) * (a.v_heads >> 3) + (nth >> 3), kh = h / (a.v_heads / a.k_heads);
  int seq, seg, start, end, last_item;
  {
    int32_t* first = reinterpret_cast<int32_t*>(lds);
    linear_plan(a, first, first + kAttnMaxSeq + 1);
    if (blockIdx.x == 0)
      for (int e = tid; e <= a.n_seq; e += kThreads) {
        if (!OUT) a.plan[e] = first[e];
        else if (a.q_start[e] != first[kAttnMaxSeq + 1 + e]) set_flag(a.flags, kFlagRows);   // of sequences without rows too
      }
    if (item >= first[a.n_seq]) return;
    int count = 0;
    for (int b = 0; b < a.n_seq; b += 64) count += __popcll(__ballot(b + lane < a.n_seq && first[b + lane] <= item));
    seq = count - 1;
    seg = item - first[seq];
    start = first[kAttnMaxSeq + 1 + seq];
    end = first[kAttnMaxSeq + 2 + seq];
    last_item = first[seq + 1] - 1;
    if (!OUT && seg == first[seq + 1] - first[seq] - 1) return;   // what the last one adds, it adds itself
  }
  const LinearSeq x = linear_seq(a, seq, start, end, &s_taken, OUT && h == 0 && seg == 0);
  const int row0 = x.row0 + seg * a.seg, rows = min(a.seg, x.rows - seg * a.seg);
  const size_t state_size = (size_t)DK * DV;
  // the lane's column and first line of its accumulators
  const int col = 32 * wave + c, line0 = 8 * hh;
  f32x16 S[NT];
  {
    const float* from = nullptr;
    if (OUT) {
      if (seg > 0) from = a.seg_state + ((size_t)(item - 1) * a.v_heads + h) * state_size;
      else if (last_item > item) from = a.seg_state + ((size_t)last_item * a.v_heads + h) * state_size;
      else if (!x.fresh) from = a.state + ((size_t)x.slot * a.v_heads + h) * state_size;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int n = 0; n < 16; ++n) S[t][n] = from ? from[(uint32_t)(line0 * DV + col) + (32 * t + 16 * (n >> 3) + (n & 7)) * DV] : 0.f;
  }
  // A state that holds an infinity or NaN has no parts.
  auto state_odd = [&]() {
    float zero = 0.f;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int n = 0; n < 16; ++n) zero = fmaf(S[t][n], 0.f, zero);
    return !(zero == 0.f);
  };
  double G_all = 0.0;
  bool bad = false;
  // where the lane's operands lie: all else is an offset in the instruction
  const uint16_t* const at_w = lds + kK + (hh * kChunk + c) * 8;
  const int q_row = c * DK, k_row = dealt(c) * DK;
  int q_turn = 8 * (hh ^ turned(c)), k_turn = 8 * (hh ^ turned(dealt(c)));
  const uint16_t* const at_kt = lds + kKT + (hh * DK + dealt(c)) * 8;
  const uint16_t* const at_vt = lds + kVT + (hh * DV + col) * 8;
  if (tid < 2) s_odd[tid] = 0;
  __syncthreads();
  constexpr int kK8 = 4 * DK / kThreads, kV8 = 4 * DV / kThreads;
  uint32_t tk[kK8][8], tv[kV8][8];
  float next_d = a.decay[(row0 + min(lane, rows - 1)) * a.decay_ld + h];
  for (int r0 = 0, turn = 0; r0 < rows; r0 += kChunk, turn ^= 1) {
    const int n_rows = min(kChunk, rows - r0);
    const int64_t g0 = row0 + r0;
    uint32_t any = 0;
    // Operands to LDS.  Rows behind the last are the last again: no row's weight reaches them, and their share
    // of the state is 0.  q's and k's rows go straight there, in whole lines; what is wanted token by token
    // goes through registers.  No load stands under a branch, so that none waits for another.
    const int last = n_rows - 1;
    auto ask = [&](int ahead) {   // k and v of the chunk so many rows on, token by token
      const int behind = min(kChunk, rows - r0 - ahead) - 1;
      auto fetch = [&](const uint16_t* src, uint32_t ld, int width, int u, uint32_t (&w)[8]) {
        const int d = 2 * (u % (width / 2)), r = 8 * (u / (width / 2));
#pragma unroll
        for (int n = 0; n < 8; ++n) w[n] = *reinterpret_cast<const uint32_t*>(src + (min(r + n, behind) * ld + d));
      };
#pragma unroll
      for (int n = 0; n < kK8; ++n)
        fetch(a.k + (g0 + ahead) * a.k_ld + kh * DK, (uint32_t)a.k_ld, DK, tid + n * kThreads, tk[n]);
#pragma unroll
      for (int n = 0; n < kV8; ++n)
        fetch(a.v + (g0 + ahead) * a.v_ld + h * DV, (uint32_t)a.v_ld, DV, tid + n * kThreads, tv[n]);
    };
    if constexpr (OUT) {
      constexpr int kRow = DK / 8;   // pieces of a row; a wave has 64 pieces at a time, whole rows
#pragma unroll
      for (int n = 0; n < kRow / kWaves; ++n) {
        const int piece = (wave * (kRow / kWaves) + n) * 64, r = (piece + lane) / kRow, from = 8 * ((lane % kRow) ^ turned(r));
        const int row = min(r, last);
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void*)(a.q + g0 * a.q_ld + kh * DK + (row * (uint32_t)a.q_ld + from)),
            (lds_void*)(lds + kQ + piece * 8), 16, 0, 0);
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void*)(a.k + g0 * a.k_ld + kh * DK + (row * (uint32_t)a.k_ld + from)),
            (lds_void*)(lds + kK + piece * 8), 16, 0, 0);
      }
    }
    {
      if (OUT || r0 == 0) ask(0);
      if (wave == kWaves - 1) {
        float d = next_d;
        if (!(d <= 0.f)) {
          bad = true;
          d = 0.f;
        }
        s_d[lane] = d;
        if (r0 + kChunk < rows) next_d = a.decay[(g0 + min(kChunk + lane, rows - r0 - 1)) * a.decay_ld + h];
        // in powers of two; exp of less than -1e5 is 0 in fp32, and sums of these stay exact to 2^-30
        double G = lane <= last ? (double)fmaxf(d, -1e5f) * 1.4426950408889634 : 0.0;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
          const double o = __shfl_up(G, off);
          if (lane >= off) G += o;
        }
        // A decay whose exp is 0 cuts off an infinite or NaN state, which a sum of others never does: the segment's
        // sum is -Inf then.
        const bool cut = !OUT && __ballot(lane <= last && expf(d) == 0.f);
        s_G[lane] = cut && lane == 63 ? -__builtin_huge_val() : G;
        s_since[lane] = a.scale * __builtin_amdgcn_exp2f((float)G);
        const float left = __builtin_amdgcn_exp2f((float)(__shfl(G, 63) - G));
        s_left[lane] = lane <= last ? left : 0.f;
      }
      auto store = [&](int width, int at, int u, const uint32_t (&w)[8]) {
        const int d = 2 * (u % (width / 2)), r = 8 * (u / (width / 2));
        u32x4 lo, hi;
#pragma unroll
        for (int n = 0; n < 8; ++n) any |= nonfinite2(w[n]);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          lo[n] = __builtin_amdgcn_perm(w[2 * n + 1], w[2 * n], 0x05040100u);
          hi[n] = __builtin_amdgcn_perm(w[2 * n + 1], w[2 * n], 0x07060302u);
        }
        uint16_t* to = lds + at + ((r >> 3) * width + d) * 8;
        *reinterpret_cast<u32x4*>(to) = lo;
        *reinterpret_cast<u32x4*>(to + 8) = hi;
      };
#pragma unroll
      for (int n = 0; n < kK8; ++n) store(DK, kKT, tid + n * kThreads, tk[n]);
#pragma unroll
      for (int n = 0; n < kV8; ++n) store(DV, kVT, tid + n * kThreads, tv[n]);
      if (!OUT && r0 + kChunk < rows) ask(kChunk);   // the next chunk's, while this one is worked on
    }
    bool odd = (any & 0x80008000u) != 0;
    odd |= state_odd();
    if constexpr (OUT) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // what goes straight to LDS
    if (odd) s_odd[turn] = 1;
    __syncthreads();
    asm volatile("" : "+v"(q_turn), "+v"(k_turn));   // or every place is formed ahead of the loop, and spilled
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
            if constexpr (OUT) o = fmaf(bf16lo(lds[kQ + t * DK + 8 * ((line >> 3) ^ turned(t)) + (line & 7)]), S[b][n], o);
            if ((n & 3) == 3) __builtin_amdgcn_sched_barrier(0);   // or all of the row's operands are read at once, and spill
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
          struct Pair { bf16x8 k, q; };
          const uint16_t *kp = lds + kK + k_row + 32 * tj * DK, *qp = lds + kQ + q_row + 32 * ti * DK;
          fed<2, DK / 16>([&](int s) { return Pair{ld8(kp + (k_turn ^ 16 * s)), ld8(qp + (q_turn ^ 16 * s))}; },
                          [&](int, const Pair& x) { w[m] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x.k, x.q, w[m], 0, 0, 0); });
          const int row = 32 * ti + c;
          const double Gi = s_G[row];
          const double* Gj = s_G + 32 * tj + line0;
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            const int j = 16 * (n >> 3) + (n & 7);
            w[m][n] = j <= row - 32 * tj - line0 ? w[m][n] * a.scale * __builtin_amdgcn_exp2f((float)(Gi - Gj[j])) : 0.f;
          }
        }
      }
      __syncthreads();   // k's rows are done with
#pragma unroll
      for (int m = 0; m < kMine; ++m) {
        const int tile = wave + m * kWaves, ti = tile > 0, tj = tile > 1;
        uint16_t* to = lds + kK + ((4 * tj + hh) * kChunk + 32 * ti + c) * 8;
        if (tile < 3)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            float f[8];
#pragma unroll
            for (int n = 0; n < 8; ++n) f[n] = w[m][8 * t + n];
            const Parts q3 = parts_of(f);
#pragma unroll
            for (int i = 0; i < 3; ++i)
              *reinterpret_cast<bf16x8*>(to + i * kChunk * kChunk + 2 * t * kChunk * 8) = q3.p[i];
          }
      }
      const float* since = s_since + 4 * hh;
      // q S, scaled by each row's decay since the chunk's beginning
      f32x16 o[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < 16; ++n) o[i][n] = 0.f;
      struct Rows { bf16x8 q[2]; };
      fed<1, 2 * NT>([&](int n) { return Rows{{ld8(lds + kQ + q_row + (q_turn ^ 16 * n)),
                                               ld8(lds + kQ + q_row + 32 * DK + (q_turn ^ 16 * n))}}; },
                     [&](int n, const Rows& x) {
                       float f[8];
#pragma unroll
                       for (int i = 0; i < 8; ++i) f[i] = S[n >> 1][8 * (n & 1) + i];
                       const Parts s3 = parts_of(f);
#pragma unroll
                       for (int k = 2; k >= 0; --k)
#pragma unroll
                         for (int i = 0; i < 2; ++i) o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x.q[i], s3.p[k], o[i], 0, 0, 0);
                     });
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int n = 0; n < 16; ++n) o[i][n] *= since[32 * i + 8 * (n >> 2) + (n & 3)];
      __syncthreads();
      // six steps of 16 keys: two of the upper rows, four of the lower
      struct Step { bf16x8 w[3], v; };
      fed<1, 6>([&](int n) {
                  const int i = n > 1, s = i ? n - 2 : n;
                  Step x;
#pragma unroll
                  for (int k = 0; k < 3; ++k) x.w[k] = ld8(at_w + k * kChunk * kChunk + (2 * s * kChunk + 32 * i) * 8);
                  x.v = ld8(at_vt + 2 * s * DV * 8);
                  return x;
                },
                [&](int n, const Step& x) {
#pragma unroll
                  for (int k = 2; k >= 0; --k) o[n > 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x.w[k], x.v, o[n > 1], 0, 0, 0);
                });
      // byte offsets of 32 bits from the chunk's first row, formed here (hoisted, they would spill)
      uint8_t* op = reinterpret_cast<uint8_t*>(a.out + (g0 * a.v_heads + h) * DV);
      uint32_t step = 4u * a.v_heads * DV;
      asm volatile("" : "+s"(step));
      const uint32_t off = 4 * hh * step + 4 * col;
      auto write = [&](auto whole) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            const int row = 32 * i + 8 * (n >> 2) + (n & 3);
            if (whole || row + 4 * hh < n_rows) *reinterpret_cast<float*>(op + (off + row * step)) = o[i][n];
          }
      };
      if (n_rows == kChunk) write(std::true_type{});
      else write(std::false_type{});
    }
    // the state
    const float f_all = __builtin_amdgcn_exp2f((float)G_last);
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
      for (int n = 0; n < 16; ++n) S[b][n] *= f_all;
    struct Tokens { bf16x8 k[NT], v; f32x4 left[2]; };
    fed<1, 4>([&](int s) {
                Tokens x;
#pragma unroll
                for (int b = 0; b < NT; ++b) x.k[b] = ld8(at_kt + (2 * s * DK + 32 * b) * 8);
                x.v = ld8(at_vt + 2 * s * DV * 8);
                x.left[0] = *reinterpret_cast<const f32x4*>(&s_left[16 * s + 8 * hh]);
                x.left[1] = *reinterpret_cast<const f32x4*>(&s_left[16 * s + 8 * hh + 4]);
                return x;
              },
              [&](int, const Tokens& x) {
                float f[8];
#pragma unroll
                for (int n = 0; n < 8; ++n) f[n] = (float)x.v[n] * x.left[n >> 2][n & 3];
                const Parts v3 = parts_of(f);
#pragma unroll
                for (int k = 2; k >= 0; --k)
#pragma unroll
                  for (int b = 0; b < NT; ++b) S[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x.k[b], v3.p[k], S[b], 0, 0, 0);
              });
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
      for (int n = 0; n < 16; ++n) to[(uint32_t)(line0 * DV + col) + (32 * t + 16 * (n >> 3) + (n & 7)) * DV] = S[t][n];
}

// The states that a sequence's segments begin with: what segment s left becomes
// what segment s + 1 begins with.  What the first begins with goes to the place
// of the last, which left nothing: the last one's end may go to where the first
// one's state is, and nothing says which of the two runs first.
template <int DK, int DV>
__global__ __launch_bounds__(256) void k_linear_carry(LinearArgs a) {
  __shared__ int32_t s_taken;
  constexpr int kParts = DK * DV / 1024, kAhead = 8;
  const int part = blockIdx.x % kParts, h = blockIdx.x / kParts, seq = blockIdx.y;
  const int first = a.plan[seq], segs = a.plan[seq + 1] - first;
  if (segs < 2) return;
  const LinearSeq x = linear_seq(a, seq, 0, 0, &s_taken, false);
  const size_t at = (size_t)part * 1024 + 4 * threadIdx.x, size = (size_t)DK * DV;
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  if (!x.fresh) S = *reinterpret_cast<const f32x4*>(a.state + ((size_t)x.slot * a.v_heads + h) * size + at);
  *reinterpret_cast<f32x4*>(a.seg_state + ((size_t)(first + segs - 1) * a.v_heads + h) * size + at) = S;
  for (int s0 = 0; s0 + 1 < segs; s0 += kAhead) {   // their loads together: they wait for nothing, the sums for each other
    f32x4 u[kAhead];
    double d[kAhead];
    const int last = segs - 2;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const size_t i = (size_t)(first + min(s0 + j, last)) * a.v_heads + h;
      d[j] = a.seg_decay[i];
      u[j] = *reinterpret_cast<const f32x4*>(a.seg_state + i * size + at);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (s0 + j > last) break;
      const float f = __builtin_amdgcn_exp2f((float)d[j]);
      const bool cut = d[j] == -__builtin_huge_val();
#pragma unroll
      for (int n = 0; n < 4; ++n)   // 0 for what has decayed so far; an infinity or NaN stays unless it is cut off
        S[n] = (cut ? 0.f : f == 0.f && !(fabsf(S[n]) <= __FLT_MAX__) ? S[n] : f * S[n]) + u[j][n];
      *reinterpret_cast<f32x4*>(a.seg_state + ((size_t)(first + s0 + j) * a.v_heads + h) * size + at) = S;
    }
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
