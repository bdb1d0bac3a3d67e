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
