// Low-rank adapters of many requests beside a shared projection:
//
//   y[m] = base[m] + scale_e * B_e (A_e x[m]),   e = ids[m]
//
// with A_e [r_e][K] and B_e [N][r_e] in bf16.  Rows of one adapter are taken
// together, so that each adapter is read once per tile of rows however the
// requests lie in the batch (the grouping that onw's technical notes, "computing
// MoE prompts together", make for experts).
//
// Launches, on one stream:
//   route   (more than 256 rows) one workgroup counts the rows of each adapter
//           and cuts them into tiles of up to 64.  Up to 256 rows every
//           workgroup of the other two finds its tile itself: workgroup t is
//           row t's, and works if row t is the first of a tile of its adapter.
//   shrink  u = A_e x for a tile, columns split over workgroups and waves,
//           bf16 matrix cores, fp32 sums: the parts go to the workspace.
//   expand  sums the parts of u in order, times scale_e, and adds B_e u to the
//           base.  u is fp32 and B bf16: u is cut into three bf16 parts that
//           hold its 24 bits (8 each, by truncation), so the products are exact
//           and the result has fp32's precision.
// Every sum has a fixed order that depends on the call's sizes only, so a
// row's bits do not depend on where its tile mates lie.
#include "lora_args.h"
#include "q4nx_dev.h"

namespace q4nx {

namespace {

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

// A tile of rows of one adapter.
struct Tile {
  int e;      // adapter, -1: rows without one
  int cnt;    // rows
  int rank;   // ranks of job j that adapter e uses
};

__device__ __forceinline__ int valid_id(const LoraArgs& a, int id) {
  return id >= 0 && id < a.n_adapters ? id : -1;
}

// Fills rows[0..cnt) and returns the tile of workgroup t (cnt = 0: none).
// Call with all 256 threads; ends with a barrier.  LIM: most rows of a tile.
template <int LIM>
__device__ __forceinline__ Tile find_tile(const LoraArgs& a, int t, int32_t* rows, int32_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Tile tile;
  if (a.M > kLoraScanRows) {
    tile.e = -1;
    tile.cnt = 0;
    if (t < (int)a.hdr[1]) {
      tile.e = a.tiles[3 * t];
      const int p0 = a.tiles[3 * t + 1];
      tile.cnt = a.tiles[3 * t + 2];
      if (tid < tile.cnt) rows[tid] = a.sorted[p0 + tid];
    }
    __syncthreads();
    return tile;
  }
  // rows with row t's id: how many come before t, and which come from t on
  const int want = valid_id(a, a.ids[t]);
  const bool same = tid < a.M && valid_id(a, a.ids[tid < a.M ? tid : 0]) == want;
  const uint64_t b = __ballot(same);
  const uint64_t below_t = t >= 64 * wave + 64 ? b : t <= 64 * wave ? 0ull : b & ((1ull << (t - 64 * wave)) - 1ull);
  if (lane == 0) {
    scratch[wave] = __popcll(b);
    scratch[4 + wave] = __popcll(below_t);
  }
  __syncthreads();
  const int before = scratch[4] + scratch[5] + scratch[6] + scratch[7];
  const int total = scratch[0] + scratch[1] + scratch[2] + scratch[3];
  int at = __popcll(b & ((1ull << lane) - 1ull));
  for (int w = 0; w < wave; ++w) at += scratch[w];
  tile.e = want;
  tile.cnt = before % LIM ? 0 : min(LIM, total - before);   // row t opens a tile, or belongs to an earlier one
  if (same && at >= before && at < before + tile.cnt) rows[at - before] = tid;
  __syncthreads();
  return tile;
}

__device__ __forceinline__ int used_rank(const LoraJob& j, int e) {
  if (!j.ranks) return j.rank;
  const int r = j.ranks[e];
  return r < 0 ? 0 : r > j.rank ? j.rank : r;
}

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

}  // namespace

// ---------------------------------------------------------------------------
// route
// ---------------------------------------------------------------------------
// Counting sort of up to 4096 rows by adapter, bin n_adapters for rows without
// one.  The order of a bin's rows follows the LDS atomics and is not fixed;
// neither a row's sums nor its place in y depend on it.
__global__ __launch_bounds__(1024) void k_lora_route(LoraArgs a) {
  constexpr int kBins = kLoraMaxAdapters + 1, kPer = (kBins + 1023) / 1024;
  __shared__ int32_t cnt[kPer * 1024], start[kPer * 1024];
  __shared__ int32_t wsum[2][16];
  __shared__ uint32_t bad;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid == 0) bad = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) cnt[i * 1024 + tid] = 0;
  __syncthreads();
  constexpr int kRowsPer = kLoraMaxRows / 1024;
  int bin[kRowsPer], slot[kRowsPer];
#pragma unroll
  for (int i = 0; i < kRowsPer; ++i) {
    const int m = i * 1024 + tid;
    bin[i] = -1;
    if (m < a.M) {
      const int id = a.ids[m];
      bin[i] = valid_id(a, id) < 0 ? a.n_adapters : id;
      if (id < -1 || id >= a.n_adapters) atomicOr(&bad, 1u);
      slot[i] = atomicAdd(&cnt[bin[i]], 1);
    }
  }
  __syncthreads();
  // prefix sums of rows and tiles over the bins, kPer neighbouring bins a thread
  int c[kPer], rows = 0, tiles = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    c[i] = cnt[tid * kPer + i];
    rows += c[i];
    tiles += (c[i] + 63) / 64;
  }
  int ir = rows, it = tiles;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int r = __shfl_up(ir, off), t = __shfl_up(it, off);
    if (lane >= off) { ir += r; it += t; }
  }
  if (lane == 63) { wsum[0][wave] = ir; wsum[1][wave] = it; }
  __syncthreads();
  int r0 = ir - rows, t0 = it - tiles;
  for (int w = 0; w < wave; ++w) { r0 += wsum[0][w]; t0 += wsum[1][w]; }
  if (tid == 1023) {
    a.hdr[0] = bad;
    a.hdr[1] = (uint32_t)(t0 + tiles);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    start[e] = r0;
    for (int k = 0; k < c[i]; k += 64) {
      a.tiles[3 * t0] = e < a.n_adapters ? e : -1;
      a.tiles[3 * t0 + 1] = r0 + k;
      a.tiles[3 * t0 + 2] = min(64, c[i] - k);
      ++t0;
    }
    r0 += c[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRowsPer; ++i)
    if (bin[i] >= 0) a.sorted[start[bin[i]] + slot[i]] = i * 1024 + tid;
}

// ---------------------------------------------------------------------------
// shrink
// ---------------------------------------------------------------------------
// Workgroup (t, s, z): tile t, part s of the columns, rank group z of up to 16
// RB ranks.  A wave takes every fourth step of 64 columns, for all ranks and
// rows of its workgroup: matrix-core tiles of 16 ranks x 16 rows x 32 columns,
// operands straight from memory (16 lanes read 16 ranks' or rows' next 128
// bytes, 32 bytes a lane; A and x use the same order of columns within a step).
// SUB: 16-row pieces of a tile.
template <int RB, int SUB>
__global__ __launch_bounds__(256) void k_lora_shrink(LoraArgs a) {
  __shared__ int32_t rows[16 * SUB], scratch[8];
  __shared__ f32x4 red[2][RB * SUB][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = lane & 15, h = lane >> 4;
  if (a.M <= kLoraScanRows && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
    const int id = tid < a.M ? a.ids[tid] : -1;
    const int bad = __syncthreads_or(id < -1 || id >= a.n_adapters);
    if (tid == 0) a.hdr[0] = bad ? 1u : 0u;
  }
  int ji = 0;
  for (int i = 1; i < a.n_jobs; ++i)
    if ((int)blockIdx.z >= a.job[i].rg_begin) ji = i;
  const LoraJob& J = a.job[ji];
  const int r0 = ((int)blockIdx.z - J.rg_begin) * kLoraRankGroup;
  const Tile tile = find_tile<16 * SUB>(a, blockIdx.x, rows, scratch);
  if (tile.cnt == 0 || tile.e < 0) return;
  const int rank = used_rank(J, tile.e);
  if (r0 >= rank) return;
  const int n_rb = min(RB, (rank - r0 + 15) / 16), n_sub = (tile.cnt + 15) / 16;

  // Ranks and rows past the last repeat one that exists: their products land
  // in rows and columns of the result that nothing reads.
  const uint16_t* pa[RB];
  const uint16_t* px[SUB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
    pa[i] = J.a + (size_t)tile.e * J.a_stride + (size_t)min(r0 + 16 * i + n, rank - 1) * a.cols + 16 * h;
#pragma unroll
  for (int i = 0; i < SUB; ++i) px[i] = a.x + (size_t)rows[min(16 * i + n, tile.cnt - 1)] * a.cols + 16 * h;

  f32x4 acc[RB][SUB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < SUB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int steps = a.cols / kLoraStepCols;
  const int s0 = (int)((int64_t)steps * blockIdx.y / a.split), s1 = (int)((int64_t)steps * (blockIdx.y + 1) / a.split);
  for (int s = s0 + wave; s < s1; s += 4) {
    const int c0 = s * kLoraStepCols;
    u32x4 va[RB][2], vx[SUB][2];
#pragma unroll
    for (int i = 0; i < RB; ++i)
      if (i < n_rb) {
        va[i][0] = load16(pa[i] + c0);
        va[i][1] = load16(pa[i] + c0 + 8);
      }
#pragma unroll
    for (int i = 0; i < SUB; ++i)
      if (i < n_sub) {
        vx[i][0] = load16(px[i] + c0);
        vx[i][1] = load16(px[i] + c0 + 8);
      }
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < SUB; ++j)
        if (i < n_rb && j < n_sub) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(va[i][0]), as_bf16x8(vx[j][0]), acc[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(va[i][1]), as_bf16x8(vx[j][1]), acc[i][j], 0, 0, 0);
        }
  }
  // the four waves' sums: (0 + 2) + (1 + 3)
  if (wave >= 2)
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < SUB; ++j) red[wave - 2][i * SUB + j][lane] = acc[i][j];
  __syncthreads();
  if (wave < 2)
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < SUB; ++j) acc[i][j] += red[wave][i * SUB + j][lane];
  __syncthreads();
  if (wave == 1)
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < SUB; ++j) red[0][i * SUB + j][lane] = acc[i][j];
  __syncthreads();
  if (wave != 0) return;
  // lane (n, h): ranks 16 i + 4 h .. + 3 of row 16 j + n
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < SUB; ++j) {
      const int rr = r0 + 16 * i + 4 * h, row = 16 * j + n;
      if (rr < J.rank && row < tile.cnt)
        *reinterpret_cast<f32x4*>(J.u + ((size_t)blockIdx.y * a.M + rows[row]) * J.rank + rr) =
            acc[i][j] + red[0][i * SUB + j][lane];
    }
}

// ---------------------------------------------------------------------------
// expand
// ---------------------------------------------------------------------------
// The three bf16 parts of u: its sign and exponent with 8 bits of the mantissa
// each (truncation leaves every remainder exact); infinities and NaNs whole in
// the first.
__device__ __forceinline__ void split3(float v, uint32_t (&p)[3]) {
  const uint32_t b = __float_as_uint(v);
  if ((b & 0x7F800000u) == 0x7F800000u) {
    p[0] = v != v ? 0x7FC0u : b >> 16;
    p[1] = p[2] = 0;
    return;
  }
  p[0] = b >> 16;
  const float r1 = v - __uint_as_float(b & 0xFFFF0000u);
  const uint32_t b1 = __float_as_uint(r1);
  p[1] = b1 >> 16;
  p[2] = __float_as_uint(r1 - __uint_as_float(b1 & 0xFFFF0000u)) >> 16;
}

// Workgroup (t, g): tile t, outputs n0 .. n0 + n_range of one job.  First u of
// the tile's rows goes to LDS in the order in which the matrix cores take it;
// then each wave takes 16 outputs at a time: B's rows straight from memory
// (16 bytes a lane, 8 ranks of one output), the base and y 16 bytes a lane.
template <int SUB>
__global__ __launch_bounds__(256) void k_lora_expand(LoraArgs a) {
  extern __shared__ u32x4 lu[];   // [3 parts][ksteps][SUB][64 lanes]
  __shared__ int32_t rows[16 * SUB], scratch[8];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = lane & 15, h = lane >> 4;
  int ji = 0;
  for (int i = 1; i < a.n_jobs; ++i)
    if ((int)blockIdx.y >= a.job[i].wg_begin) ji = i;
  const LoraJob& J = a.job[ji];
  const int n0 = ((int)blockIdx.y - J.wg_begin) * a.n_range, n1 = min(J.rows, n0 + a.n_range);
  const Tile tile = find_tile<16 * SUB>(a, blockIdx.x, rows, scratch);
  if (tile.cnt == 0) return;
  const int rank = tile.e < 0 ? 0 : used_rank(J, tile.e);
  if (rank == 0) {   // no adapter: y is the base
    if (J.base == J.y) return;
    for (int r = wave; r < tile.cnt; r += 4) {
      const size_t o = (size_t)rows[r] * J.rows;
      for (int c = n0 + 4 * lane; c < n1; c += 256)   // rows and ranges are multiples of 4
        *reinterpret_cast<f32x4u*>(J.y + o + c) = *reinterpret_cast<const f32x4u*>(J.base + o + c);
    }
    return;
  }
  const int ks = (rank + 31) / 32, n_sub = (tile.cnt + 15) / 16;
  const float scale = J.scale[tile.e];
  // item (row, 8-rank block): lane 16 * (block % 4) + row % 16 of k step block / 4
  for (int it = tid; it < 16 * n_sub * 4 * ks; it += 256) {
    const int row = it % (16 * n_sub), blk = it / (16 * n_sub), rr = 8 * blk;
    u32x4 w[3] = {};
    if (row < tile.cnt && rr < rank) {
      f32x4 v0 = {0.f, 0.f, 0.f, 0.f}, v1 = v0;
      const float* p = J.u + (size_t)rows[row] * J.rank + rr;
      for (int s = 0; s < a.split; ++s, p += (size_t)a.M * J.rank) {
        v0 += *reinterpret_cast<const f32x4*>(p);
        v1 += *reinterpret_cast<const f32x4*>(p + 4);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t part[3];
        split3(rr + i < rank ? (i < 4 ? v0[i & 3] : v1[i & 3]) * scale : 0.f, part);
#pragma unroll
        for (int q = 0; q < 3; ++q) w[q][i >> 1] |= part[q] << (16 * (i & 1));
      }
    }
#pragma unroll
    for (int q = 0; q < 3; ++q)
      lu[((q * ks + blk / 4) * SUB + row / 16) * 64 + 16 * (blk & 3) + (row & 15)] = w[q];
  }
  __syncthreads();
  const uint16_t* pb = J.b + (size_t)tile.e * J.b_stride;
  for (int o0 = n0 + 16 * wave; o0 < n1; o0 += 64) {   // rows is a multiple of 32: whole tiles of 16
    f32x4 acc[SUB];
#pragma unroll
    for (int j = 0; j < SUB; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < ks; ++s) {
      const int rr = 32 * s + 8 * h, left = rank - rr;   // ranks of this lane's 8 that the adapter uses
      u32x4 vb = {0u, 0u, 0u, 0u};
      if (left > 0) {
        vb = load16(pb + (size_t)(o0 + n) * J.rank + rr);
#pragma unroll
        for (int i = 0; i < 4; ++i) vb[i] &= 2 * i + 1 < left ? ~0u : 2 * i < left ? 0xFFFFu : 0u;
      }
#pragma unroll
      for (int j = 0; j < SUB; ++j)
        if (j < n_sub)
#pragma unroll
          for (int q = 2; q >= 0; --q)
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(vb), as_bf16x8(lu[((q * ks + s) * SUB + j) * 64 + lane]),
                                                             acc[j], 0, 0, 0);
    }
    // lane (n, h): outputs o0 + 4 h .. + 3 of row 16 j + n
#pragma unroll
    for (int j = 0; j < SUB; ++j)
      if (16 * j + n < tile.cnt) {
        const size_t o = (size_t)rows[16 * j + n] * J.rows + o0 + 4 * h;
        *reinterpret_cast<f32x4u*>(J.y + o) = *reinterpret_cast<const f32x4u*>(J.base + o) + acc[j];
      }
  }
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  int max_rank = 0, z = 0;
  for (int i = 0; i < a.n_jobs; ++i) {
    max_rank = a.job[i].rank > max_rank ? a.job[i].rank : max_rank;
    z += (a.job[i].rank + kLoraRankGroup - 1) / kLoraRankGroup;
  }
  const LoraJob& last = a.job[a.n_jobs - 1];
  const int g = last.wg_begin + (last.rows + a.n_range - 1) / a.n_range;
  if (a.M > kLoraScanRows) hipLaunchKernelGGL(k_lora_route, dim3(1), dim3(1024), 0, s, a);
  const dim3 gs(a.max_tiles, a.split, z), ge(a.max_tiles, g);
  const size_t lds_row = (size_t)3 * ((max_rank + 31) / 32) * 64 * sizeof(u32x4);
#define Q4NX_LORA(SUB)                                                                              \
  do {                                                                                              \
    if (SUB * lds_row > 65536)                                                                      \
      (void)hipFuncSetAttribute(reinterpret_cast<const void*>(k_lora_expand<SUB>),                  \
                                hipFuncAttributeMaxDynamicSharedMemorySize, (int)(SUB * lds_row));  \
    if (max_rank <= 16)                                                                             \
      hipLaunchKernelGGL((k_lora_shrink<1, SUB>), gs, dim3(256), 0, s, a);                          \
    else if (max_rank <= 32)                                                                        \
      hipLaunchKernelGGL((k_lora_shrink<2, SUB>), gs, dim3(256), 0, s, a);                          \
    else                                                                                            \
      hipLaunchKernelGGL((k_lora_shrink<4, SUB>), gs, dim3(256), 0, s, a);                          \
    hipLaunchKernelGGL((k_lora_expand<SUB>), ge, dim3(256), (size_t)SUB * lds_row, s, a);           \
  } while (0)
  if (a.M <= 64) Q4NX_LORA(1);
  else Q4NX_LORA(4);
#undef Q4NX_LORA
  return hipGetLastError();
}

}  // namespace q4nx
