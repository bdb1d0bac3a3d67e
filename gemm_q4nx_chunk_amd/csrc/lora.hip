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
//   route   (more than 64 rows) one workgroup counts the rows of each adapter
//           and cuts them into tiles of up to 64, or of 16 where few rows share
//           an adapter.  Up to 64 rows every wave of the other two finds its
//           tile, of up to 16 rows, itself.
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

// A buffer offset past every range, also with a column's or output's offset
// added (ranges are at most 2^31 bytes: the host cuts calls so): such loads give
// 0, such stores do nothing.
constexpr uint32_t kOutside = 0x80000000u;

// Keeps the compiler from moving a wave's LDS reads before its writes (which
// the hardware runs in order) or the other way round.
__device__ __forceinline__ void lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A tile of rows of one adapter, the same for the whole workgroup.
using Tile = LoraTile;

__device__ __forceinline__ int valid_id(const LoraArgs& a, int id) {
  return id >= 0 && id < a.n_adapters ? id : -1;
}

__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Fills rows[0..cnt) with the tile of workgroup t.  Call with all threads of
// the workgroup.  SUB: 16-row pieces of a tile.
//   up to 64 rows (SUB == 1): every wave finds it by itself, and all write the
//     same rows: a wave reads what it wrote, no barrier.  With few adapters, so
//     that few tiles are possible, by walking the adapters in order of their
//     first rows; else workgroup t is row t's, and has a tile if row t opens one.
//   above: from the route's tables; ends with a barrier.
template <int SUB>
__device__ __forceinline__ Tile find_tile(const LoraArgs& a, int t, int32_t* rows) {
  constexpr int kTile = 16 * SUB;
  const int tid = threadIdx.x, lane = tid & 63;
  Tile tile;
  if (SUB > 1 || a.M > kLoraWaveRows) {
    // everything at once: places past the tile's rows hold no row and are not used
    if (tid < kTile) rows[tid] = a.sorted[kTile * t + tid];
    tile.e = scalar(a.tiles[t].e);
    tile.cnt = scalar(a.tiles[t].cnt);
    __syncthreads();
    return tile;
  }
  const int id = lane < a.M ? valid_id(a, a.ids[lane]) : 0;
  const uint64_t all = __ballot(lane < a.M);
  uint64_t b;
  int before;   // rows of this adapter in tiles before this one
  if (a.max_tiles == a.M) {
    tile.e = __builtin_amdgcn_readlane(id, t);
    b = __ballot(id == tile.e) & all;
    before = __popcll(b & ((1ull << t) - 1ull));
    tile.cnt = before % kTile ? 0 : min(kTile, __popcll(b) - before);
  } else {
    tile.e = -1;
    tile.cnt = 0;
    before = 0;
    b = 0;
    int first = 0;   // tiles of the adapters passed
    for (uint64_t todo = all; todo;) {
      const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
      b = __ballot(id == e) & all;
      const int n = __popcll(b), tiles = (n + kTile - 1) / kTile;
      if (t < first + tiles) {
        before = kTile * (t - first);
        tile.e = e;
        tile.cnt = min(kTile, n - before);
        break;
      }
      first += tiles;
      todo &= ~b;
    }
  }
  const int at = __popcll(b & ((1ull << lane) - 1ull));
  if ((b >> lane & 1) && at >= before && at < before + tile.cnt) rows[at - before] = lane;
  lds_order();
  return tile;
}

__device__ __forceinline__ int used_rank(const LoraJob& j, int e) {
  if (!j.ranks) return j.rank;
  const int r = scalar(j.ranks[e]);
  return r < 0 ? 0 : r > j.rank ? j.rank : r;
}

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

}  // namespace

// ---------------------------------------------------------------------------
// route
// ---------------------------------------------------------------------------
// Sum over the lanes up to this one, by DPP: within rows of 16 lanes
// (row_shr 1, 2, 4, 8), then across them (row_bcast 15 and 31).
__device__ __forceinline__ int sum_to_here(int s) {
  s += __builtin_amdgcn_update_dpp(0, s, 0x111, 0xF, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x112, 0xF, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x114, 0xF, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x118, 0xF, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x142, 0xA, 0xF, false);
  s += __builtin_amdgcn_update_dpp(0, s, 0x143, 0xC, 0xF, false);
  return s;
}

// Counting sort of up to 4096 rows by adapter, bin n_adapters for rows without
// one: count, prefix sum of the bins' tiles, and every row goes to its place in
// its tile; a tile's first row writes its record.  The order of a bin's rows
// follows the LDS atomics and is not fixed; neither a row's sums nor its place
// in y depend on it.  Bound by its chain of latencies.
__global__ __launch_bounds__(1024) void k_lora_route(LoraArgs a) {
  constexpr int kPer = (kLoraMaxAdapters + 1 + 1023) / 1024;   // bins a thread
  constexpr int kRowsPer = kLoraMaxRows / 1024;
  __shared__ int32_t cnt[kPer * 1024], start[kPer * 1024];
  __shared__ int32_t wsum[16];
  __shared__ uint32_t bad;
  const int tid = threadIdx.x, lane = tid & 63, wave = scalar(tid >> 6);
  int id[kRowsPer];
#pragma unroll
  for (int i = 0; i < kRowsPer; ++i) id[i] = i * 1024 + tid < a.M ? a.ids[i * 1024 + tid] : -1;
  if (tid == 0) bad = 0;
  for (int e = tid; e <= a.n_adapters; e += 1024) cnt[e] = 0;
  __syncthreads();
  uint32_t wrong = 0;
  int bin[kRowsPer], slot[kRowsPer];
#pragma unroll
  for (int i = 0; i < kRowsPer; ++i) {
    const bool row = i * 1024 + tid < a.M;
    bin[i] = !row ? -1 : valid_id(a, id[i]) < 0 ? a.n_adapters : id[i];
    slot[i] = -1;
    wrong |= row && (id[i] < -1 || id[i] >= a.n_adapters) ? 1u : 0u;
  }
  if (wrong) atomicOr(&bad, 1u);
  // A prompt's rows come in runs, and a batch may have few adapters: up to four
  // of a wave's bins, each for all its lanes at once, while they have several;
  // what is left lane by lane.
#pragma unroll
  for (int i = 0; i < kRowsPer; ++i) {
    uint64_t todo = __ballot(bin[i] >= 0), mine[4] = {};
    if (todo == 0) continue;
    int first[4] = {};
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (todo == 0 || (r > 0 && __popcll(mine[r - 1]) < 4)) continue;
      const int b = __builtin_amdgcn_readlane(bin[i], __builtin_ctzll(todo));
      mine[r] = __ballot(bin[i] == b) & todo;
      if (lane == 0) first[r] = atomicAdd(&cnt[b], __popcll(mine[r]));
      todo &= ~mine[r];
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int f = __builtin_amdgcn_readfirstlane(first[r]);
      if (mine[r] >> lane & 1) slot[i] = f + __popcll(mine[r] & ((1ull << lane) - 1ull));
    }
    if (bin[i] >= 0 && slot[i] < 0) slot[i] = atomicAdd(&cnt[bin[i]], 1);
  }
  __syncthreads();
  // prefix sum of the tiles over the bins, kPer neighbouring bins a thread
  int c[kPer], tiles = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    c[i] = e <= a.n_adapters ? (cnt[e] + a.tile_rows - 1) / a.tile_rows : 0;
    tiles += c[i];
  }
  const int to_here = sum_to_here(tiles);
  if (lane == 63) wsum[wave] = to_here;
  __syncthreads();
  const int waves = sum_to_here(lane < 16 ? wsum[lane] : 0);   // lane w: tiles of waves 0 .. w
  int t0 = to_here - tiles + (wave ? __builtin_amdgcn_readlane(waves, wave - 1) : 0);
  const int n_tiles = __builtin_amdgcn_readlane(waves, 15);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    start[tid * kPer + i] = t0;
    t0 += c[i];
  }
  if (tid == 0) a.hdr[0] = (a.more ? a.hdr[0] : 0u) | bad;
  // Workgroups are dealt to the eight XCDs in turn, so place p is XCD p % 8's:
  // XCD j has tiles n j / 8 up to n (j + 1) / 8 of the n, so that neighbouring
  // tiles, of one adapter, find it and each other's u in one L2 (4096 x 4096,
  // rank 64, four adapters: the expand reads 76 MB from HBM instead of 112).
  for (int p = tid; p < a.max_tiles; p += 1024) {
    const int j = p & 7;
    if (p / 8 >= n_tiles * (j + 1) / 8 - n_tiles * j / 8) a.tiles[p] = {-1, 0};
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRowsPer; ++i) {
    if (bin[i] < 0) continue;
    const int in = slot[i] / a.tile_rows, first = in * a.tile_rows, t = start[bin[i]] + in;
    const int j = (8 * t + 7) / n_tiles, p = 8 * (t - n_tiles * j / 8) + j;
    a.sorted[p * a.tile_rows + slot[i] - first] = i * 1024 + tid;
    if (slot[i] == first)
      a.tiles[p] = {bin[i] < a.n_adapters ? bin[i] : -1, min(a.tile_rows, cnt[bin[i]] - first)};
  }
}

// ---------------------------------------------------------------------------
// shrink
// ---------------------------------------------------------------------------
// Workgroup (t, s, z): tile t, part s of the columns, rank group z of up to 16
// RB ranks.  Its eight waves take every eighth step of 64 columns each, for all ranks
// and rows of the tile: matrix-core tiles of 16 ranks x 16 rows x 32 columns.
// The matrix cores want lane l to hold row l % 16, but 16 neighbouring lanes
// that read 16 rows touch 16 cache lines for 256 bytes, so a wave loads a step
// with eight lanes to a row, a whole 128-byte line, and hands it over through
// LDS of its own: group c of 8 columns of row r at slot c ^ (r % 8) of the row,
// which spreads any eight rows over all banks.  No barrier: a wave's LDS
// operations run in order.  kAhead steps are in flight in registers.
//
// Measured (4096 rows, 14336 columns, rank 64; 64 rows of 40 adapters, 9728
// columns): operands straight from memory 75 and 14 us; 64 bytes of a row at a
// time through LDS 51 and 12; as here 37 and 11.
inline size_t lora_shrink_lds(int blocks, int sub) {
  return (size_t)kLoraShrinkWaves * blocks * 2048 + 16 * sub * sizeof(int32_t);
}

template <int RB, int SUB>
__global__ __launch_bounds__(64 * kLoraShrinkWaves, SUB == 1 ? 4 : 2) void k_lora_shrink(LoraArgs a) {
  constexpr int W = kLoraShrinkWaves;
  constexpr int kAhead = SUB == 1 && RB <= 2 ? 2 : 1;   // 128 registers a wave, 256 for SUB == 4
  constexpr int B = RB + SUB;   // 16-row blocks of a step: A's, then x's
  extern __shared__ u32x4 lds[];   // lora_shrink_lds(B, SUB) bytes
  u32x4(*stage)[B][128] = reinterpret_cast<u32x4(*)[B][128]>(lds);
  int32_t* rows = reinterpret_cast<int32_t*>(lds + W * B * 128);
  f32x4(*red)[RB][64] = reinterpret_cast<f32x4(*)[RB][64]>(stage);   // after the loop: B > RB, so it fits
  const int tid = threadIdx.x, lane = tid & 63, wave = scalar(tid >> 6);
  const int n = lane & 15, h = lane >> 4;
  if (a.M <= kLoraWaveRows && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && wave == 0) {
    const int id = lane < a.M ? a.ids[lane] : -1;
    const uint64_t bad = __ballot(id < -1 || id >= a.n_adapters);
    if (lane == 0) a.hdr[0] = (a.more ? a.hdr[0] : 0u) | (bad ? 1u : 0u);
  }
  int ji = 0;
  for (int i = 1; i < a.n_jobs; ++i)
    if ((int)blockIdx.z >= a.job[i].rg_begin) ji = i;
  const LoraJob& J = a.job[ji];
  const int r0 = ((int)blockIdx.z - J.rg_begin) * kLoraRankGroup;
  const Tile tile = find_tile<SUB>(a, blockIdx.x, rows);
  if (tile.cnt == 0 || tile.e < 0) return;
  const int rank = used_rank(J, tile.e);
  if (r0 >= rank) return;
  const int n_sub = (tile.cnt + 15) / 16;

  // Ranks and rows past the last are out of the buffers' range: they read as 0
  // without touching memory, and so do steps past the last.  No load is under
  // a branch, so none waits for another.
  const int lr = lane >> 3, lc = lane & 7;   // a load's row of half a block, its group of 8 columns
  const uint32_t row_bytes = (uint32_t)a.cols * 2;
  const uint16_t* pa = J.a + (size_t)tile.e * J.a_stride;
  const uint32_t na = rank * row_bytes, nx = a.M * row_bytes;
  uint32_t src[B][2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int r = r0 + 16 * i + 8 * p + lr;
      src[i][p] = r < rank ? r * row_bytes + 16 * lc : kOutside;
    }
#pragma unroll
    for (int i = 0; i < SUB; ++i) {
      const int r = 16 * i + 8 * p + lr;
      src[RB + i][p] = r < tile.cnt ? rows[r] * row_bytes + 16 * lc : kOutside;
    }
  }
  const int to = 8 * lr + (lc ^ lr);   // of half 1: 64 further
  const int from[2] = {8 * n + (h ^ (n & 7)), 8 * n + ((4 + h) ^ (n & 7))};

  f32x4 acc[RB][SUB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < SUB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int steps = a.cols / kLoraStepCols;
  const int s0 = steps * (int)blockIdx.y / a.split, s1 = steps * ((int)blockIdx.y + 1) / a.split;
  u32x4 in[kAhead][B][2];
  auto load = [&](u32x4 (&v)[B][2], int s) {
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(pa, s < s1 ? na : 0), rx = make_rsrc(a.x, s < s1 ? nx : 0);
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        v[i][p] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                i < RB ? ra : rx, src[i][p] + s * kLoraStepCols * 2, 0, 0));
  };
#pragma unroll
  for (int p = 0; p < kAhead; ++p) load(in[p], s0 + wave + p * W);
  for (int s = s0 + wave; s < s1; s += kAhead * W) {
#pragma unroll
    for (int p = 0; p < kAhead; ++p) {
#pragma unroll
      for (int i = 0; i < B; ++i) {
        stage[wave][i][to] = in[p][i][0];
        stage[wave][i][to + 64] = in[p][i][1];
      }
      load(in[p], s + (p + kAhead) * W);
      lds_order();
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        bf16x8 fa[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i) fa[i] = as_bf16x8(stage[wave][i][from[g]]);
#pragma unroll
        for (int j = 0; j < SUB; ++j) {
          const bf16x8 fx = as_bf16x8(stage[wave][RB + j][from[g]]);
#pragma unroll
          for (int i = 0; i < RB; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], fx, acc[i][j], 0, 0, 0);
        }
      }
      lds_order();
    }
  }
  __syncthreads();   // every wave is done with its stage
  // The waves' sums meet in LDS, 16 rows at a time, and are added in order.
  // Lane (n, h) of a piece: ranks 4 h .. + 3 of row n.
#pragma unroll
  for (int j = 0; j < SUB; ++j) {
    if (j >= n_sub) break;
    if (j > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < RB; ++i) red[wave][i][lane] = acc[i][j];
    __syncthreads();
    if (tid < 64 * RB) {
      f32x4 sum = red[0][wave][lane];
#pragma unroll
      for (int w = 1; w < W; ++w) sum += red[w][wave][lane];
      const int rr = r0 + 16 * wave + 4 * h, row = 16 * j + n;
      if (rr < J.rank && row < tile.cnt)
        *reinterpret_cast<f32x4*>(J.u + ((size_t)blockIdx.y * a.M + rows[row]) * J.rank + rr) = sum;
    }
  }
}

// ---------------------------------------------------------------------------
// expand
// ---------------------------------------------------------------------------
// The three bf16 parts of u: its sign and exponent with 8 bits of the mantissa
// each (truncation leaves every remainder exact).  Where u ends before its last
// part, the last one that it has is halved into the rest, which is exact too: a
// part of 0 would make NaN of an infinite weight of B, where u times it is
// infinite.  Infinities and NaNs, whose remainder is NaN, become all three parts.
__device__ __forceinline__ void split3(float v, uint32_t (&p)[3]) {
  float p0 = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u), r = v - p0;
  if (!(fabsf(r) > 0.f)) p0 = r = 0.5f * v;
  float p1 = __uint_as_float(__float_as_uint(r) & 0xFFFF0000u), p2 = r - p1;
  if (!(fabsf(p2) > 0.f)) p1 = p2 = 0.5f * r;
  p[0] = __float_as_uint(p0) >> 16;
  p[1] = __float_as_uint(p1) >> 16;
  p[2] = __float_as_uint(p2) >> 16;
}

// Workgroup (t, g): tile t, outputs n0 .. n0 + n_range of one job.  u of the
// tile's rows goes to LDS in the order in which the matrix cores take it; a
// wave takes 32 outputs at a time, two tiles of 16, B's rows straight from
// memory (16 bytes a lane: 8 ranks of one output).  The result of 16 rows goes
// through LDS of the wave's own, so that the base and y move eight lanes to a
// row, a whole 128-byte line (group c of 4 outputs of row r at slot c ^ (r % 8);
// 16 rows to 16 lanes instead, as the matrix cores leave them, 47 and 15 us at
// 4096 x 4096 rank 64 and 1000 x 4096 rank 16; as here 36 and 9).  B and the base of a wave's next
// outputs are loaded before the present ones are computed, the first before u
// is summed.  KS: 32-rank steps of the largest rank.
template <int KS, int SUB>
__global__ __launch_bounds__(256, KS == 1 ? 4 : KS == 2 ? 3 : 2) void k_lora_expand(LoraArgs a) {
  extern __shared__ u32x4 lu[];   // [3 parts][KS][SUB][64 lanes], then [4 waves][16 rows][8 groups]
  __shared__ int32_t rows[16 * SUB];
  const int tid = threadIdx.x, lane = tid & 63, wave = scalar(tid >> 6);
  const int n = lane & 15, h = lane >> 4;
  int ji = 0;
  for (int i = 1; i < a.n_jobs; ++i)
    if ((int)blockIdx.y >= a.job[i].wg_begin) ji = i;
  const LoraJob& J = a.job[ji];
  const int n0 = ((int)blockIdx.y - J.wg_begin) * a.n_range, n1 = min(J.rows, n0 + a.n_range);
  const Tile tile = find_tile<SUB>(a, blockIdx.x, rows);
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
  const int n_sub = (tile.cnt + 15) / 16;
  // This lane's B row within 32 outputs (of tile 0; tile 1: 16 further) and its
  // ranks 8 h .. of each step; ranks past the adapter's are not read.
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(J.b + (size_t)tile.e * J.b_stride, (uint32_t)J.rows * J.rank * 2);
  const uint32_t row_bytes = J.rank * 2;
  uint32_t pb[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) pb[s] = 32 * s + 8 * h < rank ? n * row_bytes + 64 * s + 16 * h : kOutside;
  // this lane's part of the base and y: row 16 j + 8 p + lane / 8, outputs 4 (lane % 8) .. + 3 of the 32
  const uint32_t ny = (uint32_t)a.M * J.rows * 4;
  const __amdgpu_buffer_rsrc_t rbase = make_rsrc(J.base, ny), ry = make_rsrc(J.y, ny);
  const int lr = lane >> 3, lc = lane & 7;
  uint32_t po[SUB][2];
#pragma unroll
  for (int j = 0; j < SUB; ++j)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int r = 16 * j + 8 * p + lr;
      po[j][p] = r < tile.cnt ? ((uint32_t)rows[r] * J.rows + 4 * lc) * 4 : kOutside;
    }

  constexpr bool kAheadB = KS * SUB < 32;   // else B's registers are needed twice over, which there are not
  u32x4 vb[2][KS];
  f32x4 vy[SUB][2];
  auto load_b = [&](int o0) {
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        vb[q][s] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rb, pb[s] + (o0 + 16 * q) * row_bytes, 0, 0));
  };
  auto load = [&](int o0) {
    if constexpr (kAheadB) load_b(o0);
#pragma unroll
    for (int j = 0; j < SUB; ++j)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        vy[j][p] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rbase, po[j][p] + o0 * 4, 0, 0));
  };
  const int o_first = n0 + 32 * wave, o_last = n1 - 32;   // rows is a multiple of 32
  load(min(o_first, o_last));

  const float scale = J.scale[tile.e];
  // Item (row, 8-rank block) goes to lane 16 * (block % 4) + row % 16 of k step
  // block / 4.  The parts of u are loaded four at a time; past the last they
  // are outside the buffer and add 0.
  const uint32_t part_bytes = (uint32_t)a.M * J.rank * 4;
  const __amdgpu_buffer_rsrc_t ru = make_rsrc(J.u, part_bytes * a.split);
  for (int it = tid; it < 16 * n_sub * 4 * KS; it += 256) {
    const int blk = it % (4 * KS), row = it / (4 * KS), rr = 8 * blk;
    uint32_t at = row < tile.cnt && rr < rank ? ((uint32_t)rows[row] * J.rank + rr) * 4 : kOutside;
    f32x4 v0 = {0.f, 0.f, 0.f, 0.f}, v1 = v0;
    for (int s0 = 0; s0 < a.split; s0 += 4) {
      f32x4 p0[4], p1[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        p0[s] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(ru, at + s * part_bytes, 0, 0));
        p1[s] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(ru, at + s * part_bytes + 16, 0, 0));
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        v0 += p0[s];
        v1 += p1[s];
      }
      at += 4 * part_bytes;
    }
    u32x4 w[3] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t part[3];
      split3(rr + i < rank ? (i < 4 ? v0[i & 3] : v1[i & 3]) * scale : 0.f, part);
#pragma unroll
      for (int q = 0; q < 3; ++q) w[q][i >> 1] |= part[q] << (16 * (i & 1));
    }
#pragma unroll
    for (int q = 0; q < 3; ++q)
      lu[((q * KS + blk / 4) * SUB + row / 16) * 64 + 16 * (blk & 3) + (row & 15)] = w[q];
  }
  // what the adapter does not use of the 8 ranks in which it ends counts as 0
  const int end_step = (rank - 1) / 32, left = rank - 32 * end_step - 8 * h;
  u32x4 mask;
#pragma unroll
  for (int i = 0; i < 4; ++i) mask[i] = 2 * i + 1 < left ? ~0u : 2 * i < left ? 0xFFFFu : 0u;
  f32x4* turn = reinterpret_cast<f32x4*>(lu + 3 * KS * SUB * 64) + wave * 128;
  __syncthreads();
  for (int o0 = o_first; o0 < n1; o0 += 128) {
    f32x4 cy[SUB][2];
    u32x4 cb[2][KS];
    if constexpr (!kAheadB) load_b(o0);
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int s = 0; s < KS; ++s) cb[q][s] = s == end_step ? vb[q][s] & mask : vb[q][s];
#pragma unroll
    for (int j = 0; j < SUB; ++j)
#pragma unroll
      for (int p = 0; p < 2; ++p) cy[j][p] = vy[j][p];
    load(min(o0 + 128, o_last));   // of the last outputs again, once, where there is no next
#pragma unroll
    for (int j = 0; j < SUB; ++j) {
      f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      if (j < n_sub) {
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int p = 2; p >= 0; --p) {
            const bf16x8 u = as_bf16x8(lu[((p * KS + s) * SUB + j) * 64 + lane]);
#pragma unroll
            for (int q = 0; q < 2; ++q)
              acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(cb[q][s]), u, acc[q], 0, 0, 0);
          }
      }
      // lane (n, h) has outputs 16 q + 4 h .. + 3 of row n
      turn[8 * n + (h ^ (n & 7))] = acc[0];
      turn[8 * n + ((4 + h) ^ (n & 7))] = acc[1];
      lds_order();
      // rows past the last are outside the buffer: no branch around a store, or every load would be waited for
#pragma unroll
      for (int p = 0; p < 2; ++p)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, cy[j][p] + turn[64 * p + 8 * lr + (lc ^ lr)]),
                                               ry, po[j][p] + o0 * 4, 0, 0);
      lds_order();
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
  if (a.M > kLoraWaveRows) hipLaunchKernelGGL(k_lora_route, dim3(1), dim3(1024), 0, s, a);
  const dim3 gs(a.max_tiles, a.split, z), ge(a.max_tiles, g);
  constexpr size_t kLdsStep = 3 * 64 * sizeof(u32x4);   // u of 16 rows and 32 ranks
  const int ks = (max_rank + 31) / 32;
#define Q4NX_LORA_EXPAND(KS, SUB)                                                                   \
  do {                                                                                              \
    const size_t lds = KS * SUB * kLdsStep + 4 * 128 * sizeof(f32x4);                               \
    if (lds > 65536)                                                                                \
      (void)hipFuncSetAttribute(reinterpret_cast<const void*>(k_lora_expand<KS, SUB>),              \
                                hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);              \
    hipLaunchKernelGGL((k_lora_expand<KS, SUB>), ge, dim3(256), lds, s, a);                         \
  } while (0)
#define Q4NX_LORA_SHRINK(RB, SUB)                                                                   \
  do {                                                                                              \
    const size_t lds = lora_shrink_lds(RB + SUB, SUB);                                              \
    if (lds > 65536)                                                                                \
      (void)hipFuncSetAttribute(reinterpret_cast<const void*>(k_lora_shrink<RB, SUB>),              \
                                hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);              \
    hipLaunchKernelGGL((k_lora_shrink<RB, SUB>), gs, dim3(64 * kLoraShrinkWaves), lds, s, a);       \
  } while (0)
#define Q4NX_LORA(SUB)                                                                              \
  do {                                                                                              \
    if (max_rank <= 16) Q4NX_LORA_SHRINK(1, SUB);                                                   \
    else if (max_rank <= 32) Q4NX_LORA_SHRINK(2, SUB);                                              \
    else Q4NX_LORA_SHRINK(4, SUB);                                                                  \
    if (ks <= 1) Q4NX_LORA_EXPAND(1, SUB);                                                          \
    else if (ks <= 2) Q4NX_LORA_EXPAND(2, SUB);                                                     \
    else if (ks <= 4) Q4NX_LORA_EXPAND(4, SUB);                                                     \
    else Q4NX_LORA_EXPAND(8, SUB);                                                                  \
  } while (0)
  if (a.tile_rows == 16) Q4NX_LORA(1);
  else Q4NX_LORA(4);
#undef Q4NX_LORA
#undef Q4NX_LORA_SHRINK
#undef Q4NX_LORA_EXPAND
  return hipGetLastError();
}

}  // namespace q4nx
