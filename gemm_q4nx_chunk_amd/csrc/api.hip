// C ABI of libq4nx.so (declared in include/q4nx.h): host-side checks, then
// launches.  Every check runs before anything is enqueued, and no check
// touches the device, so the error paths can be exercised without a GPU.
//
// Check rules for a weight follow the 1bit engine docs, page "NPU engine"
// (section "Q4NX chunks": the chunk size names the kind, the two Q8 layouts
// cannot be told apart; section "From a GGUF": a checker refuses an unknown
// chunk size or a tensor shorter than its layout needs).
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <algorithm>
#include <cstring>
#include <mutex>
#include <queue>
#include <tuple>
#include <string>
#include <vector>

#include "../../include/q4nx.h"
#include "gemm_args.h"
#include "kv_args.h"
#include "logprobs_args.h"
#include "lora_args.h"
#include "moe_args.h"
#include "plan_args.h"
#include "q4nx_dev.h"
#include "topk.h"

static_assert(Q4NX_GEMM_BATCH_MAX_JOBS == q4nx::kGemmMaxJobs, "GEMM job table size");
static_assert(Q4NX_LORA_BATCH_MAX_JOBS == q4nx::kLoraMaxJobs, "adapter job table size");
static_assert(Q4NX_ATTN_MAX_SEQ == q4nx::kAttnMaxSeq, "sequences of one attention call");
static_assert(Q4NX_LORA_MAX_M == q4nx::kLoraMaxRows, "adapter rows of one call");

namespace {

thread_local std::string g_last_error;

int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = std::string(q4nx_status_str(status)) + ": " + buf;
  return status;
}

int ok() {
  g_last_error.clear();
  return Q4NX_OK;
}

int hip_status(hipError_t e, const char* where) {
  if (e == hipSuccess) return ok();
  return fail(Q4NX_E_HIP, "%s: %s", where, hipGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int kind_of(const q4nx_weight* w) {
  switch (w->chunk_bytes) {
    case Q4NX_Q4_1_BYTES: return q4nx::KIND_Q4_1;
    case Q4NX_Q4_K_BYTES: return q4nx::KIND_Q4_K;
    default: return w->q8_layout == Q4NX_Q8_LAYOUT_A ? q4nx::KIND_Q8_A : q4nx::KIND_Q8_B;
  }
}

int check_weight(const q4nx_weight* w, const char* name) {
  if (!w) return fail(Q4NX_E_ARG, "%s: null descriptor", name);
  if (!w->chunks) return fail(Q4NX_E_ARG, "%s: null chunk pointer", name);
  const int cb = w->chunk_bytes;
  if (cb != Q4NX_Q4_1_BYTES && cb != Q4NX_Q4_K_BYTES && cb != Q4NX_Q8_BYTES)
    return fail(Q4NX_E_CHUNK_KIND, "%s: unknown chunk size %d (5120 q4_1, 4736 Q4_K, 8704 Q8)",
                name, cb);
  if (cb == Q4NX_Q8_BYTES && w->q8_layout != Q4NX_Q8_LAYOUT_A && w->q8_layout != Q4NX_Q8_LAYOUT_B)
    return fail(Q4NX_E_Q8_LAYOUT, "%s: Q8 weight needs its code layout (A or B); it cannot be "
                "detected from the data", name);
  if (w->rows <= 0 || w->rows % 32 || w->cols <= 0 || w->cols % 256)
    return fail(Q4NX_E_SHAPE, "%s: %d x %d is not a whole number of 32 x 256 tiles", name,
                w->rows, w->cols);
  const int64_t need = (int64_t)(w->rows / 32) * (w->cols / 256) * cb;
  if (w->nbytes < need)
    return fail(Q4NX_E_SHORT, "%s: %lld bytes given, the %d x %d grid needs %lld", name,
                (long long)w->nbytes, w->rows, w->cols, (long long)need);
  if (!aligned(w->chunks, 16)) return fail(Q4NX_E_ALIGN, "%s: chunks not 16-byte aligned", name);
  return Q4NX_OK;
}

// Launch shape of a batch.  Many tile rows: 4-wave workgroups, waves per tile
// row chosen so the launch has about 2048 waves; each wave streams a run of
// chunks.  Few tile rows of long K (more than 16 tile columns): the launch is
// latency-bound on each wave's run of chunks, so 16-wave workgroups spread a
// tile row over enough waves that every wave holds about two chunks.  (Measured
// on the decode shapes: this halves the time of a 2560 x 9728 GEMV and slows
// the K = 2560 and K = 4096 ones, which keep 4-wave workgroups.)
#ifndef Q4NX_SMALL_ROWS
#define Q4NX_SMALL_ROWS 1024
#endif
#ifndef Q4NX_MKS_SHIFT
#define Q4NX_MKS_SHIFT 2
#endif
#ifndef Q4NX_SMALL_CPW
#define Q4NX_SMALL_CPW 2
#endif

int pow2_at_least(int v, int cap) {
  int p = 1;
  while (p < v && p < cap) p <<= 1;
  return p;
}

#ifndef Q4NX_SMALL_MIN_TC
#define Q4NX_SMALL_MIN_TC 17
#endif

// Launches of at most Q4NX_ROWSPLIT_TR tile rows (q4 kinds, prepared
// activations) split each tile's rows into two units of 16, and of at most
// Q4NX_ROWSPLIT4_TR into four units of 8, so they reach more CUs.
#ifndef Q4NX_ROWSPLIT_TR
#define Q4NX_ROWSPLIT_TR 1024
#endif
#ifndef Q4NX_ROWSPLIT4_TR
#define Q4NX_ROWSPLIT4_TR 0
#endif

// Three or four activation rows (q4 kinds): 4-wave workgroups hold their
// 168-235 registers three or two to a CU, so a launch of long K (at least
// Q4NX_MID_MIN_TC tile columns) or of few tile rows (at most Q4NX_MID_MAX_TR)
// would leave a wave alone on its SIMD with a long run of chunks; 8-wave
// workgroups split K eight ways instead.
#ifndef Q4NX_MID_MIN_TC
#define Q4NX_MID_MIN_TC 17
#endif
#ifndef Q4NX_MID_MAX_TR
#define Q4NX_MID_MAX_TR 0
#endif

int pick_waves(int kind, int64_t total_tr, int M, int max_tc) {
  const bool q4 = kind == q4nx::KIND_Q4_1 || kind == q4nx::KIND_Q4_K;
  if (q4 && (M == 3 || M == 4) && (max_tc >= Q4NX_MID_MIN_TC || total_tr <= Q4NX_MID_MAX_TR)) return 8;
  return (total_tr >= Q4NX_SMALL_ROWS || M > 2 || max_tc < Q4NX_SMALL_MIN_TC) ? 4 : 16;
}

int pick_ks(int waves, int64_t total_tr, int TC, bool mfma = false) {
  if (waves == 16) return pow2_at_least((TC + Q4NX_SMALL_CPW - 1) / Q4NX_SMALL_CPW, 16);
  if (waves == 8) return pow2_at_least((TC + Q4NX_SMALL_CPW - 1) / Q4NX_SMALL_CPW, 8);
  // the matrix-core kernel stages M >= 3 rows of records per workgroup, so
  // it takes fewer, longer workgroups
  if (mfma) total_tr <<= Q4NX_MKS_SHIFT;
  int ks = total_tr >= 2048 ? 1 : (total_tr >= 1024 ? 2 : 4);
  const int lim = TC >= 4 ? 4 : (TC >= 2 ? 2 : 1);
  return ks < lim ? ks : lim;
}

// Launch shape of one kind's jobs (all valid, same M) in one launch.
struct BatchShape {
  int waves, xl, parts;   // parts: units per tile row
  bool mfma;              // k_gemv_q4m (q4 kinds, prepared records, M >= kGemvMfmaMinM)
};

BatchShape batch_shape(int kind, int64_t total_tr, int max_tc, int M) {
  BatchShape sh;
  sh.waves = pick_waves(kind, total_tr, M, max_tc);
  sh.xl = q4nx::gemv_xl_bytes(kind, M, sh.waves, max_tc);
  if (sh.waves == 8 && sh.xl <= 0) {   // the 8-wave kernel stages its activations in LDS
    sh.waves = 4;
    sh.xl = q4nx::gemv_xl_bytes(kind, M, 4, max_tc);
  }
  const bool q4 = kind == q4nx::KIND_Q4_1 || kind == q4nx::KIND_Q4_K;
  sh.parts = !(q4 && sh.xl > 0) ? 1 : total_tr <= Q4NX_ROWSPLIT4_TR ? 4 : total_tr <= Q4NX_ROWSPLIT_TR ? 2 : 1;
  sh.mfma = q4 && sh.xl > 0 && M >= q4nx::kGemvMfmaMinM;
  return sh;
}

// Fills the kernel's job record of j, its workgroups starting at wg_begin;
// returns its workgroup count.
int fill_job(q4nx::GemvJob& g, const q4nx_gemv_job* j, const BatchShape& sh, int64_t total_tr, int wg_begin) {
  g.w = static_cast<const uint8_t*>(j->w.chunks);
  g.x = j->x;
  g.y = j->y;
  g.TR = j->w.rows / 32;
  g.TC = j->w.cols / 256;
  g.ldx = j->w.cols;
  g.ldy = j->w.rows;
  g.ks = pick_ks(sh.waves, total_tr, g.TC, sh.mfma);
  g.wg_begin = wg_begin;
  const int rpw = sh.waves / g.ks;
  return (g.TR * sh.parts + rpw - 1) / rpw;
}

// Launch one kind's jobs (all valid, same M) in as few launches as the job
// table allows.
int run_batch(int kind, const q4nx_gemv_job* const* jobs, int n, int M, hipStream_t s) {
  int64_t total_tr = 0;
  int max_tc = 0;
  for (int i = 0; i < n; ++i) {
    total_tr += jobs[i]->w.rows / 32;
    max_tc = std::max(max_tc, jobs[i]->w.cols / 256);
  }
  const BatchShape sh = batch_shape(kind, total_tr, max_tc, M);
  // q4 kinds at M = 5..8 whose records do not fit in LDS (long K): two passes
  // of 4 rows through the matrix-core kernel, rows 0..3 and then M-4..M-1,
  // instead of the kernel that loads activations per chunk.  Each pass reads
  // the weights once; a row computed by both comes out with the same bits
  // both times (same kernel, shape and K split), so the second write changes
  // nothing and a row's bits do not depend on its slot.
  const bool q4 = kind == q4nx::KIND_Q4_1 || kind == q4nx::KIND_Q4_K;
  if (q4 && M > 4 && sh.xl <= 0 && q4nx::gemv_xl_bytes(kind, 4, 4, max_tc) > 0) {
    std::vector<q4nx_gemv_job> part(n);
    std::vector<const q4nx_gemv_job*> ptr(n);
    for (int m0 : {0, M - 4}) {
      for (int i = 0; i < n; ++i) {
        part[i] = *jobs[i];
        part[i].x = jobs[i]->x + (size_t)m0 * jobs[i]->w.cols;
        part[i].y = jobs[i]->y + (size_t)m0 * jobs[i]->w.rows;
        ptr[i] = &part[i];
      }
      const int st = run_batch(kind, ptr.data(), n, 4, s);
      if (st != Q4NX_OK) return st;
    }
    return Q4NX_OK;
  }
  for (int i0 = 0; i0 < n; i0 += q4nx::kMaxBatch) {
    const int cnt = n - i0 < q4nx::kMaxBatch ? n - i0 : q4nx::kMaxBatch;
    q4nx::GemvBatch b;
    memset(&b, 0, sizeof b);
    b.sl = 4 / sh.parts;
    int wg = 0;
    for (int t = 0; t < cnt; ++t) wg += fill_job(b.job[t], jobs[i0 + t], sh, total_tr, wg);
    b.n_jobs = cnt;
    const hipError_t e = q4nx::launch_gemv(kind, M, sh.waves, b, wg, sh.xl, s);
    if (e != hipSuccess) return hip_status(e, "gemv launch");
  }
  return Q4NX_OK;
}

// Launch shape of the top-k GEMV (one job, 4-wave workgroups, the rules of
// run_batch otherwise).  Returns false when the shape does not fit it.
struct TopkShape {
  q4nx::GemvBatch b;
  int n_wg, xl;
  size_t ws_bytes;
};

constexpr size_t kTopkCntBytes = 256;   // n_grp + 1 <= 65 counters

bool topk_shape(const q4nx_weight* w, int M, int k, TopkShape& t) {
  const int kind = kind_of(w);
  const int TR = w->rows / 32, TC = w->cols / 256;
  t.xl = q4nx::gemv_xl_bytes(kind, M, 4, TC);
  if (t.xl <= 0) return false;
  const bool q4 = kind == q4nx::KIND_Q4_1 || kind == q4nx::KIND_Q4_K;
  const int parts = !q4 ? 1 : TR <= Q4NX_ROWSPLIT4_TR ? 4 : TR <= Q4NX_ROWSPLIT_TR ? 2 : 1;
  memset(&t.b, 0, sizeof t.b);
  t.b.sl = 4 / parts;
  q4nx::GemvJob& g = t.b.job[0];
  g.w = static_cast<const uint8_t*>(w->chunks);
  g.TR = TR;
  g.TC = TC;
  g.ldx = w->cols;
  g.ldy = w->rows;
  // the K split q4nx_gemv takes for this weight and M (so the logits agree bit for bit)
  g.ks = pick_ks(4, TR, TC, q4 && M >= q4nx::kGemvMfmaMinM);
  g.wg_begin = 0;
  t.b.n_jobs = 1;
  const int rpw = 4 / g.ks;
  t.n_wg = (TR * parts + rpw - 1) / rpw;
  if (t.n_wg > q4nx::kTopkMaxWg) return false;
  t.b.tk.k = k;
  t.b.tk.n_wg = t.n_wg;
  t.b.tk.n_grp = (t.n_wg + q4nx::kTopkGroup - 1) / q4nx::kTopkGroup;
  t.ws_bytes = kTopkCntBytes + (size_t)(t.n_wg + t.b.tk.n_grp) * M * k * 8;
  return true;
}

int check_gemv_io(const q4nx_weight* w, const void* x, const float* y, int M, const char* name) {
  int st = check_weight(w, name);
  if (st) return st;
  if (!x || !y) return fail(Q4NX_E_ARG, "%s: null x or y", name);
  if (M < 1 || M > Q4NX_GEMV_MAX_M)
    return fail(Q4NX_E_ARG, "%s: M = %d outside 1..%d", name, M, (int)Q4NX_GEMV_MAX_M);
  if (!aligned(x, 16)) return fail(Q4NX_E_ALIGN, "%s: x not 16-byte aligned", name);
  if (!aligned(y, 4)) return fail(Q4NX_E_ALIGN, "%s: y not 4-byte aligned", name);
  return Q4NX_OK;
}

}  // namespace

extern "C" {

const char* q4nx_status_str(int status) {
  switch (status) {
    case Q4NX_OK: return "ok";
    case Q4NX_E_ARG: return "invalid argument";
    case Q4NX_E_CHUNK_KIND: return "unknown or unsupported chunk kind";
    case Q4NX_E_SHAPE: return "bad shape";
    case Q4NX_E_SHORT: return "tensor shorter than its layout needs";
    case Q4NX_E_ALIGN: return "misaligned pointer";
    case Q4NX_E_WORKSPACE: return "workspace missing or too small";
    case Q4NX_E_Q8_LAYOUT: return "Q8 code layout not given";
    case Q4NX_E_HIP: return "HIP runtime error";
  }
  return "unknown status";
}

const char* q4nx_last_error(void) { return g_last_error.c_str(); }

int q4nx_version(void) { return 100; }

int q4nx_weight_check(const q4nx_weight* w) {
  const int st = check_weight(w, "weight");
  return st ? st : ok();
}

int q4nx_gemv(const q4nx_weight* w, const uint16_t* x, float* y, int M, void* stream) {
  const int st = check_gemv_io(w, x, y, M, "gemv");
  if (st) return st;
  q4nx_gemv_job j{*w, x, y};
  const q4nx_gemv_job* pj = &j;
  const int r = run_batch(kind_of(w), &pj, 1, M, static_cast<hipStream_t>(stream));
  return r ? r : ok();
}

int q4nx_gemv_batched(const q4nx_gemv_job* jobs, int n_jobs, int M, void* stream) {
  if (!jobs) return fail(Q4NX_E_ARG, "gemv_batched: null job array");
  if (n_jobs < 1 || n_jobs > Q4NX_BATCH_MAX_JOBS)
    return fail(Q4NX_E_ARG, "gemv_batched: %d jobs outside 1..%d", n_jobs,
                (int)Q4NX_BATCH_MAX_JOBS);
  for (int i = 0; i < n_jobs; ++i) {
    char name[48];
    snprintf(name, sizeof name, "gemv_batched job %d", i);
    const int st = check_gemv_io(&jobs[i].w, jobs[i].x, jobs[i].y, M, name);
    if (st) return st;
  }
  const q4nx_gemv_job* by_kind[4][Q4NX_BATCH_MAX_JOBS];
  int cnt[4] = {0, 0, 0, 0};
  for (int i = 0; i < n_jobs; ++i) {
    const int k = kind_of(&jobs[i].w);
    by_kind[k][cnt[k]++] = &jobs[i];
  }
  for (int k = 0; k < 4; ++k) {
    if (!cnt[k]) continue;
    const int r = run_batch(k, by_kind[k], cnt[k], M, static_cast<hipStream_t>(stream));
    if (r) return r;
  }
  return ok();
}

size_t q4nx_gemv_topk_ws(const q4nx_weight* w, int M, int k) {
  TopkShape t;
  if (check_weight(w, "gemv_topk_ws") || M < 1 || M > 4 || k < 1 || k > q4nx::kTopkMax ||
      !topk_shape(w, M, k, t))
    return 0;
  return t.ws_bytes;
}

int q4nx_gemv_topk(const q4nx_weight* w, const uint16_t* x, int M, int k, float* y, int32_t* ids,
                   float* vals, void* ws, size_t ws_bytes, void* stream) {
  int st = check_weight(w, "gemv_topk");
  if (st) return st;
  if (!x || !ids) return fail(Q4NX_E_ARG, "gemv_topk: null x or ids");
  if (M < 1 || M > 4) return fail(Q4NX_E_ARG, "gemv_topk: M = %d outside 1..4", M);
  if (k < 1 || k > q4nx::kTopkMax || k > w->rows)
    return fail(Q4NX_E_ARG, "gemv_topk: k = %d outside 1..min(%d, rows)", k, q4nx::kTopkMax);
  if (!aligned(x, 16)) return fail(Q4NX_E_ALIGN, "gemv_topk: x not 16-byte aligned");
  if ((y && !aligned(y, 4)) || !aligned(ids, 4) || (vals && !aligned(vals, 4)))
    return fail(Q4NX_E_ALIGN, "gemv_topk: y, ids and vals must be 4-byte aligned");
  TopkShape t;
  if (!topk_shape(w, M, k, t))
    return fail(Q4NX_E_SHAPE, "gemv_topk: %d x %d at M = %d does not fit the prepared-activation GEMV "
                "with at most %d workgroups", w->rows, w->cols, M, q4nx::kTopkMaxWg);
  if (!ws || ws_bytes < t.ws_bytes)
    return fail(Q4NX_E_WORKSPACE, "gemv_topk: workspace of %zu bytes, %zu needed", ws_bytes, t.ws_bytes);
  if (!aligned(ws, 256)) return fail(Q4NX_E_ALIGN, "gemv_topk: workspace not 256-byte aligned");
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  t.b.job[0].x = x;
  t.b.job[0].y = y;
  t.b.tk.cnt = reinterpret_cast<uint32_t*>(wsb);
  t.b.tk.cand = reinterpret_cast<uint64_t*>(wsb + kTopkCntBytes);
  t.b.tk.ids = ids;
  t.b.tk.vals = vals;
  const hipError_t e = q4nx::launch_gemv_topk(kind_of(w), M, t.b, t.n_wg, t.xl, static_cast<hipStream_t>(stream));
  return hip_status(e, "gemv_topk launch");
}

}  // extern "C"

namespace {

// q4nx_gemm_exchange_mode: 0 default, 1 odd groups act displaced, 2 device-coherent exchange.
std::atomic<int> g_gemm_exchange_mode{0};

// Checks a block-GEMM launch over weights w[0..n-1] sharing X and fills the
// kernel arguments (all but the workspace).  Returns a status.
int gemm_setup(const q4nx_weight* const* w, float* const* Y, int n, const uint16_t* X, int M,
               const char* name, q4nx::GemmArgs& a) {
  if (n < 1 || n > q4nx::kGemmMaxJobs)
    return fail(Q4NX_E_ARG, "%s: %d weights outside 1..%d", name, n, q4nx::kGemmMaxJobs);
  for (int i = 0; i < n; ++i) {
    const int st = check_weight(w[i], name);
    if (st) return st;
    if (w[i]->chunk_bytes == Q4NX_Q8_BYTES)
      return fail(Q4NX_E_CHUNK_KIND, "%s: Q8 weights are not supported by the block GEMM", name);
    if (kind_of(w[i]) != kind_of(w[0]) || w[i]->cols != w[0]->cols)
      return fail(Q4NX_E_SHAPE, "%s: weight %d differs from weight 0 in chunk kind or columns", name, i);
    if (!Y[i]) return fail(Q4NX_E_ARG, "%s: null Y of weight %d", name, i);
    if (!aligned(Y[i], 4)) return fail(Q4NX_E_ALIGN, "%s: Y of weight %d not 4-byte aligned", name, i);
  }
  if (!X) return fail(Q4NX_E_ARG, "%s: null X", name);
  if (M < 1 || M > Q4NX_GEMM_MAX_M)
    return fail(Q4NX_E_ARG, "%s: M = %d outside 1..%d", name, M, (int)Q4NX_GEMM_MAX_M);
  if (!aligned(X, 16)) return fail(Q4NX_E_ALIGN, "%s: X not 16-byte aligned", name);
  a = q4nx::GemmArgs{};
  int nb = 0;
  for (int i = 0; i < n; ++i) {
    a.job[i].w = static_cast<const uint8_t*>(w[i]->chunks);
    a.job[i].Y = Y[i];
    a.job[i].TR = (int32_t)(w[i]->rows / 32);
    a.job[i].nb0 = nb;
    nb += q4nx::gemm_blocks(a.job[i].TR, M);
  }
  a.n_jobs = n;
  a.X = X;
  a.TC = (int32_t)(w[0]->cols / 256);
  a.M = M;
  a.NB = nb;
  a.S = q4nx::gemm_parts(nb, a.TC);
  return Q4NX_OK;
}

int gemm_launch(q4nx::GemmArgs& a, int kind, void* ws, size_t ws_bytes, void* stream,
                const char* name, bool may_probe = true) {
  const size_t need = q4nx::gemm_ws_bytes(a.NB, a.TC, a.M);
  if (need && (!ws || ws_bytes < need))
    return fail(Q4NX_E_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", name, ws_bytes, need);
  if (need && !aligned(ws, 256)) return fail(Q4NX_E_ALIGN, "%s: workspace not 256-byte aligned", name);
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.cnt = need ? reinterpret_cast<uint32_t*>(w) : nullptr;
  a.claim = need ? reinterpret_cast<uint32_t*>(w + q4nx::kGemmClaimOff) : nullptr;
  a.rescued = need ? reinterpret_cast<uint32_t*>(w + q4nx::kGemmRescueOff) : nullptr;
  a.diag = need ? reinterpret_cast<uint32_t*>(w + q4nx::kGemmDiagOff) : nullptr;
  a.partial = need ? reinterpret_cast<float*>(w + q4nx::kGemmCntBytes) : nullptr;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const int mode = g_gemm_exchange_mode.load(std::memory_order_relaxed);
  a.test_mode = mode == 1 ? 1 : 0;
  const bool local = a.S > 1 && mode != 2 &&
                     (may_probe ? q4nx::xcd_round_robin(st) : q4nx::xcd_round_robin_known()) == 1;
  const hipError_t e = q4nx::launch_gemm(kind, a, local, st);
  return hip_status(e, name);
}

}  // namespace

extern "C" {

int q4nx_gemm_block(const q4nx_weight* w, const uint16_t* X, float* Y, int M, void* ws,
                    size_t ws_bytes, void* stream) {
  q4nx::GemmArgs a;
  const int st = gemm_setup(&w, &Y, 1, X, M, "gemm_block", a);
  if (st) return st;
  const int r = gemm_launch(a, kind_of(w), ws, ws_bytes, stream, "gemm_block");
  return r ? r : ok();
}

}  // extern "C"

// ---------------------------------------------------------------------------
// the allocation-free block GEMM
// ---------------------------------------------------------------------------
// Its workspace is `scratch`, in the code object: every GPU the library runs
// on holds one until the process ends.  Each call clears the header words
// that must start at zero (arrival counters, claim words, rescue flags) with a
// small kernel on the caller's stream before the GEMM; the partial tiles are
// written before they are read.  Calls that overlap on one GPU share the array
// and race.  Host code never passes the array's name to a kernel: its device
// address comes from hipGetSymbolAddress, once per device, with that device
// current.
constexpr size_t kNoAllocGemmBytes = q4nx::kGemmCntBytes + ((size_t)16 << 20);
static_assert(kNoAllocGemmBytes >= q4nx::kGemmCntBytes + (size_t)Q4NX_GEMM_WG_TARGET * 64 *
                                       q4nx::kGemmRowsPerWg * 32 * 4,
              "scratch holds the largest split any call makes (workgroup rows x parts <= the target)");

static __device__ __align__(256) uint8_t scratch[kNoAllocGemmBytes];

namespace {

constexpr int kHeaderZeroWords = (int)(q4nx::kGemmDiagOff / 4);

__global__ void __launch_bounds__(256) k_clear_words(uint32_t* p, int n) {
  for (int i = threadIdx.x; i < n; i += 256) p[i] = 0u;
}

std::once_flag g_scratch_once[64];
void* g_scratch_ptr[64];
hipError_t g_scratch_err[64];

int scratch_address(void** out) {
  int dev = 0;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_status(e, "gemm_block_noalloc: current device");
  if (dev < 0 || dev >= 64) return fail(Q4NX_E_HIP, "gemm_block_noalloc: device %d beyond 63", dev);
  std::call_once(g_scratch_once[dev], [dev] {
    void* p = nullptr;
    g_scratch_err[dev] = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    g_scratch_ptr[dev] = g_scratch_err[dev] == hipSuccess ? p : nullptr;
  });
  if (g_scratch_err[dev] != hipSuccess) return hip_status(g_scratch_err[dev], "gemm_block_noalloc: scratch address");
  if (!g_scratch_ptr[dev]) return fail(Q4NX_E_HIP, "gemm_block_noalloc: scratch address is null");
  *out = g_scratch_ptr[dev];
  return Q4NX_OK;
}

}  // namespace

extern "C" {

size_t q4nx_gemm_block_noalloc_max(void) { return kNoAllocGemmBytes; }

int q4nx_gemm_block_noalloc(const q4nx_weight* w, const uint16_t* X, float* Y, int M, void* stream) {
  q4nx::GemmArgs a;
  const int st = gemm_setup(&w, &Y, 1, X, M, "gemm_block_noalloc", a);
  if (st) return st;
  const size_t need = q4nx::gemm_ws_bytes(a.NB, a.TC, a.M);
  if (need > kNoAllocGemmBytes)
    return fail(Q4NX_E_WORKSPACE, "gemm_block_noalloc: this call needs %zu bytes of scratch, the static "
                "array holds %zu", need, kNoAllocGemmBytes);
  void* ws = nullptr;
  if (need) {
    const int s2 = scratch_address(&ws);
    if (s2) return s2;
    k_clear_words<<<1, 256, 0, static_cast<hipStream_t>(stream)>>>(static_cast<uint32_t*>(ws), kHeaderZeroWords);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return hip_status(e, "gemm_block_noalloc: clearing the scratch header");
  }
  const int r = gemm_launch(a, kind_of(w), ws, need, stream, "gemm_block_noalloc", false);
  return r ? r : ok();
}

size_t q4nx_gemm_block_ws(const q4nx_weight* w) {
  if (check_weight(w, "gemm_block_ws")) return 0;
  const int TR = (int)(w->rows / 32);
  return q4nx::gemm_ws_bytes_any_m(&TR, 1, (int)(w->cols / 256));
}

int q4nx_gemm_batched(const q4nx_gemm_job* jobs, int n_jobs, const uint16_t* X, int M, void* ws,
                      size_t ws_bytes, void* stream) {
  if (!jobs) return fail(Q4NX_E_ARG, "gemm_batched: null job array");
  if (n_jobs < 1 || n_jobs > Q4NX_GEMM_BATCH_MAX_JOBS)
    return fail(Q4NX_E_ARG, "gemm_batched: %d jobs outside 1..%d", n_jobs, (int)Q4NX_GEMM_BATCH_MAX_JOBS);
  const q4nx_weight* w[Q4NX_GEMM_BATCH_MAX_JOBS];
  float* Y[Q4NX_GEMM_BATCH_MAX_JOBS];
  for (int i = 0; i < n_jobs; ++i) {
    w[i] = &jobs[i].w;
    Y[i] = jobs[i].Y;
  }
  q4nx::GemmArgs a;
  const int st = gemm_setup(w, Y, n_jobs, X, M, "gemm_batched", a);
  if (st) return st;
  const int r = gemm_launch(a, kind_of(w[0]), ws, ws_bytes, stream, "gemm_batched");
  return r ? r : ok();
}

int q4nx_gemm_exchange_mode(int mode) {
  if (mode < 0 || mode > 2) return fail(Q4NX_E_ARG, "gemm_exchange_mode: %d is not 0, 1 or 2", mode);
  g_gemm_exchange_mode.store(mode, std::memory_order_relaxed);
  return ok();
}

size_t q4nx_gemm_batched_ws(const q4nx_gemm_job* jobs, int n_jobs) {
  if (!jobs || n_jobs < 1 || n_jobs > Q4NX_GEMM_BATCH_MAX_JOBS) {
    fail(Q4NX_E_ARG, "gemm_batched_ws: bad job array");
    return 0;
  }
  int TR[Q4NX_GEMM_BATCH_MAX_JOBS];
  for (int i = 0; i < n_jobs; ++i) {
    if (check_weight(&jobs[i].w, "gemm_batched_ws")) return 0;
    TR[i] = (int)(jobs[i].w.rows / 32);
  }
  return q4nx::gemm_ws_bytes_any_m(TR, n_jobs, (int)(jobs[0].w.cols / 256));
}

// ---------------------------------------------------------------------------
// plans
// ---------------------------------------------------------------------------
}  // extern "C"

struct q4nx_plan_s {
  struct Seg {
    int kind, grid;
    bool step = false;   // the step kernel (static schedule) instead of the unit-dealing one
    size_t lds = 0;
    q4nx::PlanArgs args;
    q4nx::StepArgs sargs;
  };
  int M = 1;
  int mode = 0;          // 0: one GEMV launch per phase; 1: one persistent launch per segment
  std::vector<Seg> segs;
  struct Phase {         // mode 0: one batched GEMV launch over a device job table
    int kind, waves, xl, n_wg;
    q4nx::GemvBatch b;
  };
  std::vector<Phase> phases;
  void* dev = nullptr;
  size_t bytes = 0;
  std::vector<uint32_t*> ctl;   // per segment control words (device)
};

namespace {

constexpr int kPlanSpinLimit = 1 << 22;

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

extern "C" {

int q4nx_plan_create(const q4nx_gemv_job* jobs, const int32_t* phase, int n_jobs, int M,
                     q4nx_plan* out) {
  if (!jobs || !phase || !out) return fail(Q4NX_E_ARG, "plan: null jobs, phase or out");
  *out = nullptr;
  if (n_jobs < 1 || n_jobs > 65536)
    return fail(Q4NX_E_ARG, "plan: %d jobs outside 1..65536", n_jobs);
  if (M < 1 || M > 4) return fail(Q4NX_E_ARG, "plan: M = %d outside 1..4", M);
  for (int i = 0; i < n_jobs; ++i) {
    char name[40];
    snprintf(name, sizeof name, "plan job %d", i);
    const int st = check_gemv_io(&jobs[i].w, jobs[i].x, jobs[i].y, M, name);
    if (st) return st;
    if (phase[i] < 0) return fail(Q4NX_E_ARG, "plan job %d: negative phase", i);
  }
  std::vector<int> order(n_jobs);
  for (int i = 0; i < n_jobs; ++i) order[i] = i;
  std::stable_sort(order.begin(), order.end(), [&](int a, int b) { return phase[a] < phase[b]; });
  // segments: maximal runs of phases whose jobs share one kind
  struct SegH {
    int kind;
    std::vector<int> jobs;
    std::vector<int> phase_of;   // local phase of each job
    int n_phases;
  };
  std::vector<SegH> segs;
  for (size_t t = 0; t < order.size();) {
    const int ph = phase[order[t]];
    const int kind = kind_of(&jobs[order[t]].w);
    size_t e = t;
    while (e < order.size() && phase[order[e]] == ph) {
      if (kind_of(&jobs[order[e]].w) != kind)
        return fail(Q4NX_E_CHUNK_KIND, "plan: phase %d mixes chunk kinds", ph);
      ++e;
    }
    if (segs.empty() || segs.back().kind != kind) segs.push_back({kind, {}, {}, 0});
    SegH& sg = segs.back();
    for (size_t i = t; i < e; ++i) {
      sg.jobs.push_back(order[i]);
      sg.phase_of.push_back(sg.n_phases);
    }
    ++sg.n_phases;
    t = e;
  }
  int n_cu = 0;
  {
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&n_cu, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return hip_status(e, "plan device query");
  }
  // q4 segments whose activations fit the step kernel's LDS run on it
  struct StepT {
    bool use = false;
    size_t lds = 0, rec = 0;
    int ns = 0;
    std::vector<q4nx::StepJob> sj;
    std::vector<q4nx::StepUnit> units;
    std::vector<int32_t> first;
    size_t o_jobs = 0, o_units = 0, o_first = 0, o_sync = 0, o_ctl = 0;
  };
  std::vector<StepT> steps(segs.size());
  for (size_t si = 0; si < segs.size(); ++si) {
    SegH& sg = segs[si];
    if (sg.kind != q4nx::KIND_Q4_1 && sg.kind != q4nx::KIND_Q4_K) continue;
    int max_tc = 0;
    for (int ji : sg.jobs) max_tc = std::max(max_tc, (int)(jobs[ji].w.cols / 256));
    const q4nx::StepLds lds = q4nx::step_lds(M, max_tc);
    if (lds.ns < 2) continue;
    StepT& S = steps[si];
    S.use = true;
    S.lds = lds.total;
    S.rec = lds.rec;
    S.ns = lds.ns;
    for (int ji : sg.jobs) {
      const q4nx_gemv_job& j = jobs[ji];
      S.sj.push_back({static_cast<const uint8_t*>(j.w.chunks), j.x, j.y, (int32_t)(j.w.rows / 32),
                      (int32_t)(j.w.cols / 256), (int32_t)j.w.cols, (int32_t)j.w.rows});
    }
    // whole tile rows to workgroups, largest first, each to the least loaded in
    // its phase (then overall); a workgroup's rows in (job, row) order, cut into
    // pieces of at most kStepPieceCols chunk columns
    const int cap = q4nx::kStepPieceCols;
    std::vector<std::vector<q4nx::StepUnit>> per(n_cu);
    std::vector<long long> total(n_cu, 0);
    for (int ph = 0; ph < sg.n_phases; ++ph) {
      struct Row { int cost, job, tr; };
      std::vector<Row> rows;
      for (size_t i = 0; i < sg.jobs.size(); ++i)
        if (sg.phase_of[i] == ph)
          for (int tr = 0; tr < S.sj[i].TR; ++tr) rows.push_back({S.sj[i].TC, (int)i, tr});
      std::stable_sort(rows.begin(), rows.end(), [](const Row& a, const Row& b) { return a.cost > b.cost; });
      typedef std::tuple<long long, long long, int> Key;
      std::priority_queue<Key, std::vector<Key>, std::greater<Key>> heap;
      for (int b = 0; b < n_cu; ++b) heap.push(Key(0, total[b], b));
      std::vector<std::vector<Row>> mine(n_cu);
      for (const Row& r : rows) {
        Key k = heap.top();
        heap.pop();
        const int b = std::get<2>(k);
        mine[b].push_back(r);
        total[b] += r.cost;
        heap.push(Key(std::get<0>(k) + r.cost, total[b], b));
      }
      for (int b = 0; b < n_cu; ++b) {
        std::sort(mine[b].begin(), mine[b].end(),
                  [](const Row& a, const Row& c) { return a.job != c.job ? a.job < c.job : a.tr < c.tr; });
        for (const Row& r : mine[b]) {
          const int TC = S.sj[r.job].TC, n_sub = (TC + cap - 1) / cap;
          for (int t = 0; t < n_sub; ++t) {
            q4nx::StepUnit u;
            u.job = r.job;
            u.tr = r.tr;
            u.c0 = (int16_t)(t * TC / n_sub);
            u.c1 = (int16_t)((t + 1) * TC / n_sub);
            u.phase = (int16_t)ph;
            u.flags = (int16_t)((t == 0 ? q4nx::kStepFirst : 0) | (t == n_sub - 1 ? q4nx::kStepLast : 0));
            per[b].push_back(u);
          }
        }
      }
    }
    S.first.push_back(0);
    for (int b = 0; b < n_cu; ++b) {
      S.units.insert(S.units.end(), per[b].begin(), per[b].end());
      S.first.push_back((int32_t)S.units.size());
    }
  }
  // mode 0: every phase as one batched GEMV launch whose jobs come from a
  // device table (no limit on their number), shaped as q4nx_gemv_batched
  // shapes one kind's jobs
  struct PhaseT {
    int kind;
    BatchShape sh;
    int n_wg;
    std::vector<q4nx::GemvJob> jobs;
    std::vector<int32_t> wg_job;
    size_t o_jobs = 0, o_wg = 0;
  };
  std::vector<PhaseT> pts;
  for (size_t t = 0; t < order.size();) {
    const int ph = phase[order[t]];
    size_t e = t;
    int64_t total_tr = 0;
    int max_tc = 0;
    while (e < order.size() && phase[order[e]] == ph) {
      total_tr += jobs[order[e]].w.rows / 32;
      max_tc = std::max(max_tc, jobs[order[e]].w.cols / 256);
      ++e;
    }
    PhaseT P;
    P.kind = kind_of(&jobs[order[t]].w);
    P.sh = batch_shape(P.kind, total_tr, max_tc, M);
    int wg = 0;
    for (size_t i = t; i < e; ++i) {
      q4nx::GemvJob g;
      const int n = fill_job(g, &jobs[order[i]], P.sh, total_tr, wg);
      for (int b = 0; b < n; ++b) P.wg_job.push_back((int32_t)P.jobs.size());
      P.jobs.push_back(g);
      wg += n;
    }
    P.n_wg = wg;
    pts.push_back(std::move(P));
    t = e;
  }
  // host tables and device layout
  struct SegT {
    std::vector<q4nx::PlanJob> pj;
    std::vector<int32_t> unit_job;
    std::vector<uint32_t> need;
    int n_slots = 0, smax = 1;
    size_t o_jobs, o_unit, o_need, o_done, o_cnt, o_part, o_ctl;
  };
  std::vector<SegT> tabs(segs.size());
  size_t total = 0;
  for (size_t si = 0; si < segs.size(); ++si) {
    SegH& sg = segs[si];
    SegT& T = tabs[si];
    T.need.assign(sg.n_phases, 0);
    const int cpw = q4nx::plan_cpw(sg.kind);
    int units = 0;
    for (size_t i = 0; i < sg.jobs.size(); ++i) {
      const q4nx_gemv_job& j = jobs[sg.jobs[i]];
      q4nx::PlanJob p;
      p.w = static_cast<const uint8_t*>(j.w.chunks);
      p.x = j.x;
      p.y = j.y;
      p.TR = j.w.rows / 32;
      p.TC = j.w.cols / 256;
      p.ldx = j.w.cols;
      p.ldy = j.w.rows;
      p.S = (p.TC + 4 * cpw - 1) / (4 * cpw);
      p.unit0 = units;
      p.phase = sg.phase_of[i];
      p.slot0 = 0;
      if (p.S > 1) {
        p.slot0 = T.n_slots;
        T.n_slots += p.TR;
        T.smax = std::max(T.smax, p.S);
      }
      T.need[p.phase] += (uint32_t)p.TR;
      for (int u = 0; u < p.TR * p.S; ++u) T.unit_job.push_back((int32_t)i);
      units += p.TR * p.S;
      T.pj.push_back(p);
    }
    T.o_jobs = total;  total = align256(total + T.pj.size() * sizeof(q4nx::PlanJob));
    T.o_unit = total;  total = align256(total + T.unit_job.size() * 4);
    T.o_need = total;  total = align256(total + T.need.size() * 4);
    T.o_done = total;  total = align256(total + T.need.size() * 4);
    T.o_cnt = total;   total = align256(total + (size_t)std::max(T.n_slots, 1) * 4);
    T.o_part = total;  total = align256(total + (size_t)T.n_slots * T.smax * 32 * M * 4);
    T.o_ctl = total;   total = align256(total + 16);
    StepT& S = steps[si];
    if (S.use) {
      S.o_jobs = total;  total = align256(total + S.sj.size() * sizeof(q4nx::StepJob));
      S.o_units = total; total = align256(total + S.units.size() * sizeof(q4nx::StepUnit));
      S.o_first = total; total = align256(total + S.first.size() * 4);
      S.o_sync = total;  total = align256(total + q4nx::step_sync_words(segs[si].n_phases) * 4);
      S.o_ctl = total;   total = align256(total + 16);
    }
  }
  for (PhaseT& P : pts) {
    P.o_jobs = total; total = align256(total + P.jobs.size() * sizeof(q4nx::GemvJob));
    P.o_wg = total;   total = align256(total + P.wg_job.size() * 4);
  }
  // check every kernel can be resident before allocating anything
  std::vector<int> grids(segs.size());
  for (size_t si = 0; si < segs.size(); ++si) {
    int blocks = 0;
    const hipError_t e = q4nx::plan_resident_blocks(segs[si].kind, M, &blocks);
    if (e != hipSuccess) return hip_status(e, "plan occupancy");
    if (blocks < 1) return fail(Q4NX_E_HIP, "plan: kernel cannot be resident");
    grids[si] = std::min(blocks, (int)tabs[si].unit_job.size());
  }
  void* dev = nullptr;
  hipError_t e = hipMalloc(&dev, total);
  if (e != hipSuccess) return hip_status(e, "plan allocation");
  std::vector<uint8_t> host(total, 0);
  for (size_t si = 0; si < segs.size(); ++si) {
    SegT& T = tabs[si];
    memcpy(host.data() + T.o_jobs, T.pj.data(), T.pj.size() * sizeof(q4nx::PlanJob));
    memcpy(host.data() + T.o_unit, T.unit_job.data(), T.unit_job.size() * 4);
    memcpy(host.data() + T.o_need, T.need.data(), T.need.size() * 4);
    const StepT& S = steps[si];
    if (S.use) {
      memcpy(host.data() + S.o_jobs, S.sj.data(), S.sj.size() * sizeof(q4nx::StepJob));
      memcpy(host.data() + S.o_units, S.units.data(), S.units.size() * sizeof(q4nx::StepUnit));
      memcpy(host.data() + S.o_first, S.first.data(), S.first.size() * 4);
    }
  }
  for (const PhaseT& P : pts) {
    memcpy(host.data() + P.o_jobs, P.jobs.data(), P.jobs.size() * sizeof(q4nx::GemvJob));
    memcpy(host.data() + P.o_wg, P.wg_job.data(), P.wg_job.size() * 4);
  }
  e = hipMemcpy(dev, host.data(), total, hipMemcpyHostToDevice);
  if (e != hipSuccess) {
    (void)hipFree(dev);
    return hip_status(e, "plan upload");
  }
  q4nx_plan_s* plan = new q4nx_plan_s;
  plan->M = M;
  plan->dev = dev;
  plan->bytes = total;
  uint8_t* d = static_cast<uint8_t*>(dev);
  for (size_t si = 0; si < segs.size(); ++si) {
    SegT& T = tabs[si];
    q4nx_plan_s::Seg s;
    s.kind = segs[si].kind;
    s.grid = grids[si];
    s.args.jobs = reinterpret_cast<const q4nx::PlanJob*>(d + T.o_jobs);
    s.args.unit_job = reinterpret_cast<const int32_t*>(d + T.o_unit);
    s.args.need = reinterpret_cast<const uint32_t*>(d + T.o_need);
    s.args.done = reinterpret_cast<uint32_t*>(d + T.o_done);
    s.args.row_cnt = reinterpret_cast<uint32_t*>(d + T.o_cnt);
    s.args.partial = reinterpret_cast<float*>(d + T.o_part);
    s.args.ctl = reinterpret_cast<uint32_t*>(d + T.o_ctl);
    s.args.n_units = (int32_t)T.unit_job.size();
    s.args.n_phases = segs[si].n_phases;
    s.args.spin_limit = kPlanSpinLimit;
    s.args.smax = T.smax;
    const StepT& S = steps[si];
    if (S.use) {
      s.step = true;
      s.grid = n_cu;
      s.lds = S.lds;
      s.sargs.jobs = reinterpret_cast<const q4nx::StepJob*>(d + S.o_jobs);
      s.sargs.units = reinterpret_cast<const q4nx::StepUnit*>(d + S.o_units);
      s.sargs.wg_first = reinterpret_cast<const int32_t*>(d + S.o_first);
      s.sargs.sync = reinterpret_cast<uint32_t*>(d + S.o_sync);
      s.sargs.ctl = reinterpret_cast<uint32_t*>(d + S.o_ctl);
      s.sargs.n_phases = segs[si].n_phases;
      s.sargs.spin_limit = kPlanSpinLimit;
      s.sargs.ring_off = (int32_t)S.rec;
      s.sargs.ns = S.ns;
      s.args.ctl = s.sargs.ctl;
    }
    plan->segs.push_back(s);
    plan->ctl.push_back(s.args.ctl);
  }
  for (const PhaseT& P : pts) {
    q4nx_plan_s::Phase ph;
    ph.kind = P.kind;
    ph.waves = P.sh.waves;
    ph.xl = P.sh.xl;
    ph.n_wg = P.n_wg;
    memset(&ph.b, 0, sizeof ph.b);
    ph.b.sl = 4 / P.sh.parts;
    ph.b.tab = reinterpret_cast<const q4nx::GemvJob*>(d + P.o_jobs);
    ph.b.tab_wg = reinterpret_cast<const int32_t*>(d + P.o_wg);
    plan->phases.push_back(ph);
  }
  *out = plan;
  return ok();
}

int q4nx_plan_set_mode(q4nx_plan plan, int mode) {
  if (!plan) return fail(Q4NX_E_ARG, "plan_set_mode: null plan");
  if (mode != 0 && mode != 1) return fail(Q4NX_E_ARG, "plan_set_mode: mode %d is neither 0 nor 1", mode);
  plan->mode = mode;
  return ok();
}

int q4nx_plan_run(q4nx_plan plan, void* stream) {
  if (!plan) return fail(Q4NX_E_ARG, "plan_run: null plan");
  if (plan->mode == 0) {
    for (const auto& ph : plan->phases) {
      const hipError_t e = q4nx::launch_gemv(ph.kind, plan->M, ph.waves, ph.b, ph.n_wg, ph.xl,
                                             static_cast<hipStream_t>(stream));
      if (e != hipSuccess) return hip_status(e, "plan phase launch");
    }
    return ok();
  }
  for (const auto& s : plan->segs) {
    const hipError_t e = s.step ? q4nx::launch_step(s.kind, plan->M, s.sargs, s.grid, s.lds,
                                                    static_cast<hipStream_t>(stream))
                                : q4nx::launch_plan(s.kind, plan->M, s.args, s.grid,
                                                    static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_status(e, "plan launch");
  }
  return ok();
}

int q4nx_plan_errors(q4nx_plan plan, uint32_t* flags) {
  if (!plan || !flags) return fail(Q4NX_E_ARG, "plan_errors: null argument");
  uint32_t acc = 0;
  for (uint32_t* c : plan->ctl) {
    uint32_t v = 0;
    hipError_t e = hipMemcpy(&v, c + 1, 4, hipMemcpyDeviceToHost);
    if (e != hipSuccess) return hip_status(e, "plan_errors read");
    acc |= v;
    if (v) {
      const uint32_t zero = 0;
      e = hipMemcpy(c + 1, &zero, 4, hipMemcpyHostToDevice);
      if (e != hipSuccess) return hip_status(e, "plan_errors clear");
    }
  }
  *flags = acc;
  return ok();
}

size_t q4nx_plan_bytes(q4nx_plan plan) { return plan ? plan->bytes : 0; }

void q4nx_plan_destroy(q4nx_plan plan) {
  if (!plan) return;
  if (plan->dev) (void)hipFree(plan->dev);
  delete plan;
}

// ---------------------------------------------------------------------------
// MoE
// ---------------------------------------------------------------------------
static int check_arena(const void* base, int64_t stride, int64_t bytes, int n, int64_t need,
                       const char* name) {
  if (!base) return fail(Q4NX_E_ARG, "moe: null %s arena", name);
  if (!aligned(base, 16) || stride % 16)
    return fail(Q4NX_E_ALIGN, "moe: %s arena or stride not 16-byte aligned", name);
  if (stride < need) return fail(Q4NX_E_SHAPE, "moe: %s stride %lld below one expert's %lld bytes",
                                 name, (long long)stride, (long long)need);
  const int64_t total = (int64_t)(n - 1) * stride + need;
  if (bytes < total)
    return fail(Q4NX_E_SHORT, "moe: %s arena holds %lld bytes, %d experts need %lld", name,
                (long long)bytes, n, (long long)total);
  return Q4NX_OK;
}

static int check_moe_layer(const q4nx_moe_layer* L) {
  if (!L) return fail(Q4NX_E_ARG, "moe: null layer");
  if (L->n_experts < 1 || L->n_experts >= (1 << 19))
    return fail(Q4NX_E_ARG, "moe: n_experts = %d outside 1..524287", L->n_experts);
  if (L->chunk_bytes != Q4NX_Q4_1_BYTES && L->chunk_bytes != Q4NX_Q4_K_BYTES)
    return fail(Q4NX_E_CHUNK_KIND, "moe: experts must be q4_1 (5120) or Q4_K (4736), got %d",
                L->chunk_bytes);
  if (L->d_model <= 0 || L->d_model % 256 || L->d_expert <= 0 || L->d_expert % 256 ||
      L->d_shared < 0 || L->d_shared % 256)
    return fail(Q4NX_E_SHAPE, "moe: d_model, d_expert, d_shared must be multiples of 256 "
                "(d_shared may be 0), got %d, %d, %d", L->d_model, L->d_expert, L->d_shared);
  if (L->d_model > (1 << 20) || L->d_expert > (1 << 20) || L->d_shared > (1 << 20))
    return fail(Q4NX_E_SHAPE, "moe: d_model, d_expert, d_shared must be at most 1048576, got %d, %d, %d",
                L->d_model, L->d_expert, L->d_shared);
  const int64_t cb = L->chunk_bytes;
  const int64_t gu = (int64_t)(L->d_expert / 32) * (L->d_model / 256) * cb;
  const int64_t dn = (int64_t)(L->d_model / 32) * (L->d_expert / 256) * cb;
  int st = check_arena(L->gate, L->gate_stride, L->gate_bytes, L->n_experts, gu, "gate");
  if (!st) st = check_arena(L->up, L->up_stride, L->up_bytes, L->n_experts, gu, "up");
  if (!st) st = check_arena(L->down, L->down_stride, L->down_bytes, L->n_experts, dn, "down");
  if (st) return st;
  if (L->d_shared) {
    const q4nx_weight* sw[3] = {&L->sh_gate, &L->sh_up, &L->sh_down};
    const char* nm[3] = {"moe shared gate", "moe shared up", "moe shared down"};
    for (int i = 0; i < 3; ++i) {
      st = check_weight(sw[i], nm[i]);
      if (st) return st;
      if (sw[i]->chunk_bytes != L->chunk_bytes)
        return fail(Q4NX_E_CHUNK_KIND, "%s: kind differs from the routed experts'", nm[i]);
      const int rows = i < 2 ? L->d_shared : L->d_model;
      const int cols = i < 2 ? L->d_model : L->d_shared;
      if (sw[i]->rows != rows || sw[i]->cols != cols)
        return fail(Q4NX_E_SHAPE, "%s: %d x %d, expected %d x %d", nm[i], sw[i]->rows,
                    sw[i]->cols, rows, cols);
    }
  }
  return Q4NX_OK;
}

static int moe_hstride(const q4nx_moe_layer* L) {
  return L->d_expert > L->d_shared ? L->d_expert : L->d_shared;
}

size_t q4nx_moe_ws(const q4nx_moe_layer* L, int T, int k) {
  if (check_moe_layer(L) || T < 1 || k < 1 || T > 4096 || k > q4nx::kMoeMaxK || T * k > q4nx::kMoeMaxPairs)
    return 0;
  return q4nx::moe_ws_layout(T * k, T, L->d_model, moe_hstride(L)).total;
}

int q4nx_moe_experts(const q4nx_moe_layer* L, const uint16_t* X, const int32_t* ids,
                     const float* p, int T, int k, float* Y, const q4nx_moe_debug* dbg, void* ws,
                     size_t ws_bytes, void* stream) {
  int st = check_moe_layer(L);
  if (st) return st;
  if (!X || !ids || !p || !Y) return fail(Q4NX_E_ARG, "moe: null X, ids, p or Y");
  if (T < 1 || T > 4096 || k < 1 || k > q4nx::kMoeMaxK || T * k > q4nx::kMoeMaxPairs)
    return fail(Q4NX_E_ARG, "moe: T = %d, k = %d outside T 1..4096, k 1..16, T*k <= %d", T, k,
                q4nx::kMoeMaxPairs);
  if (!aligned(X, 16) || !aligned(ids, 4) || !aligned(p, 4) || !aligned(Y, 4))
    return fail(Q4NX_E_ALIGN, "moe: X must be 16-byte, ids/p/Y 4-byte aligned");
  {
    // a batch's prepared activation records (576 bytes per token and tile
    // column, of x for gate/up and of h for down) are staged in at most 64 KB
    // of LDS
    const int tb = T == 1 ? 1 : 4;
    const int inner = std::max(L->d_expert, L->d_shared);
    const int max_d = 65536 / (tb * q4nx::kMoeRecGateUp) * 256;
    const int max_inner = 65536 / (tb * q4nx::kMoeRecDown) * 256;
    if (L->d_model > max_d || inner > max_inner)
      return fail(Q4NX_E_SHAPE, "moe: for T = %d, d_model must be at most %d and d_expert, d_shared at most %d",
                  T, max_d, max_inner);
  }
  const q4nx::MoeWsLayout lay = q4nx::moe_ws_layout(T * k, T, L->d_model, moe_hstride(L));
  if (!ws || ws_bytes < lay.total)
    return fail(Q4NX_E_WORKSPACE, "moe: workspace of %zu bytes, %zu needed", ws_bytes, lay.total);
  if (!aligned(ws, 256)) return fail(Q4NX_E_ALIGN, "moe: workspace not 256-byte aligned");

  q4nx::MoeArgs a;
  memset(&a, 0, sizeof a);
  a.gate = static_cast<const uint8_t*>(L->gate);
  a.up = static_cast<const uint8_t*>(L->up);
  a.down = static_cast<const uint8_t*>(L->down);
  a.gate_stride = L->gate_stride;
  a.up_stride = L->up_stride;
  a.down_stride = L->down_stride;
  if (L->d_shared) {
    a.sgate = static_cast<const uint8_t*>(L->sh_gate.chunks);
    a.sup = static_cast<const uint8_t*>(L->sh_up.chunks);
    a.sdown = static_cast<const uint8_t*>(L->sh_down.chunks);
  }
  a.n_experts = L->n_experts;
  a.D = L->d_model;
  a.De = L->d_expert;
  a.Ds = L->d_shared;
  a.X = X;
  a.ids = ids;
  a.p = p;
  a.Y = Y;
  a.T = T;
  a.k = k;
  a.tb = T == 1 ? 1 : 4;
  a.hstride = moe_hstride(L);
  a.hot_min = L->hot_tokens > 0 ? L->hot_tokens : 0;
  if (dbg) {
    a.dbg_h = dbg->h;
    a.dbg_d = dbg->d;
    a.dbg_h_shared = dbg->h_shared;
    a.dbg_d_shared = dbg->d_shared;
  }
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.hdr = reinterpret_cast<uint32_t*>(w + lay.hdr);
  a.sorted = reinterpret_cast<int32_t*>(w + lay.sorted);
  a.seg = reinterpret_cast<int32_t*>(w + lay.seg);
  a.batch0 = reinterpret_cast<int32_t*>(w + lay.batch0);
  a.btab = reinterpret_cast<int32_t*>(w + lay.btab);
  a.hot = reinterpret_cast<int32_t*>(w + lay.hot);
  a.hbuf = reinterpret_cast<float*>(w + lay.hbuf);
  a.dbuf = reinterpret_cast<float*>(w + lay.dbuf);
  const hipError_t e = q4nx::launch_moe(L->chunk_bytes == Q4NX_Q4_1_BYTES ? q4nx::KIND_Q4_1
                                                                          : q4nx::KIND_Q4_K,
                                        a, static_cast<hipStream_t>(stream));
  return hip_status(e, "moe launch");
}

// ---------------------------------------------------------------------------
// decoders
// ---------------------------------------------------------------------------
int q4nx_unpack(const q4nx_weight* w, uint8_t* codes, uint16_t* meta0, uint16_t* meta1,
                uint16_t* row_meta, void* stream) {
  int st = check_weight(w, "unpack");
  if (st) return st;
  if (!codes || !meta0) return fail(Q4NX_E_ARG, "unpack: null codes or meta0");
  if (!aligned(meta0, 2) || (meta1 && !aligned(meta1, 2)) || (row_meta && !aligned(row_meta, 2)))
    return fail(Q4NX_E_ALIGN, "unpack: metadata outputs must be 2-byte aligned");
  const hipError_t e = q4nx::launch_unpack(kind_of(w), static_cast<const uint8_t*>(w->chunks),
                                           w->rows / 32, w->cols / 256, codes, meta0, meta1,
                                           row_meta, static_cast<hipStream_t>(stream));
  return hip_status(e, "unpack launch");
}

int q4nx_repack_q4k_to_q41(const q4nx_weight* w, void* out, size_t out_bytes, void* stream) {
  int st = check_weight(w, "repack");
  if (st) return st;
  if (w->chunk_bytes != Q4NX_Q4_K_BYTES)
    return fail(Q4NX_E_CHUNK_KIND, "repack: input must be Q4_K (4736-byte chunks), got %d", w->chunk_bytes);
  if (!out) return fail(Q4NX_E_ARG, "repack: null output");
  if (!aligned(out, 16)) return fail(Q4NX_E_ALIGN, "repack: output not 16-byte aligned");
  const int64_t tiles = (int64_t)(w->rows / 32) * (w->cols / 256);
  if (out_bytes < (size_t)tiles * Q4NX_Q4_1_BYTES)
    return fail(Q4NX_E_SHORT, "repack: output holds %zu bytes, %lld needed", out_bytes,
                (long long)(tiles * Q4NX_Q4_1_BYTES));
  if (tiles > 0x7FFFFFFF) return fail(Q4NX_E_SHAPE, "repack: too many tiles");
  const hipError_t e = q4nx::launch_repack_q4k(static_cast<const uint8_t*>(w->chunks), (int)tiles,
                                               static_cast<uint8_t*>(out), static_cast<hipStream_t>(stream));
  return hip_status(e, "repack launch");
}

static_assert(sizeof(q4nx_chunk_layout) == sizeof(q4nx::ChunkLayout), "layout descriptor");

int q4nx_chunk_layout_default(int chunk_bytes, q4nx_chunk_layout* out) {
  if (!out) return fail(Q4NX_E_ARG, "chunk_layout_default: null output");
  if (chunk_bytes != Q4NX_Q4_1_BYTES && chunk_bytes != Q4NX_Q4_K_BYTES)
    return fail(Q4NX_E_CHUNK_KIND, "chunk_layout_default: %d is not 5120 (q4_1) or 4736 (Q4_K)", chunk_bytes);
  q4nx_chunk_layout L;
  memset(&L, 0, sizeof L);
  L.chunk_bytes = chunk_bytes;
  L.code_off = 0; L.code_row = 128; L.code_group = 16; L.code_step = 1;
  L.code_pairing = 0; L.code_high_first = 0;
  if (chunk_bytes == Q4NX_Q4_1_BYTES) {
    L.f0_off = 4096; L.f0_row = 32; L.f0_group = 4;
    L.f1_off = 4098; L.f1_row = 32; L.f1_group = 4;
  } else {
    L.f0_off = 4096; L.f0_row = 16; L.f0_group = 2;
    L.f1_off = 4097; L.f1_row = 16; L.f1_group = 2;
    L.s_off = 4608; L.s_row = 4;
    L.m_off = 4610; L.m_row = 4;
  }
  *out = L;
  return ok();
}

int q4nx_chunk_layout_check(const q4nx_chunk_layout* L) {
  if (!L) return fail(Q4NX_E_ARG, "chunk_layout_check: null layout");
  const int CB = L->chunk_bytes;
  if (CB != Q4NX_Q4_1_BYTES && CB != Q4NX_Q4_K_BYTES)
    return fail(Q4NX_E_CHUNK_KIND, "chunk_layout: chunk size %d is not 5120 (q4_1) or 4736 (Q4_K)", CB);
  if (L->code_pairing != 0 && L->code_pairing != 1)
    return fail(Q4NX_E_ARG, "chunk_layout: code_pairing %d is not 0 or 1", L->code_pairing);
  std::vector<uint8_t> used(CB, 0);
  // a field of `len` bytes at `off`: inside the chunk and on bytes nothing else uses
  auto mark = [&](int64_t off, int len, const char* what, int r, int g) -> int {
    if (off < 0 || off + len > CB)
      return fail(Q4NX_E_ARG, "chunk_layout: %s of row %d, group %d at byte %lld leaves the %d-byte chunk",
                  what, r, g, (long long)off, CB);
    for (int i = 0; i < len; ++i)
      if (used[off + i]++)
        return fail(Q4NX_E_ARG, "chunk_layout: %s of row %d, group %d shares byte %lld with another field",
                    what, r, g, (long long)(off + i));
    return Q4NX_OK;
  };
  for (int r = 0; r < 32; ++r)
    for (int g = 0; g < 8; ++g) {
      for (int b = 0; b < 16; ++b) {   // each code byte holds two codes: mark it once
        const int st = mark((int64_t)L->code_off + (int64_t)r * L->code_row + (int64_t)g * L->code_group +
                                (int64_t)b * L->code_step, 1, "a code byte", r, g);
        if (st) return st;
      }
      const int fl = CB == Q4NX_Q4_1_BYTES ? 2 : 1;
      int st = mark((int64_t)L->f0_off + (int64_t)r * L->f0_row + (int64_t)g * L->f0_group, fl, "field 0", r, g);
      if (!st) st = mark((int64_t)L->f1_off + (int64_t)r * L->f1_row + (int64_t)g * L->f1_group, fl, "field 1", r, g);
      if (st) return st;
    }
  if (CB == Q4NX_Q4_K_BYTES)
    for (int r = 0; r < 32; ++r) {
      int st = mark((int64_t)L->s_off + (int64_t)r * L->s_row, 2, "S", r, 0);
      if (!st) st = mark((int64_t)L->m_off + (int64_t)r * L->m_row, 2, "M", r, 0);
      if (st) return st;
    }
  for (int i = 0; i < CB; ++i)
    if (!used[i]) return fail(Q4NX_E_ARG, "chunk_layout: byte %d of the chunk belongs to no field", i);
  return ok();
}

int q4nx_relayout(const q4nx_chunk_layout* L, const q4nx_weight* src, void* out, size_t out_bytes, void* stream) {
  int st = q4nx_chunk_layout_check(L);
  if (st) return st;
  st = check_weight(src, "relayout");
  if (st) return st;
  if (src->chunk_bytes != L->chunk_bytes)
    return fail(Q4NX_E_CHUNK_KIND, "relayout: weight chunks of %d bytes, layout for %d", src->chunk_bytes,
                L->chunk_bytes);
  if (!out) return fail(Q4NX_E_ARG, "relayout: null output");
  if (!aligned(out, 16)) return fail(Q4NX_E_ALIGN, "relayout: output not 16-byte aligned");
  const int64_t tiles = (int64_t)(src->rows / 32) * (src->cols / 256);
  if (out_bytes < (size_t)(tiles * L->chunk_bytes))
    return fail(Q4NX_E_SHORT, "relayout: output holds %zu bytes, %lld needed", out_bytes,
                (long long)(tiles * L->chunk_bytes));
  if (tiles > 0x7FFFFFFF) return fail(Q4NX_E_SHAPE, "relayout: too many tiles");
  q4nx::ChunkLayout d;
  memcpy(&d, L, sizeof d);
  const hipError_t e = q4nx::launch_relayout(d, static_cast<const uint8_t*>(src->chunks), (int)tiles,
                                             static_cast<uint8_t*>(out), static_cast<hipStream_t>(stream));
  return hip_status(e, "relayout launch");
}

static int gguf_geometry(int gtype, int* block_bytes, int* block_cols, int* align) {
  switch (gtype) {
    case Q4NX_GGUF_Q4_0: *block_bytes = 18; *block_cols = 32; *align = 2; return 1;
    case Q4NX_GGUF_Q4_1: *block_bytes = 20; *block_cols = 32; *align = 4; return 1;
    case Q4NX_GGUF_Q4_K: *block_bytes = 144; *block_cols = 256; *align = 16; return 1;
    default: return 0;
  }
}

size_t q4nx_gguf_bytes(int gguf_type, int rows, int cols) {
  int bb, bc, al;
  if (!gguf_geometry(gguf_type, &bb, &bc, &al) || rows <= 0 || cols <= 0 || cols % bc) return 0;
  return (size_t)rows * (size_t)(cols / bc) * (size_t)bb;
}

int q4nx_gguf_to_q41(int gguf_type, const void* src, size_t src_bytes, int rows, int cols, void* out,
                     size_t out_bytes, void* stream) {
  int bb, bc, al;
  if (!gguf_geometry(gguf_type, &bb, &bc, &al))
    return fail(Q4NX_E_ARG, "gguf: type %d is not Q4_0 (2), Q4_1 (3) or Q4_K (12)", gguf_type);
  if (!src || !out) return fail(Q4NX_E_ARG, "gguf: null source or output");
  if (rows <= 0 || cols <= 0 || rows % 32 || cols % 256)
    return fail(Q4NX_E_SHAPE, "gguf: %d x %d is not a whole number of 32 x 256 tiles", rows, cols);
  const int64_t tiles = (int64_t)(rows / 32) * (cols / 256);
  if (tiles > 0x7FFFFFFF) return fail(Q4NX_E_SHAPE, "gguf: too many tiles");
  if (!aligned(src, al)) return fail(Q4NX_E_ALIGN, "gguf: source not %d-byte aligned", al);
  if (!aligned(out, 16)) return fail(Q4NX_E_ALIGN, "gguf: output not 16-byte aligned");
  const size_t need = q4nx_gguf_bytes(gguf_type, rows, cols);
  if (src_bytes < need)
    return fail(Q4NX_E_SHORT, "gguf: source holds %zu bytes, %zu needed", src_bytes, need);
  if (out_bytes < (size_t)tiles * Q4NX_Q4_1_BYTES)
    return fail(Q4NX_E_SHORT, "gguf: output holds %zu bytes, %lld needed", out_bytes,
                (long long)(tiles * Q4NX_Q4_1_BYTES));
  const hipError_t e = q4nx::launch_gguf_q41(gguf_type, static_cast<const uint8_t*>(src), rows / 32, cols / 256,
                                             static_cast<uint8_t*>(out), static_cast<hipStream_t>(stream));
  return hip_status(e, "gguf launch");
}

int q4nx_q8_rows(const q4nx_weight* w, const int32_t* ids, int T, float* out, void* stream) {
  int st = check_weight(w, "q8_rows");
  if (st) return st;
  if (w->chunk_bytes != Q4NX_Q8_BYTES)
    return fail(Q4NX_E_CHUNK_KIND, "q8_rows: weight must be Q8 (8704-byte chunks), got %d", w->chunk_bytes);
  if (!ids || !out) return fail(Q4NX_E_ARG, "q8_rows: null ids or output");
  if (T < 1 || T > 65535) return fail(Q4NX_E_ARG, "q8_rows: T = %d outside 1..65535", T);
  if (!aligned(ids, 4) || !aligned(out, 4)) return fail(Q4NX_E_ALIGN, "q8_rows: ids and out must be 4-byte aligned");
  const hipError_t e = q4nx::launch_q8_rows(kind_of(w), static_cast<const uint8_t*>(w->chunks), w->rows,
                                            w->cols / 256, ids, T, out, static_cast<hipStream_t>(stream));
  return hip_status(e, "q8_rows launch");
}

size_t q4nx_argmax_ws(int n, int M) {
  if (n < 1 || M < 1 || M > 65535) return 0;
  return (size_t)M * q4nx::argmax_parts(n) * 8;
}

int q4nx_argmax(const float* y, int n, int ldy, int M, int32_t* idx, float* val, void* ws,
                size_t ws_bytes, void* stream) {
  if (!y || !idx) return fail(Q4NX_E_ARG, "argmax: null y or idx");
  if (n < 1 || ldy < n || M < 1 || M > 65535)
    return fail(Q4NX_E_ARG, "argmax: n = %d, ldy = %d, M = %d (need 1 <= n <= ldy, 1 <= M <= 65535)", n, ldy, M);
  if (!aligned(y, 4) || !aligned(idx, 4) || (val && !aligned(val, 4)))
    return fail(Q4NX_E_ALIGN, "argmax: y, idx and val must be 4-byte aligned");
  if (ws) {
    const size_t need = q4nx_argmax_ws(n, M);
    if (ws_bytes < need)
      return fail(Q4NX_E_WORKSPACE, "argmax: workspace of %zu bytes, %zu needed", ws_bytes, need);
    if (!aligned(ws, 8)) return fail(Q4NX_E_ALIGN, "argmax: workspace not 8-byte aligned");
  }
  const hipError_t e = q4nx::launch_argmax(y, n, ldy, M, idx, val, ws, static_cast<hipStream_t>(stream));
  return hip_status(e, "argmax launch");
}

int q4nx_moe_router(const uint16_t* R, const uint16_t* X, int T, int D, int E, int k, int renorm,
                    int32_t* ids, float* p, float* logits, void* stream) {
  if (!R || !X || !ids || !p || !logits) return fail(Q4NX_E_ARG, "router: null R, X, ids, p or logits");
  if (T < 1 || T > 65535) return fail(Q4NX_E_ARG, "router: T = %d outside 1..65535", T);
  if (!(D == 512 || D == 1024 || D == 2048 || D == 4096))
    return fail(Q4NX_E_SHAPE, "router: D = %d is not 512, 1024, 2048 or 4096", D);
  if (E < 1 || E > 1024) return fail(Q4NX_E_ARG, "router: E = %d outside 1..1024", E);
  if (k < 1 || k > 16 || k > E) return fail(Q4NX_E_ARG, "router: k = %d outside 1..min(16, E)", k);
  if (!aligned(R, 16) || !aligned(X, 16) || !aligned(ids, 4) || !aligned(p, 4) || !aligned(logits, 4))
    return fail(Q4NX_E_ALIGN, "router: R and X must be 16-byte, ids/p/logits 4-byte aligned");
  const hipError_t e = q4nx::launch_moe_router(R, X, T, D, E, k, renorm ? 1 : 0, ids, p, logits,
                                               static_cast<hipStream_t>(stream));
  return hip_status(e, "router launch");
}

// ---------------------------------------------------------------------------
// low-rank adapters
// ---------------------------------------------------------------------------
}  // extern "C"

namespace {

// Whether [p, p + pn) and [q, q + qn) share a byte.
bool overlap(const void* p, uint64_t pn, const void* q, uint64_t qn) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b ? b - a < pn : a - b < qn;
}

int check_lora(const q4nx_lora* L, const char* name) {
  if (!L) return fail(Q4NX_E_ARG, "%s: null descriptor", name);
  if (!L->a || !L->b || !L->scale) return fail(Q4NX_E_ARG, "%s: null a, b or scale", name);
  if (L->n_adapters < 1 || L->n_adapters > q4nx::kLoraMaxAdapters)
    return fail(Q4NX_E_ARG, "%s: n_adapters = %d outside 1..%d", name, L->n_adapters, q4nx::kLoraMaxAdapters);
  if (L->rank < 8 || L->rank % 8 || L->rank > q4nx::kLoraMaxRank)
    return fail(Q4NX_E_SHAPE, "%s: rank %d is not a multiple of 8 in 8..%d", name, L->rank, q4nx::kLoraMaxRank);
  if (L->rows <= 0 || L->rows % 32 || L->cols <= 0 || L->cols % 256 || L->rows > (1 << 20) || L->cols > (1 << 20))
    return fail(Q4NX_E_SHAPE, "%s: %d x %d is not a whole number of 32 x 256 tiles of at most 1048576 each way",
                name, L->rows, L->cols);
  if (!aligned(L->a, 16) || !aligned(L->b, 16) || L->a_stride % 16 || L->b_stride % 16)
    return fail(Q4NX_E_ALIGN, "%s: arenas and strides must be 16-byte aligned", name);
  if (!aligned(L->scale, 4) || !aligned(L->ranks, 4))
    return fail(Q4NX_E_ALIGN, "%s: scale and ranks must be 4-byte aligned", name);
  const int64_t need[2] = {(int64_t)L->rank * L->cols * 2, (int64_t)L->rank * L->rows * 2};
  const int64_t stride[2] = {L->a_stride, L->b_stride}, bytes[2] = {L->a_bytes, L->b_bytes};
  for (int i = 0; i < 2; ++i) {
    const char which = i ? 'b' : 'a';
    if (stride[i] < need[i])
      return fail(Q4NX_E_SHAPE, "%s: %c_stride %lld below one adapter's %lld bytes", name, which,
                  (long long)stride[i], (long long)need[i]);
    if (L->n_adapters > 1 && stride[i] > (INT64_MAX - need[i]) / (L->n_adapters - 1))
      return fail(Q4NX_E_SHAPE, "%s: %c_stride %lld too large", name, which, (long long)stride[i]);
    const int64_t total = (int64_t)(L->n_adapters - 1) * stride[i] + need[i];
    if (bytes[i] < total)
      return fail(Q4NX_E_SHORT, "%s: arena %c holds %lld bytes, %d adapters need %lld", name, which,
                  (long long)bytes[i], L->n_adapters, (long long)total);
  }
  return Q4NX_OK;
}

// Whether [p, p + n) shares a byte with what a call reads of a checked table.
bool overlaps_table(const q4nx_lora& L, const void* p, uint64_t n) {
  const uint64_t others = (uint64_t)L.n_adapters - 1, e = (uint64_t)L.n_adapters * 4;
  return overlap(p, n, L.a, others * L.a_stride + (uint64_t)L.rank * L.cols * 2) ||
         overlap(p, n, L.b, others * L.b_stride + (uint64_t)L.rank * L.rows * 2) || overlap(p, n, L.scale, e) ||
         (L.ranks && overlap(p, n, L.ranks, e));
}

// Launch shape and workspace layout of a call over checked tables.
struct LoraShape {
  q4nx::LoraArgs a;
  size_t hdr, sorted, tiles, u[q4nx::kLoraMaxJobs], total;
};

// Most rows of one set of launches: the kernels address x and y by 31-bit
// offsets, so longer calls are cut, each piece after the other with the same
// workspace.
int lora_rows(const q4nx_lora* const* L, int n, int M) {
  int64_t row_bytes = (int64_t)L[0]->cols * 2;
  for (int i = 0; i < n; ++i) row_bytes = std::max(row_bytes, (int64_t)L[i]->rows * 4);
  return (int)std::min((int64_t)M, ((int64_t)1 << 31) / row_bytes);
}

// room: the rows that the workspace is laid out for, at least M.
void lora_shape(const q4nx_lora* const* L, int n, int M, int room, LoraShape& sh) {
  memset(&sh, 0, sizeof sh);
  q4nx::LoraArgs& a = sh.a;
  a.n_jobs = n;
  a.n_adapters = L[0]->n_adapters;
  a.M = M;
  a.cols = L[0]->cols;
  a.tile_rows = q4nx::lora_tile_rows(M, a.n_adapters, a.cols);
  a.max_tiles = q4nx::lora_max_tiles(M, a.n_adapters, a.tile_rows);
  const int tiles = (M + a.tile_rows - 1) / a.tile_rows;   // at least
  int groups = 0;
  int64_t rows = 0;
  for (int i = 0; i < n; ++i) {
    a.job[i].rg_begin = groups;
    groups += (L[i]->rank + q4nx::kLoraRankGroup - 1) / q4nx::kLoraRankGroup;
    rows += L[i]->rows;
  }
  // Parts of the columns.  Each part is a row of u that the expand reads again
  // for each of its ranges, so no more than give a wave two steps, than fill
  // the GPU, or than the expand loads at once.  Up to 64 rows as if each had an
  // adapter of its own, as measured: 64 rows of 9728 columns, rank 64, 17.6 us
  // with 4 parts, 19.6 with 8, 22.9 with 10; 32 rows of 14336 columns 19.7, 18.9,
  // 22.1.  Rows that share adapters get the same parts, and leave more of the GPU
  // empty (64 rows of 9728 columns, rank 64, of one adapter 12.9 us, of three
  // 13.5); more parts were not measured for them.  More rows: 4096 of 14336
  // columns, rank 64, 91 us with 3 parts, 104 with 7.
  const int steps = a.cols / q4nx::kLoraStepCols;
  const int per = q4nx::kLoraShrinkWaves * 2;
  a.split = std::max(1, std::min((steps + per - 1) / per, q4nx::kLoraMaxSplit));
  if (M <= q4nx::kLoraWaveRows) a.split = std::min(a.split, std::max(4, 256 / (M * groups)));
  else a.split = std::max(1, std::min(a.split, 256 / (std::min(a.max_tiles, 2 * tiles) * groups)));
  int max_rank = 0;
  int64_t blocks = 0;   // of 128 outputs
  for (int i = 0; i < n; ++i) {
    max_rank = std::max(max_rank, L[i]->rank);
    blocks += (L[i]->rows + 127) / 128;
  }
  // Outputs of a workgroup, a multiple of 128: as many as make one round of
  // workgroups at rank 64 and up (three a CU; 4096 x 4096, rank 64: 77 us a call,
  // 81 with two rounds, 88 with three), where summing u costs most, and two
  // below (4096 x 14336, rank 32: 122 us, 129 with one).
  const int64_t slots = max_rank <= 32 || a.tile_rows == 16 ? 2048 : 768;
  a.n_range = 128 * (int)((a.max_tiles * blocks + slots - 1) / slots);
  while (rows / a.n_range > 32768) a.n_range *= 2;   // grid limit
  int wg = 0;
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  size_t o = 256;
  sh.sorted = o;
  o = up(o + q4nx::lora_places(room, a.n_adapters) * 4);
  sh.tiles = o;
  o = up(o + q4nx::lora_tiles(room, a.n_adapters) * sizeof(q4nx::LoraTile));
  for (int i = 0; i < n; ++i) {
    a.job[i].wg_begin = wg;
    wg += (L[i]->rows + a.n_range - 1) / a.n_range;
    sh.u[i] = o;
    o = up(o + q4nx::lora_u_rows(room) * L[i]->rank * 4);
  }
  sh.total = o;
}

int check_lora_jobs(const q4nx_lora_job* jobs, int n, int M, const char* name) {
  if (!jobs) return fail(Q4NX_E_ARG, "%s: null job array", name);
  if (n < 1 || n > Q4NX_LORA_BATCH_MAX_JOBS)
    return fail(Q4NX_E_ARG, "%s: %d jobs outside 1..%d", name, n, (int)Q4NX_LORA_BATCH_MAX_JOBS);
  if (M < 1 || M > Q4NX_LORA_MAX_M)
    return fail(Q4NX_E_ARG, "%s: M = %d outside 1..%d", name, M, (int)Q4NX_LORA_MAX_M);
  for (int i = 0; i < n; ++i) {
    char job[64];
    snprintf(job, sizeof job, "%s job %d", name, i);
    const int st = check_lora(&jobs[i].lora, n > 1 ? job : name);
    if (st) return st;
    if (jobs[i].lora.cols != jobs[0].lora.cols || jobs[i].lora.n_adapters != jobs[0].lora.n_adapters)
      return fail(Q4NX_E_SHAPE, "%s: job %d differs from job 0 in cols or n_adapters", name, i);
  }
  return Q4NX_OK;
}

int run_lora(const q4nx_lora_job* jobs, int n, const uint16_t* x, const int32_t* ids, int M, void* ws,
             size_t ws_bytes, void* stream, const char* name) {
  const int st = check_lora_jobs(jobs, n, M, name);
  if (st) return st;
  if (!x || !ids) return fail(Q4NX_E_ARG, "%s: null x or ids", name);
  if (!aligned(x, 16) || !aligned(ids, 4))
    return fail(Q4NX_E_ALIGN, "%s: x must be 16-byte, ids 4-byte aligned", name);
  const q4nx_lora* L[q4nx::kLoraMaxJobs];
  for (int i = 0; i < n; ++i) {
    const q4nx_lora_job& j = jobs[i];
    if (!j.base || !j.y) return fail(Q4NX_E_ARG, "%s: null base or y of job %d", name, i);
    if (!aligned(j.base, 4) || !aligned(j.y, 4))
      return fail(Q4NX_E_ALIGN, "%s: base and y of job %d must be 4-byte aligned", name, i);
    const uint64_t bytes = (uint64_t)M * j.lora.rows * 4;
    if (j.base != j.y && overlap(j.base, bytes, j.y, bytes))
      return fail(Q4NX_E_ARG, "%s: y of job %d overlaps its base without being it", name, i);
    for (int k = 0; k < n; ++k) {
      const uint64_t kb = (uint64_t)M * jobs[k].lora.rows * 4;
      if (k != i && (overlap(j.y, bytes, jobs[k].y, kb) || overlap(j.y, bytes, jobs[k].base, kb)))
        return fail(Q4NX_E_ARG, "%s: y of job %d overlaps y or base of job %d", name, i, k);
      if (overlaps_table(jobs[k].lora, j.y, bytes))
        return fail(Q4NX_E_ARG, "%s: y of job %d overlaps an arena, the scales or the ranks of job %d", name, i, k);
    }
    if (overlap(j.y, bytes, x, (uint64_t)M * j.lora.cols * 2) || overlap(j.y, bytes, ids, (uint64_t)M * 4))
      return fail(Q4NX_E_ARG, "%s: y of job %d overlaps x or ids", name, i);
    L[i] = &j.lora;
  }
  LoraShape sh;
  // pieces of one shape, equal but for a last one that is a few rows shorter (and
  // has more than kLoraWaveRows: a piece may have 512), so that a row's sums do not
  // depend on its place
  const int room = lora_rows(L, n, M), pieces = (M + room - 1) / room, per = (M + pieces - 1) / pieces;
  lora_shape(L, n, per, room, sh);
  if (!ws || ws_bytes < sh.total)
    return fail(Q4NX_E_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", name, ws_bytes, sh.total);
  if (!aligned(ws, 256)) return fail(Q4NX_E_ALIGN, "%s: workspace not 256-byte aligned", name);
  bool over = overlap(ws, sh.total, x, (uint64_t)M * L[0]->cols * 2) || overlap(ws, sh.total, ids, (uint64_t)M * 4);
  for (int i = 0; i < n; ++i) {
    const uint64_t bytes = (uint64_t)M * L[i]->rows * 4;
    over |= overlap(ws, sh.total, jobs[i].y, bytes) || overlap(ws, sh.total, jobs[i].base, bytes) ||
            overlaps_table(*L[i], ws, sh.total);
  }
  if (over) return fail(Q4NX_E_ARG, "%s: the workspace overlaps an input or output", name);
  uint8_t* w = static_cast<uint8_t*>(ws);
  for (int m0 = 0; m0 < M; m0 += per) {
    q4nx::LoraArgs& a = sh.a;
    a.M = std::min(per, M - m0);
    a.more = m0 > 0;
    a.x = x + (size_t)m0 * a.cols;
    a.ids = ids + m0;
    a.hdr = reinterpret_cast<uint32_t*>(w + sh.hdr);
    a.sorted = reinterpret_cast<int32_t*>(w + sh.sorted);
    a.tiles = reinterpret_cast<q4nx::LoraTile*>(w + sh.tiles);
    for (int i = 0; i < n; ++i) {
      q4nx::LoraJob& j = a.job[i];
      j.a = L[i]->a;
      j.b = L[i]->b;
      j.a_stride = L[i]->a_stride / 2;
      j.b_stride = L[i]->b_stride / 2;
      j.scale = L[i]->scale;
      j.ranks = L[i]->ranks;
      j.base = jobs[i].base + (size_t)m0 * L[i]->rows;
      j.y = jobs[i].y + (size_t)m0 * L[i]->rows;
      j.u = reinterpret_cast<float*>(w + sh.u[i]);
      j.rank = L[i]->rank;
      j.rows = L[i]->rows;
    }
    const hipError_t e = q4nx::launch_lora(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_status(e, name);
  }
  return ok();
}

}  // namespace

extern "C" {

size_t q4nx_lora_batched_ws(const q4nx_lora_job* jobs, int n_jobs, int M) {
  if (check_lora_jobs(jobs, n_jobs, M, "lora_batched_ws")) return 0;
  const q4nx_lora* L[q4nx::kLoraMaxJobs];
  for (int i = 0; i < n_jobs; ++i) L[i] = &jobs[i].lora;
  LoraShape sh;
  const int room = lora_rows(L, n_jobs, M);
  lora_shape(L, n_jobs, room, room, sh);
  return sh.total;
}

size_t q4nx_lora_ws(const q4nx_lora* L, int M) {
  if (!L) return 0;
  const q4nx_lora_job j{*L, nullptr, nullptr};
  return q4nx_lora_batched_ws(&j, 1, M);
}

int q4nx_lora_add_batched(const q4nx_lora_job* jobs, int n_jobs, const uint16_t* x, const int32_t* ids, int M,
                          void* ws, size_t ws_bytes, void* stream) {
  return run_lora(jobs, n_jobs, x, ids, M, ws, ws_bytes, stream, "lora_add_batched");
}

int q4nx_lora_add(const q4nx_lora* L, const uint16_t* x, const int32_t* ids, int M, const float* base, float* y,
                  void* ws, size_t ws_bytes, void* stream) {
  if (!L) return fail(Q4NX_E_ARG, "lora_add: null descriptor");
  const q4nx_lora_job j{*L, base, y};
  return run_lora(&j, 1, x, ids, M, ws, ws_bytes, stream, "lora_add");
}

// ---------------------------------------------------------------------------
// residual addition and RMS norm, log probabilities
// ---------------------------------------------------------------------------
int q4nx_add_rmsnorm(const float* y, const float* r, const uint16_t* w, int M, int D, float eps, float* r_out,
                     uint16_t* x, void* stream) {
  if (!r || !w || !x) return fail(Q4NX_E_ARG, "add_rmsnorm: null r, w or x");
  if (M < 1 || M > (1 << 20)) return fail(Q4NX_E_ARG, "add_rmsnorm: M = %d outside 1..1048576", M);
  if (D < 1 || D > q4nx::kNormMaxD)
    return fail(Q4NX_E_SHAPE, "add_rmsnorm: D = %d outside 1..%d", D, q4nx::kNormMaxD);
  if (!(eps >= 0.f) || eps > 3.4e38f) return fail(Q4NX_E_ARG, "add_rmsnorm: eps = %g is not a finite number >= 0", eps);
  if (!aligned(y, 4) || !aligned(r, 4) || !aligned(r_out, 4) || !aligned(w, 2) || !aligned(x, 2))
    return fail(Q4NX_E_ALIGN, "add_rmsnorm: y, r and r_out must be 4-byte, w and x 2-byte aligned");
  const uint64_t f = (uint64_t)M * D * 4, h = (uint64_t)M * D * 2, d = (uint64_t)D * 2;
  if (overlap(x, h, r, f) || (y && overlap(x, h, y, f)) || (r_out && overlap(x, h, r_out, f)) || overlap(x, h, w, d))
    return fail(Q4NX_E_ARG, "add_rmsnorm: x overlaps another array");
  if (r_out && ((r_out != r && overlap(r_out, f, r, f)) || (y && r_out != y && overlap(r_out, f, y, f)) ||
                overlap(r_out, f, w, d)))
    return fail(Q4NX_E_ARG, "add_rmsnorm: r_out overlaps an input without being r or y");
  return hip_status(q4nx::launch_add_rmsnorm(y, r, w, M, D, eps, r_out, x, static_cast<hipStream_t>(stream)),
                    "add_rmsnorm launch");
}

size_t q4nx_token_logprobs_ws(int n, int M, int k) {
  if (n < 1 || n > q4nx::kLogprobMaxN || M < 1 || M > 65535 || k < 0 || k > q4nx::kLogprobMaxK || k > n)
    return 0;
  return q4nx::logprob_ws_layout(n, M, k).total;
}

int q4nx_token_logprobs(const float* y, int n, int ldy, int M, const int32_t* tokens, int n_tok, float* logp,
                        float* entropy, int k, int32_t* top_ids, float* top_logp, void* ws, size_t ws_bytes,
                        void* stream) {
  if (!y) return fail(Q4NX_E_ARG, "token_logprobs: null y");
  if (n < 1 || n > q4nx::kLogprobMaxN || ldy < n || M < 1 || M > 65535)
    return fail(Q4NX_E_ARG, "token_logprobs: n = %d, ldy = %d, M = %d (need 1 <= n <= min(ldy, %d), 1 <= M <= 65535)",
                n, ldy, M, q4nx::kLogprobMaxN);
  if (n_tok < 0 || n_tok > q4nx::kLogprobMaxTok)
    return fail(Q4NX_E_ARG, "token_logprobs: n_tok = %d outside 0..%d", n_tok, q4nx::kLogprobMaxTok);
  if (k < 0 || k > q4nx::kLogprobMaxK || k > n)
    return fail(Q4NX_E_ARG, "token_logprobs: k = %d outside 0..min(%d, n)", k, q4nx::kLogprobMaxK);
  if (n_tok > 0 && (!tokens || !logp)) return fail(Q4NX_E_ARG, "token_logprobs: null tokens or logp");
  if (k > 0 && !top_ids) return fail(Q4NX_E_ARG, "token_logprobs: null top_ids");
  if (n_tok == 0 && k == 0 && !entropy) return fail(Q4NX_E_ARG, "token_logprobs: nothing is asked for");
  if (!aligned(y, 4) || !aligned(tokens, 4) || !aligned(logp, 4) || !aligned(entropy, 4) || !aligned(top_ids, 4) ||
      !aligned(top_logp, 4))
    return fail(Q4NX_E_ALIGN, "token_logprobs: every array must be 4-byte aligned");
  const struct { const void* p; uint64_t bytes; } part[] = {   // the outputs first
      {n_tok ? logp : nullptr, (uint64_t)M * n_tok * 4}, {entropy, (uint64_t)M * 4},
      {k ? top_ids : nullptr, (uint64_t)M * k * 4},      {k ? top_logp : nullptr, (uint64_t)M * k * 4},
      {y, ((uint64_t)(M - 1) * ldy + n) * 4},            {n_tok ? tokens : nullptr, (uint64_t)M * n_tok * 4}};
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 6; ++j)
      if (part[i].p && part[j].p && overlap(part[i].p, part[i].bytes, part[j].p, part[j].bytes))
        return fail(Q4NX_E_ARG, "token_logprobs: an output overlaps another array");
  const q4nx::LogprobWsLayout lay = q4nx::logprob_ws_layout(n, M, k);
  if (!ws || ws_bytes < lay.total)
    return fail(Q4NX_E_WORKSPACE, "token_logprobs: workspace of %zu bytes, %zu needed", ws_bytes, lay.total);
  if (!aligned(ws, 256)) return fail(Q4NX_E_ALIGN, "token_logprobs: workspace not 256-byte aligned");
  for (const auto& p : part)
    if (p.p && overlap(ws, lay.total, p.p, p.bytes))
      return fail(Q4NX_E_ARG, "token_logprobs: the workspace overlaps an input or output");
  q4nx::LogprobArgs a;
  memset(&a, 0, sizeof a);
  a.y = y;
  a.n = n;
  a.ldy = ldy;
  a.M = M;
  a.k = k;
  a.n_tok = n_tok;
  a.part_n = q4nx::logprob_part_n(n, M);
  a.parts = (n + a.part_n - 1) / a.part_n;
  a.tokens = tokens;
  a.logp = logp;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_logp = top_logp;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  a.stats = reinterpret_cast<q4nx::f32x4*>(wsb + lay.stats);
  a.keys = reinterpret_cast<uint64_t*>(wsb + lay.keys);
  return hip_status(q4nx::launch_token_logprobs(a, static_cast<hipStream_t>(stream)), "token_logprobs launch");
}

}  // extern "C"

// ---------------------------------------------------------------------------
// the cache, attention, linear attention
// ---------------------------------------------------------------------------
namespace {

int check_cache(const q4nx_kv_cache* c, const char* name, bool pointers) {
  if (!c) return fail(Q4NX_E_ARG, "%s: null cache", name);
  if (c->kv_heads < 1 || c->kv_heads > 256) return fail(Q4NX_E_ARG, "%s: kv_heads = %d outside 1..256", name, c->kv_heads);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(Q4NX_E_SHAPE, "%s: head_dim = %d is not 64, 128 or 256", name, c->head_dim);
  if (c->page_tokens < 16 || c->page_tokens > 1024 || (c->page_tokens & (c->page_tokens - 1)))
    return fail(Q4NX_E_SHAPE, "%s: page_tokens = %d is not a power of two in 16..1024", name, c->page_tokens);
  if (c->n_pages < 1 || (int64_t)c->n_pages * c->page_tokens > INT32_MAX)
    return fail(Q4NX_E_ARG, "%s: n_pages = %d (1 at least, 2^31 - 1 tokens at most)", name, c->n_pages);
  if (c->type != Q4NX_KV_BF16 && c->type != Q4NX_KV_INT8)
    return fail(Q4NX_E_ARG, "%s: cache type %d is not bf16 or int8", name, c->type);
  if (!pointers) return Q4NX_OK;
  const bool i8 = c->type == Q4NX_KV_INT8;
  if (!c->k || !c->v) return fail(Q4NX_E_ARG, "%s: null k or v pages", name);
  if (i8 != (c->k_scale != nullptr) || i8 != (c->v_scale != nullptr))
    return fail(Q4NX_E_ARG, "%s: an int8 cache has k_scale and v_scale, a bf16 cache neither", name);
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))
    return fail(Q4NX_E_ALIGN, "%s: pages and scales must be 16-byte aligned", name);
  const int64_t tokens = (int64_t)c->n_pages * c->page_tokens * c->kv_heads;
  const int64_t need = tokens * c->head_dim * (i8 ? 1 : 2);
  if (c->k_bytes < need || c->v_bytes < need)
    return fail(Q4NX_E_SHORT, "%s: pages of %lld and %lld bytes, %lld needed", name, (long long)c->k_bytes,
                (long long)c->v_bytes, (long long)need);
  if (i8 && (c->k_scale_bytes < tokens * 4 || c->v_scale_bytes < tokens * 4))
    return fail(Q4NX_E_SHORT, "%s: scales of %lld and %lld bytes, %lld needed", name, (long long)c->k_scale_bytes,
                (long long)c->v_scale_bytes, (long long)tokens * 4);
  return Q4NX_OK;
}

struct Span { const void* p; uint64_t bytes; };

bool overlap(const Span& x, const Span& y) { return x.p && y.p && x.bytes && y.bytes && overlap(x.p, x.bytes, y.p, y.bytes); }

// Whether two of the first `outs` of the spans, or one of them and another, share a byte.
template <size_t N>
bool outputs_overlap(const Span (&part)[N], size_t outs) {
  for (size_t i = 0; i < outs; ++i)
    for (size_t j = i + 1; j < N; ++j)
      if (overlap(part[i], part[j])) return true;
  return false;
}

// The four arrays of a checked cache.
void cache_spans(const q4nx_kv_cache* c, Span* s) {
  const uint64_t tokens = (uint64_t)c->n_pages * c->page_tokens * c->kv_heads;
  const uint64_t bytes = tokens * c->head_dim * (c->type == Q4NX_KV_INT8 ? 1 : 2);
  s[0] = {c->k, bytes};
  s[1] = {c->v, bytes};
  s[2] = {c->k_scale, tokens * 4};
  s[3] = {c->v_scale, tokens * 4};
}

q4nx::KvCache device_cache(const q4nx_kv_cache* c) {
  q4nx::KvCache d;
  d.k = c->k;
  d.v = c->v;
  d.ks = c->k_scale;
  d.vs = c->v_scale;
  d.heads = c->kv_heads;
  d.dim = c->head_dim;
  d.page_shift = __builtin_ctz((unsigned)c->page_tokens);
  d.n_pages = c->n_pages;
  return d;
}

int check_heads(const q4nx_heads* h, const char* name, int dim, int heads) {
  if (!h || !h->p) return fail(Q4NX_E_ARG, "kv_append: null %s", name);
  if (h->type != Q4NX_F32 && h->type != Q4NX_BF16) return fail(Q4NX_E_ARG, "kv_append: type %d of %s", h->type, name);
  if (heads && h->heads != heads) return fail(Q4NX_E_SHAPE, "kv_append: %s has %d heads, the cache %d", name, h->heads, heads);
  if (h->heads < 1 || (int64_t)h->heads * dim > 16384)
    return fail(Q4NX_E_SHAPE, "kv_append: %d heads of %s (1 at least, 16384 columns at most)", h->heads, name);
  if (h->ld < (int64_t)h->heads * dim || h->ld > (int64_t)1 << 40)
    return fail(Q4NX_E_SHAPE, "kv_append: ld %lld of %s below its %d columns, or too large", (long long)h->ld, name, h->heads * dim);
  if (!aligned(h->p, h->type == Q4NX_F32 ? 4 : 2)) return fail(Q4NX_E_ALIGN, "kv_append: %s is not aligned to its element", name);
  return Q4NX_OK;
}

Span heads_span(const q4nx_heads* h, int dim, int M) {
  if (!h) return {nullptr, 0};
  return {h->p, ((uint64_t)(M - 1) * h->ld + (uint64_t)h->heads * dim) * (h->type == Q4NX_F32 ? 4 : 2)};
}

q4nx::HeadRows device_heads(const q4nx_heads* h) {
  if (!h) return {nullptr, 0, 0, 0};
  return {h->p, h->ld, h->heads, h->type == Q4NX_BF16};
}

// How one q4nx_attention runs: the kernels of its sequences and, where several
// sequences share a prefix, of the prefix; and where their parts lie.
struct AttnShape {
  q4nx::AttnParts own, pre;   // pre.rows = 0: the prefix comes with each sequence's own keys
  int own_grid, pre_grid;
  size_t own_plan, own_o, own_ml, pre_plan, pre_o, pre_ml, total;
};

void attn_shape(const q4nx_kv_cache* c, const q4nx_attn_batch* b, int q_heads, int M, AttnShape& sh) {
  memset(&sh, 0, sizeof sh);
  const int KH = c->kv_heads, group = q_heads / KH;
  const int64_t rows = (int64_t)M * group;
  const bool apart = b->prefix_len > 0 && b->n_seq > 1 && (int64_t)b->max_q * group < 128;
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  size_t o = 0;
  auto place = [&](q4nx::AttnParts& p, int set, int tile, int slots, int& grid, size_t& plan, size_t& po, size_t& ml) {
    p.set = set;
    p.rows = tile;
    p.slots = slots;
    p.shares = tile == 128 ? slots : 1024;
    const int64_t parts = q4nx::attn_max_parts(p, b->n_seq, rows, KH);
    grid = (int)std::min<int64_t>(parts, tile == 128 ? 1 << 20 : 2048);
    plan = o;
    o = up(o + (2 + 2 * (size_t)q4nx::attn_entries(set, b->n_seq)) * 4);
    po = o;
    o = up(o + (size_t)parts * p.rows * c->head_dim * 4);
    ml = o;
    o = up(o + (size_t)parts * p.rows * 8);
  };
  const int64_t mine = (int64_t)b->max_q * group;
  const int tile = mine > 32 ? 128 : mine > 16 ? 32 : 16;
  const int slots = c->head_dim == 256 ? 256 : c->head_dim == 64 && tile == 128 ? 768 : 512;
  place(sh.own, apart ? q4nx::ATTN_OWN : q4nx::ATTN_ALL, tile, slots, sh.own_grid, sh.own_plan, sh.own_o, sh.own_ml);
  if (apart)
    place(sh.pre, q4nx::ATTN_PREFIX, rows > 32 ? 128 : tile, 256, sh.pre_grid, sh.pre_plan, sh.pre_o, sh.pre_ml);
  sh.total = o;
}

int check_linear(const q4nx_linear* L, int M) {
  if (!L) return fail(Q4NX_E_ARG, "linear_attn: null descriptor");
  if (L->n_seq < 1 || L->n_seq > Q4NX_ATTN_MAX_SEQ || L->max_q < 1 || L->max_q > Q4NX_ATTN_MAX_M || L->n_slots < 1 ||
      L->n_slots > (1 << 20))
    return fail(Q4NX_E_ARG, "linear_attn: n_seq = %d, max_q = %d, n_slots = %d (1..%d, 1..%d, 1..1048576)", L->n_seq, L->max_q,
                L->n_slots, (int)Q4NX_ATTN_MAX_SEQ, (int)Q4NX_ATTN_MAX_M);
  if (M < 1 || M > Q4NX_ATTN_MAX_M) return fail(Q4NX_E_ARG, "linear_attn: M = %d outside 1..%d", M, (int)Q4NX_ATTN_MAX_M);
  if (L->k_heads < 1 || L->k_heads > 256 || L->v_heads < 1 || L->v_heads > 1024 || L->v_heads % L->k_heads)
    return fail(Q4NX_E_SHAPE, "linear_attn: %d key and %d value heads (1..256, a multiple of them up to 1024)", L->k_heads,
                L->v_heads);
  if ((L->dk != 64 && L->dk != 128) || (L->dv != 64 && L->dv != 128))
    return fail(Q4NX_E_SHAPE, "linear_attn: dk = %d, dv = %d are not 64 or 128 each", L->dk, L->dv);
  return Q4NX_OK;
}

// How one q4nx_linear_attn runs.
struct LinearShape {
  bool chunks;
  int seg, items;      // rows of a segment; segments at most
  bool carried;        // a sequence may have several
  size_t plan, decay, state, total;
};

LinearShape linear_shape(const q4nx_linear* L, int M) {
  LinearShape sh;
  memset(&sh, 0, sizeof sh);
  sh.total = 256;
  // Rows one by one cost about 0.7 us each, a chunk 13 us with its launch (32 heads of 128 x 128: 16 rows 15.4 us, 17
  // in a chunk 13.0).
  sh.chunks = L->max_q > 12;
  if (!sh.chunks) return sh;
  // Sequences that fill the GPU by themselves, or have three chunks at most, run from end to end (8 of 512 rows, 32
  // heads: 70 us, 87 in segments; one of 128 rows 19).  Others are cut so that segments fill it, in single chunks
  // while there are few (one of 4096 rows: segments of 2, 4, 8 chunks 114, 92, 110 us; 3 of 333, 8 heads: segments of
  // 1, 2 chunks 21, 27 us).
  const int64_t chunks = ((int64_t)M + 63) / 64 * L->v_heads;
  sh.seg = 64 * (int)(chunks <= 384 ? 1 : std::max<int64_t>(2, (chunks + 511) / 512));
  const bool few = L->max_q > 192 && L->n_seq * (int64_t)L->v_heads < 256;
  sh.carried = few && L->max_q > sh.seg;
  if (!sh.carried) sh.seg = 1 << 30;
  sh.items = sh.carried ? M / sh.seg + L->n_seq : L->n_seq;
  if (!few) return sh;
  // Room for the most segments that M rows or fewer are cut into, so that a workspace for many rows holds fewer: whole
  // segments are M / 64 at most, and 512 / v_heads, as seg is 64 * chunks / 512 at least (or, of up to 384, one).
  const size_t items = std::min<int64_t>(M / 64, 512 / L->v_heads) + L->n_seq;
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  size_t o = up(((size_t)L->n_seq + 1) * 4);
  sh.decay = o;
  o = up(o + items * L->v_heads * 8);
  sh.state = o;
  sh.total = up(o + items * L->v_heads * L->dk * L->dv * 4);
  return sh;
}

int check_attn(const q4nx_kv_cache* c, const q4nx_attn_batch* b, int q_heads, int M, bool pointers) {
  const int st = check_cache(c, "attention", pointers);
  if (st) return st;
  if (!b) return fail(Q4NX_E_ARG, "attention: null batch");
  if (b->n_seq < 1 || b->n_seq > Q4NX_ATTN_MAX_SEQ)
    return fail(Q4NX_E_ARG, "attention: n_seq = %d outside 1..%d", b->n_seq, (int)Q4NX_ATTN_MAX_SEQ);
  if (M < 1 || M > Q4NX_ATTN_MAX_M) return fail(Q4NX_E_ARG, "attention: M = %d outside 1..%d", M, (int)Q4NX_ATTN_MAX_M);
  if (b->max_q < 1 || b->max_q > Q4NX_ATTN_MAX_M) return fail(Q4NX_E_ARG, "attention: max_q = %d", b->max_q);
  if (q_heads < 1 || q_heads % c->kv_heads || (int64_t)q_heads * c->head_dim > 16384)
    return fail(Q4NX_E_SHAPE, "attention: %d query heads over %d of %d columns (a multiple, 16384 columns at most)",
                q_heads, c->kv_heads, c->head_dim);
  if (b->pages_ld < 1) return fail(Q4NX_E_ARG, "attention: pages_ld = %d", b->pages_ld);
  if (b->prefix_len < 0 || (int64_t)b->prefix_len + (int64_t)b->pages_ld * c->page_tokens > INT32_MAX - 1024)
    return fail(Q4NX_E_ARG, "attention: a prefix of %d tokens before %d pages (2^31 - 1024 tokens at most)", b->prefix_len,
                b->pages_ld);
  return Q4NX_OK;
}

}  // namespace

extern "C" {

int q4nx_kv_append(const q4nx_kv_cache* cache, const q4nx_rope* rope, const q4nx_heads* q, uint16_t* q_out,
                   const q4nx_heads* k, const q4nx_heads* v, const int32_t* slots, int M, uint32_t* flags,
                   void* stream) {
  int st = check_cache(cache, "kv_append", true);
  if (st) return st;
  const int D = cache->head_dim;
  if (M < 1 || M > Q4NX_KV_MAX_M) return fail(Q4NX_E_ARG, "kv_append: M = %d outside 1..%d", M, (int)Q4NX_KV_MAX_M);
  if (q && !q->p) q = nullptr;
  if ((q != nullptr) != (q_out != nullptr)) return fail(Q4NX_E_ARG, "kv_append: q without q_out, or q_out without q");
  if (q && (st = check_heads(q, "q", D, 0))) return st;
  if ((st = check_heads(k, "k", D, cache->kv_heads)) || (st = check_heads(v, "v", D, cache->kv_heads))) return st;
  if (!slots) return fail(Q4NX_E_ARG, "kv_append: null slots");
  if (!aligned(slots, 4) || !aligned(flags, 4) || !aligned(q_out, 16))
    return fail(Q4NX_E_ALIGN, "kv_append: slots and flags must be 4-byte, q_out 16-byte aligned");
  if (rope) {
    if (!rope->inv_freq || !rope->pos) return fail(Q4NX_E_ARG, "kv_append: null inv_freq or pos");
    if (rope->dim < 16 || rope->dim % 16 || rope->dim > D)
      return fail(Q4NX_E_SHAPE, "kv_append: rope over %d dimensions is not a multiple of 16 in 16..%d", rope->dim, D);
    if (!aligned(rope->inv_freq, 4) || !aligned(rope->pos, 4))
      return fail(Q4NX_E_ALIGN, "kv_append: inv_freq and pos must be 4-byte aligned");
  }
  Span part[13] = {{q_out, q ? (uint64_t)M * q->heads * D * 2 : 0}};
  cache_spans(cache, part + 1);
  part[5] = {flags, 4};
  part[6] = heads_span(q, D, M);
  part[7] = heads_span(k, D, M);
  part[8] = heads_span(v, D, M);
  part[9] = {slots, (uint64_t)M * 4};
  if (rope) {
    part[10] = {rope->pos, (uint64_t)M * 4};
    part[11] = {rope->inv_freq, (uint64_t)rope->dim * 2};
  }
  if (outputs_overlap(part, 6)) return fail(Q4NX_E_ARG, "kv_append: q_out, the cache or flags overlap another array");
  q4nx::AppendArgs a;
  memset(&a, 0, sizeof a);
  a.c = device_cache(cache);
  a.q = device_heads(q);
  a.k = device_heads(k);
  a.v = device_heads(v);
  a.q_out = q_out;
  a.slots = slots;
  a.flags = flags;
  a.M = M;
  if (rope) {
    a.inv_freq = rope->inv_freq;
    a.pos = rope->pos;
    a.rot = rope->dim;
    a.interleaved = rope->interleaved != 0;
  }
  // One token a workgroup, its heads over several of them, until there are many; then eight, so that values can be
  // stored eight tokens at a time (32 + 8 heads of 128, fp32 in: 64 tokens 4.9 us, eight a workgroup 6.3; 256 tokens
  // 6.5 and 7.0; 512 tokens 9.2 and 7.6; 4096 tokens 48 and 30).  About 2048 workgroups (4001 tokens: 31 us, 36
  // with half of them, 35 with half as many more).
  a.tile = M >= 512 ? q4nx::kAppendTile : 1;
  const int tiles = q4nx::append_tiles(a), heads = a.q.heads + 2 * a.c.heads;
  const int head_parts = std::min((a.tile * heads * D / 16 + 255) / 256, std::max(1, 2048 / tiles));
  return hip_status(q4nx::launch_kv_append(a, head_parts, static_cast<hipStream_t>(stream)), "kv_append launch");
}

size_t q4nx_attention_ws(const q4nx_kv_cache* cache, const q4nx_attn_batch* batch, int q_heads, int M) {
  if (check_attn(cache, batch, q_heads, M, false)) return 0;
  AttnShape sh;
  attn_shape(cache, batch, q_heads, M, sh);
  return sh.total;
}

int q4nx_attention(const q4nx_kv_cache* cache, const q4nx_attn_batch* batch, const uint16_t* q, int q_heads, int M,
                   float scale, uint16_t* out, float* lse, void* ws, size_t ws_bytes, uint32_t* flags, void* stream) {
  const int st = check_attn(cache, batch, q_heads, M, true);
  if (st) return st;
  const q4nx_attn_batch& b = *batch;
  if (!q || !out) return fail(Q4NX_E_ARG, "attention: null q or out");
  if (!b.q_start || !b.kv_len || !b.pages || (b.prefix_len && !b.prefix_pages))
    return fail(Q4NX_E_ARG, "attention: null q_start, kv_len, pages or prefix_pages");
  if (!(scale >= -1e38f && scale <= 1e38f))   // times log2(e) it is still finite
    return fail(Q4NX_E_ARG, "attention: scale = %g is beyond 1e38 in size, or NaN", scale);
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(flags, 4) || !aligned(b.q_start, 4) ||
      !aligned(b.kv_len, 4) || !aligned(b.pages, 4) || !aligned(b.prefix_pages, 4))
    return fail(Q4NX_E_ALIGN, "attention: q and out must be 16-byte, every other array 4-byte aligned");
  const uint64_t bytes = (uint64_t)M * q_heads * cache->head_dim * 2;
  AttnShape sh;
  attn_shape(cache, batch, q_heads, M, sh);
  if (!ws || ws_bytes < sh.total)
    return fail(Q4NX_E_WORKSPACE, "attention: workspace of %zu bytes, %zu needed", ws_bytes, sh.total);
  if (!aligned(ws, 256)) return fail(Q4NX_E_ALIGN, "attention: workspace not 256-byte aligned");
  Span part[13] = {{out, bytes}, {lse, (uint64_t)M * q_heads * 4}, {ws, sh.total}, {flags, 4}, {q, bytes}};
  part[5] = {b.q_start, ((uint64_t)b.n_seq + 1) * 4};
  part[6] = {b.kv_len, (uint64_t)b.n_seq * 4};
  part[7] = {b.pages, (uint64_t)b.n_seq * b.pages_ld * 4};
  part[8] = {b.prefix_len ? b.prefix_pages : nullptr, ((uint64_t)b.prefix_len + cache->page_tokens - 1) / cache->page_tokens * 4};
  cache_spans(cache, part + 9);
  if (outputs_overlap(part, 4))
    return fail(Q4NX_E_ARG, "attention: out, lse, the workspace or flags overlap another array");
  q4nx::AttnArgs a;
  memset(&a, 0, sizeof a);
  a.c = device_cache(cache);
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.q_start = b.q_start;
  a.kv_len = b.kv_len;
  a.pages = b.pages;
  a.prefix_pages = b.prefix_pages;
  a.flags = flags;
  a.n_seq = b.n_seq;
  a.M = M;
  a.q_heads = q_heads;
  a.group = q_heads / cache->kv_heads;
  a.pages_ld = b.pages_ld;
  a.prefix_len = b.prefix_len;
  a.scale = scale * 1.4426950408889634f;
  uint8_t* w = static_cast<uint8_t*>(ws);
  auto at = [&](q4nx::AttnParts& p, size_t plan, size_t o, size_t ml) {
    p.plan = reinterpret_cast<int32_t*>(w + plan);
    p.o = reinterpret_cast<float*>(w + o);
    p.ml = reinterpret_cast<float*>(w + ml);
  };
  at(sh.own, sh.own_plan, sh.own_o, sh.own_ml);
  if (sh.pre.rows) at(sh.pre, sh.pre_plan, sh.pre_o, sh.pre_ml);
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = q4nx::launch_attn(a, sh.own, sh.own_grid, sh.pre, sh.pre_grid, s);
  if (e == hipSuccess) e = q4nx::launch_attn_join(a, sh.own, sh.pre, s);
  return hip_status(e, "attention launch");
}

size_t q4nx_linear_attn_ws(const q4nx_linear* L, int M) {
  if (check_linear(L, M)) return 0;
  return linear_shape(L, M).total;
}

int q4nx_linear_attn(const q4nx_linear* L, const uint16_t* q, int64_t q_ld, const uint16_t* k, int64_t k_ld,
                     const uint16_t* v, int64_t v_ld, const float* decay, int64_t decay_ld, int M, float scale,
                     const float* state, float* state_out, float* out, void* ws, size_t ws_bytes, uint32_t* flags,
                     void* stream) {
  const int st = check_linear(L, M);
  if (st) return st;
  if (!q || !k || !v || !decay || !state || !state_out || !out) return fail(Q4NX_E_ARG, "linear_attn: null array");
  if (!L->q_start || !L->slots) return fail(Q4NX_E_ARG, "linear_attn: null q_start or slots");
  const int64_t kc = (int64_t)L->k_heads * L->dk, vc = (int64_t)L->v_heads * L->dv, most = 1 << 24;
  if (q_ld < kc || k_ld < kc || v_ld < vc || q_ld > most || k_ld > most || v_ld > most)
    return fail(Q4NX_E_SHAPE, "linear_attn: row strides %lld, %lld, %lld below %lld, %lld, %lld columns, or too large",
                (long long)q_ld, (long long)k_ld, (long long)v_ld, (long long)kc, (long long)kc, (long long)vc);
  if (decay_ld != 0 && (decay_ld < L->v_heads || decay_ld > most))
    return fail(Q4NX_E_SHAPE, "linear_attn: decay_ld %lld is neither 0 nor at least %d", (long long)decay_ld, L->v_heads);
  if (!(scale >= -3.4e38f && scale <= 3.4e38f)) return fail(Q4NX_E_ARG, "linear_attn: scale = %g is not finite", scale);
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || q_ld % 8 || k_ld % 8 || v_ld % 8 || !aligned(state, 16) ||
      !aligned(state_out, 16) || !aligned(out, 16))
    return fail(Q4NX_E_ALIGN, "linear_attn: q, k, v, the states and out must be 16-byte aligned, strides multiples of 8");
  if (!aligned(decay, 4) || !aligned(L->q_start, 4) || !aligned(L->slots, 4) || !aligned(L->fresh, 4) || !aligned(flags, 4))
    return fail(Q4NX_E_ALIGN, "linear_attn: decay, q_start, slots, fresh and flags must be 4-byte aligned");
  const LinearShape sh = linear_shape(L, M);
  const size_t need = sh.total;
  if (!ws || ws_bytes < need) return fail(Q4NX_E_WORKSPACE, "linear_attn: workspace of %zu bytes, %zu needed", ws_bytes, need);
  if (!aligned(ws, 256)) return fail(Q4NX_E_ALIGN, "linear_attn: workspace not 256-byte aligned");
  const uint64_t sb = (uint64_t)L->n_slots * L->v_heads * L->dk * L->dv * 4, r = (uint64_t)M - 1;
  const Span part[] = {{out, (uint64_t)M * vc * 4}, {state_out, sb}, {ws, need}, {flags, 4},
                       {state_out == state ? nullptr : state, sb}, {q, (r * q_ld + kc) * 2}, {k, (r * k_ld + kc) * 2},
                       {v, (r * v_ld + vc) * 2}, {decay, (r * decay_ld + L->v_heads) * 4},
                       {L->q_start, ((uint64_t)L->n_seq + 1) * 4}, {L->slots, (uint64_t)L->n_seq * 4},
                       {L->fresh, (uint64_t)L->n_seq * 4}};
  if (outputs_overlap(part, 4))
    return fail(Q4NX_E_ARG, "linear_attn: out, state_out, the workspace or flags overlap another array");
  q4nx::LinearArgs a;
  memset(&a, 0, sizeof a);
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_ld = q_ld;
  a.k_ld = k_ld;
  a.v_ld = v_ld;
  a.decay = decay;
  a.decay_ld = decay_ld;
  a.state = state;
  a.state_out = state_out;
  a.out = out;
  a.q_start = L->q_start;
  a.slots = L->slots;
  a.fresh = L->fresh;
  a.flags = flags;
  a.k_heads = L->k_heads;
  a.v_heads = L->v_heads;
  a.dk = L->dk;
  a.dv = L->dv;
  a.n_seq = L->n_seq;
  a.n_slots = L->n_slots;
  a.M = M;
  a.scale = scale;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (!sh.chunks) return hip_status(q4nx::launch_linear_rows(a, s), "linear_attn launch");
  a.seg = sh.seg;
  if (sh.carried) {
    uint8_t* w = static_cast<uint8_t*>(ws);
    a.plan = reinterpret_cast<int32_t*>(w + sh.plan);
    a.seg_decay = reinterpret_cast<double*>(w + sh.decay);
    a.seg_state = reinterpret_cast<float*>(w + sh.state);
  }
  return hip_status(q4nx::launch_linear_chunks(a, sh.items, s), "linear_attn launch");
}

int q4nx_decode(const q4nx_weight* w, float* out, void* stream) {
  int st = check_weight(w, "decode");
  if (st) return st;
  if (!out) return fail(Q4NX_E_ARG, "decode: null output");
  if (!aligned(out, 4)) return fail(Q4NX_E_ALIGN, "decode: output not 4-byte aligned");
  const hipError_t e = q4nx::launch_decode(kind_of(w), static_cast<const uint8_t*>(w->chunks),
                                           w->rows / 32, w->cols / 256, out,
                                           static_cast<hipStream_t>(stream));
  return hip_status(e, "decode launch");
}

}  // extern "C"
