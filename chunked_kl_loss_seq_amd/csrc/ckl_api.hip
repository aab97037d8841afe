// C ABI of the fused chunked KL loss: argument checks, chunk planner,
// workspace cache and the chunk loop that enqueues the kernels, for the fused
// call and for the forward / recomputing-backward pair.
#include <hip/hip_runtime.h>

#include <dlfcn.h>

#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <utility>
#include <vector>

#include "../../include/ckl.h"
#include "launch.hpp"

using namespace ckl;

// Workspace of ckl_fwd_bwd_noalloc, for callers that cannot allocate device
// memory.  Each GPU the library runs on holds its own copy of this array until
// the process ends.  In host code `scratch` names a host-side stand-in, not a
// device address: kernels get the address that hipGetSymbolAddress returns
// for the current device (scratch_ptr below).
static __device__ __align__(256) char scratch[CKL_NOALLOC_MAX_BYTES];

namespace {

constexpr uint64_t kScratchBytes = CKL_NOALLOC_MAX_BYTES;

constexpr uint64_t kDefaultBudget = 6ull << 30;
constexpr int64_t kRowStep = 256;
// Rows per chunk at most: keeps every grid dimension and tile count of a
// chunk's launches far inside 32 bits.
constexpr int64_t kMaxChunk = (int64_t)1 << 20;

inline uint64_t align256(uint64_t x) { return (x + 255) & ~uint64_t(255); }
inline int64_t roundup(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Which call a chunk loop serves: the fused forward + backward, the forward
// alone (loss and log-normalisers), or the backward that recomputes the logits.
enum Pass : int { PASS_FUSED = CKL_PASS_FUSED, PASS_FWD = CKL_PASS_FWD, PASS_BWD = CKL_PASS_BWD };

// Device workspace of one call with chunks of C rows.
struct Layout {
  int64_t C = 0;
  int64_t pblk = 0;     // elements between tile rows of the exp / gradient tiles
  int n_slices = 0;     // (max, sum exp) pairs per row
  int splits = 0;       // k-splits of the dH contraction
  int64_t cpad = 0;     // rows of the id tables (C rounded up to 256)
  uint64_t w_off = 0, p_off = 0, part_off = 0, scat_off = 0, slab_off = 0, kl_off = 0, lse_off = 0, scal_off = 0,
           hc_off = 0, idc_off = 0, tlc_off = 0, vidx_off = 0, pos_off = 0, bits_off = 0, pre_off = 0, rank_off = 0,
           zs_off = 0, total = 0;
};

Layout make_layout(Pass pass, int64_t N, int64_t d, int64_t V, int64_t K, int64_t C, size_t esz) {
  Layout L;
  L.C = C;
  L.pblk = tile_row_stride(V);
  L.n_slices = (int)((V + 127) / 128);
  L.splits = pass == PASS_FWD ? 0 : dh_splits(esz == 2 ? DT_BF16 : DT_F32, C, d, V);
  const int64_t tile_rows = (C + 63) / 64;
  uint64_t off = 0;
  L.w_off = off;  // tiled copy of W
  off += align256((uint64_t)((V + 63) / 64) * tile_row_stride(d) * esz);
  L.p_off = off;  // the forward alone keeps no exp values
  if (pass != PASS_FWD) off += align256((uint64_t)tile_rows * L.pblk * esz);
  L.part_off = off;
  off += align256((uint64_t)C * L.n_slices * 8);
  L.scat_off = off;
  off += align256((uint64_t)C * K * 4);
  L.slab_off = off;
  off += align256((uint64_t)L.splits * C * d * 4);
  L.kl_off = off;
  off += align256((uint64_t)N * 4);
  L.lse_off = off;
  off += align256((uint64_t)N * 4);
  L.scal_off = off;
  off += 256;
  // compacted chunk (calls with a mask): valid rows of H, ids and teacher
  // logits, and the index maps
  L.hc_off = off;
  off += align256((uint64_t)C * d * esz);
  L.idc_off = off;
  off += align256((uint64_t)C * K * 4);
  L.tlc_off = off;
  off += align256((uint64_t)C * K * 4);
  L.vidx_off = off;
  off += align256((uint64_t)C * 4);
  L.pos_off = off;
  off += align256((uint64_t)C * 4);
  // id tables of the chunk's cached ids: per (row, slice) a 128-bit mask and
  // a uint16 count, per cached id its rank, and the exact logits by rank
  L.cpad = roundup(C, 256);
  L.bits_off = off;
  off += align256((uint64_t)id_table_pairs(V) * L.cpad * 32);
  L.pre_off = off;
  off += align256((uint64_t)id_table_pairs(V) * L.cpad * 4);
  L.rank_off = off;
  off += align256((uint64_t)C * K * 4);
  L.zs_off = off;
  off += align256((uint64_t)C * K * 4);
  L.total = off;
  return L;
}

uint64_t budget_from_env(uint64_t b) {
  if (b) return b;
  const char* e = std::getenv("CKL_WORKSPACE_BYTES");
  if (e && *e) {
    char* end = nullptr;
    unsigned long long v = std::strtoull(e, &end, 10);
    if (end != e && v > 0) return (uint64_t)v;
  }
  return kDefaultBudget;
}

int plan_impl(Pass pass, int64_t N, int64_t d, int64_t V, int64_t K, int64_t chunk, uint64_t budget, size_t esz,
              Layout* out) {
  if (N < 0 || d <= 0 || V <= 0 || K <= 0 || chunk < 0) return CKL_EINVAL;
  if (K > V) return CKL_EINVAL;
  if (d % 8 != 0 || K > kMaxK) return CKL_EUNSUPPORTED;
  if (V > (int64_t)1 << 26 || N > (int64_t)1 << 31 || d > (int64_t)1 << 20) return CKL_EUNSUPPORTED;
  if (N == 0) {  // an empty batch: no chunk, no workspace
    *out = Layout{};
    return CKL_OK;
  }
  budget = budget_from_env(budget);
  if (chunk > 0) {
    const int64_t C = chunk < N ? chunk : N;
    if (C > kMaxChunk) return CKL_EUNSUPPORTED;
    Layout L = make_layout(pass, N, d, V, K, C, esz);
    if (L.total > budget) return CKL_EBUDGET;
    *out = L;
    return CKL_OK;
  }
  // largest fitting multiple of 256 rows (or N itself when smaller)
  int64_t cmax = 0;
  if (N <= kRowStep) {
    if (make_layout(pass, N, d, V, K, N, esz).total <= budget) cmax = N;
  } else {
    int64_t lo = 1, hi = roundup(N < kMaxChunk ? N : kMaxChunk, kRowStep) / kRowStep;  // in units of 256 rows
    if (make_layout(pass, N, d, V, K, kRowStep, esz).total > budget) return CKL_EBUDGET;
    while (lo < hi) {
      const int64_t mid = (lo + hi + 1) / 2;
      if (make_layout(pass, N, d, V, K, mid * kRowStep, esz).total <= budget)
        lo = mid;
      else
        hi = mid - 1;
    }
    cmax = lo * kRowStep;
    if (cmax > N) cmax = N;
  }
  if (cmax == 0) return CKL_EBUDGET;
  // even out: same number of chunks, the smallest 256-multiple that covers N
  const int64_t nch = (N + cmax - 1) / cmax;
  int64_t C = roundup((N + nch - 1) / nch, kRowStep);
  if (C > cmax) C = cmax;
  if (C > N) C = N;
  // The dH split count, and with it the slab bytes, depends on the chunk, so
  // the workspace is not monotonic in C: the search above only guarantees a
  // fitting multiple of 256 below the one it returns.  Step down until the
  // chunk really fits.
  for (int64_t c = C; c > 0; c = (c % kRowStep) ? c - c % kRowStep : c - kRowStep) {
    const Layout L = make_layout(pass, N, d, V, K, c, esz);
    if (L.total <= budget) {
      *out = L;
      return CKL_OK;
    }
  }
  return CKL_EBUDGET;
}

// ------------------------------------------------------------------ workspace cache
struct WsKey {
  int dev;
  hipStream_t stream;
  bool operator<(const WsKey& o) const { return dev != o.dev ? dev < o.dev : stream < o.stream; }
};
struct WsBuf {
  void* ptr = nullptr;
  uint64_t bytes = 0;
};
std::mutex g_ws_mu;
std::map<WsKey, WsBuf> g_ws;

int get_workspace(int dev, hipStream_t s, uint64_t bytes, void** ptr) {
  std::lock_guard<std::mutex> lk(g_ws_mu);
  WsBuf& b = g_ws[WsKey{dev, s}];
  if (b.bytes >= bytes) {
    *ptr = b.ptr;
    return CKL_OK;
  }
  if (b.ptr) {
    // the previous call on this stream may still be using the old buffer
    if (hipStreamSynchronize(s) != hipSuccess) return CKL_EHIP;
    if (hipFree(b.ptr) != hipSuccess) return CKL_EHIP;
    b.ptr = nullptr;
    b.bytes = 0;
  }
  const char* fail = std::getenv("CKL_TEST_FAIL_ALLOC");
  if (fail && fail[0] == '1') return CKL_ENOMEM;
  void* p = nullptr;
  hipError_t e = hipMalloc(&p, bytes);
  if (e != hipSuccess || !p) {
    (void)hipGetLastError();
    return CKL_ENOMEM;
  }
  b.ptr = p;
  b.bytes = bytes;
  *ptr = p;
  return CKL_OK;
}

// ------------------------------------------------------------------ fixed scratch
// Address of this device's copy of `scratch` (defined at file scope above),
// taken once per device with that device current.
constexpr int kMaxDevices = 64;
std::mutex g_scr_mu;
void* g_scratch[kMaxDevices] = {};

int scratch_ptr(int dev, void** out) {
  if (dev < 0 || dev >= kMaxDevices) return CKL_EUNSUPPORTED;
  std::lock_guard<std::mutex> lk(g_scr_mu);
  if (!g_scratch[dev]) {
    void* p = nullptr;
    const hipError_t e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess || !p) {
      (void)hipGetLastError();
      return CKL_EHIP;
    }
    g_scratch[dev] = p;
  }
  *out = g_scratch[dev];
  return CKL_OK;
}

// ------------------------------------------------------------------ tracing
// CKL_TRACE=1: roctx ranges around each loss call and around each chunk's
// launches (host enqueue time; `rocprofv3 --marker-trace` records them next to
// the kernels).  The roctx library is opened at run time, so the library has
// no link-time dependency on the profiler; without it the ranges are skipped.
struct Roctx {
  int (*push)(const char*) = nullptr;
  int (*pop)() = nullptr;
  bool tried = false;
};
Roctx g_roctx;
std::mutex g_roctx_mu;

bool trace_requested() {
  const char* e = std::getenv("CKL_TRACE");
  return e && e[0] == '1';
}

const Roctx* roctx_api() {
  std::lock_guard<std::mutex> lk(g_roctx_mu);
  if (!g_roctx.tried) {
    g_roctx.tried = true;
    void* h = dlopen("librocprofiler-sdk-roctx.so.1", RTLD_NOW | RTLD_LOCAL);
    if (!h) h = dlopen("libroctx64.so.4", RTLD_NOW | RTLD_LOCAL);
    if (h) {
      g_roctx.push = (int (*)(const char*))dlsym(h, "roctxRangePushA");
      g_roctx.pop = (int (*)())dlsym(h, "roctxRangePop");
      if (!g_roctx.push || !g_roctx.pop) g_roctx.push = nullptr;
    }
  }
  return g_roctx.push ? &g_roctx : nullptr;
}

struct TraceRange {
  const Roctx* api = nullptr;
  explicit TraceRange(const char* fmt, ...) __attribute__((format(printf, 2, 3))) {
    if (!trace_requested()) return;
    api = roctx_api();
    if (!api) return;
    char buf[192];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    api->push(buf);
  }
  ~TraceRange() {
    if (api) api->pop();
  }
  TraceRange(const TraceRange&) = delete;
  TraceRange& operator=(const TraceRange&) = delete;
};

// ------------------------------------------------------------------ timing
enum Kind { T_LOGITS = 0, T_ROWS, T_DH, T_DHRED, T_DW, T_OTHER, T_TOPK, T_EMBED, T_SAMPLE, T_FP8, T_KINDS };
struct TimingState {
  bool on = false;
  std::vector<std::pair<hipEvent_t, hipEvent_t>> pool;
  std::vector<std::pair<int, int>> recs;  // (kind, pool index)
};
TimingState g_tm;

struct Timed {
  int idx = -1;
  hipStream_t s;
  Timed(int kind, hipStream_t st, bool enabled = true) : s(st) {
    if (!g_tm.on || !enabled) return;
    const int i = (int)g_tm.recs.size();
    if (i >= (int)g_tm.pool.size()) {
      hipEvent_t a, b;
      if (hipEventCreate(&a) != hipSuccess) return;
      if (hipEventCreate(&b) != hipSuccess) return;
      g_tm.pool.push_back({a, b});
    }
    g_tm.recs.push_back({kind, i});
    idx = i;
    (void)hipEventRecord(g_tm.pool[i].first, s);
  }
  ~Timed() {
    if (idx >= 0) (void)hipEventRecord(g_tm.pool[idx].second, s);
  }
};

#define CKL_TRY(expr)                     \
  do {                                    \
    hipError_t e_ = (expr);               \
    if (e_ != hipSuccess) return CKL_EHIP; \
  } while (0)

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

bool debug_checks() {
  const char* e = std::getenv("CKL_DEBUG");
  return e && e[0] == '1';
}

// One call of any pass.  Inputs common to all: H, W, ids, tlogit, mask.
//   PASS_FUSED: out_loss, dH, dW (+ optional row_kl, row_lse)
//   PASS_FWD:   out_loss, row_lse (+ optional row_kl); no exp values are kept
//   PASS_BWD:   lse_in (the forward's row_lse), optional gscale; dH, dW; the
//               logits epilogue writes the gradient, so no dense pass runs
// With fixed_ws set, the call runs in the fixed scratch array of this device
// (budget kScratchBytes) and allocates nothing: no workspace cache, no timing
// events.
int run_impl(Pass pass, Dtype dt, const void* H, const void* W, const int32_t* ids, const float* tlogit,
             const uint8_t* mask, const float* lse_in, const float* gscale, int64_t N, int64_t d, int64_t V,
             int64_t K, int64_t chunk, float* out_loss, void* dH, float* dW, float* row_kl, float* row_lse,
             hipStream_t stream, bool fixed_ws = false) {
  const bool want_loss = pass != PASS_BWD, want_grad = pass != PASS_FWD;
  if (N == 0) {
    // An empty batch reads no row (its row arrays may be null) and has no
    // valid position: the loss is 0 and dW is 0.
    if (!W || (want_loss && !out_loss) || (want_grad && !dW)) return CKL_EINVAL;
    if (!aligned(W, 16) || !aligned(dW, 16) || !aligned(out_loss, 4)) return CKL_EINVAL;
    Layout L;
    const int st = plan_impl(pass, 0, d, V, K, chunk, 0, dt == DT_BF16 ? 2 : 4, &L);
    if (st != CKL_OK) return st;
    if (want_loss) CKL_TRY(launch_fill_f32(out_loss, 1, 0.f, stream));
    if (want_grad) CKL_TRY(launch_fill_f32(dW, V * d, 0.f, stream));
    return CKL_OK;
  }
  if (!H || !W || !ids || !tlogit) return CKL_EINVAL;
  if (want_loss && !out_loss) return CKL_EINVAL;
  if (want_grad && (!dH || !dW)) return CKL_EINVAL;
  if (pass == PASS_FWD && !row_lse) return CKL_EINVAL;
  if (pass == PASS_BWD && !lse_in) return CKL_EINVAL;
  if (!aligned(H, 16) || !aligned(W, 16) || !aligned(dH, 16) || !aligned(dW, 16)) return CKL_EINVAL;
  if (!aligned(ids, 4) || !aligned(tlogit, 4) || !aligned(out_loss, 4)) return CKL_EINVAL;
  if (!aligned(row_kl, 4) || !aligned(row_lse, 4) || !aligned(lse_in, 4) || !aligned(gscale, 4)) return CKL_EINVAL;
  const size_t esz = dt == DT_BF16 ? 2 : 4;
  Layout L;
  int st = plan_impl(pass, N, d, V, K, chunk, fixed_ws ? kScratchBytes : 0, esz, &L);
  if (st != CKL_OK) return st;
  if ((N + L.C - 1) / L.C > (int64_t)1 << 24) return CKL_EUNSUPPORTED;

  int dev = 0;
  CKL_TRY(hipGetDevice(&dev));
  void* ws = nullptr;
  st = fixed_ws ? scratch_ptr(dev, &ws) : get_workspace(dev, stream, L.total, &ws);
  if (st != CKL_OK) return st;
  const bool tm = !fixed_ws;
  static const char* const kPassName[] = {"ckl fused", "ckl forward", "ckl backward"};
  TraceRange call_range("%s N=%lld d=%lld V=%lld K=%lld chunk=%lld%s%s", kPassName[pass], (long long)N, (long long)d,
                        (long long)V, (long long)K, (long long)L.C, mask ? " masked" : "", fixed_ws ? " noalloc" : "");
  char* base = (char*)ws;
  void* Wt = base + L.w_off;
  void* P = pass == PASS_FWD ? nullptr : base + L.p_off;
  float2* part = (float2*)(base + L.part_off);
  float* scat = (float*)(base + L.scat_off);
  float* slab = (float*)(base + L.slab_off);
  float* kl = row_kl ? row_kl : (float*)(base + L.kl_off);
  float* lse = row_lse ? row_lse : (float*)(base + L.lse_off);
  void* scal = base + L.scal_off;
  // with a mask, every chunk is compacted to its valid rows; their count lives
  // in the scalar block, after the valid count and scale
  int* live = mask ? (int*)((char*)scal + 64) : nullptr;
  void* Hcc = base + L.hc_off;
  int32_t* idc = (int32_t*)(base + L.idc_off);
  float* tlc = (float*)(base + L.tlc_off);
  int* vidx = (int*)(base + L.vidx_off);
  int* pos = (int*)(base + L.pos_off);
  IdTables tab{};
  tab.bits = base + L.bits_off;
  tab.pre = base + L.pre_off;
  tab.cpad = L.cpad;
  tab.rank = (const int32_t*)(base + L.rank_off);
  tab.zs = (float*)(base + L.zs_off);
  tab.K = (int)K;
  unsigned* err = (unsigned*)((char*)scal + kErrOffset);

  {
    Timed t(T_OTHER, stream, tm);
    CKL_TRY(launch_mask_count(mask, N, scal, stream));
    CKL_TRY(launch_tile_copy(dt, W, V, d, Wt, stream));
  }
  for (int64_t r0 = 0; r0 < N; r0 += L.C) {
    const int64_t rows = (N - r0) < L.C ? (N - r0) : L.C;
    TraceRange chunk_range("chunk %lld: rows %lld-%lld", (long long)(r0 / L.C), (long long)r0,
                           (long long)(r0 + rows - 1));
    const void* Hc = (const char*)H + (size_t)r0 * d * esz;
    const int32_t* ids_c = ids + r0 * K;
    const float* tl_c = tlogit + r0 * K;
    float* lse_c = pass == PASS_BWD ? nullptr : lse + r0;
    if (live) {
      Timed t(T_OTHER, stream, tm);
      CKL_TRY(launch_compact(dt, mask + r0, rows, L.C, Hc, d, ids_c, tl_c, (int)K, vidx, pos, live, kl + r0, lse_c,
                             Hcc, idc, tlc, stream));
      Hc = Hcc;
      ids_c = idc;
      tl_c = tlc;
    }
    {
      Timed t(T_ROWS, stream, tm);
      CKL_TRY(launch_id_tables(ids_c, (int)K, rows, V, live, base + L.bits_off, base + L.pre_off, L.cpad,
                               (int32_t*)(base + L.rank_off), err, stream));
    }
    // The recomputing backward knows the log-normalisers before the logits:
    // their epilogue stores the gradient's dense part, and no dense pass runs.
    GradTerms gt{};
    if (pass == PASS_BWD) {
      gt.lse = lse_in + r0;
      gt.rowmap = live ? vidx : nullptr;
      gt.scale = (const float*)((const char*)scal + kScaleOffset);
      gt.gscale = gscale;
    }
    {
      Timed t(T_LOGITS, stream, tm);
      CKL_TRY(launch_logits(dt, Wt, Hc, V, d, rows, P, L.pblk, part, L.n_slices, &tab,
                            pass == PASS_BWD ? &gt : nullptr, live, stream));
    }
    {
      RowArgs a{};
      a.P = P;
      a.pblk = L.pblk;
      a.part = part;
      a.n_slices = L.n_slices;
      a.ids = ids_c;
      a.tlogit = tl_c;
      a.mask = nullptr;  // without a mask every row counts; with one, the compacted rows all do
      a.scal = scal;
      a.V = V;
      a.K = (int)K;
      a.rows = rows;
      a.scat = scat;
      a.kl_out = kl + r0;
      a.lse_out = lse_c;
      a.lse_in = pass == PASS_BWD ? lse_in + r0 : nullptr;
      a.gscale = pass == PASS_BWD ? gscale : nullptr;
      a.live = live;
      a.vidx = live ? vidx : nullptr;
      a.rank = tab.rank;
      a.zs = tab.zs;
      Timed t(T_ROWS, stream, tm);
      CKL_TRY(launch_row_stats(dt, a, stream));
      if (want_grad) {
        if (pass != PASS_BWD) CKL_TRY(launch_dense(dt, a, stream));
        CKL_TRY(launch_scatter(dt, a, stream));
      }
    }
    if (!want_grad) continue;
    int splits = dh_splits(dt, rows, d, V);
    const int64_t cap = (int64_t)L.splits * L.C / rows;  // slab capacity in splits of this chunk
    if (splits > cap) splits = dh_fit_splits(dt, V, (int)cap);
    {
      Timed t(T_DH, stream, tm);
      CKL_TRY(launch_dh(dt, P, L.pblk, Wt, V, d, rows, slab, splits, live, stream));
    }
    {
      Timed t(T_DHRED, stream, tm);
      CKL_TRY(launch_dh_reduce(dt, slab, splits, rows, d, live ? pos : nullptr, (char*)dH + (size_t)r0 * d * esz,
                               stream));
    }
    {
      Timed t(T_DW, stream, tm);
      CKL_TRY(launch_dw(dt, P, L.pblk, Hc, V, d, rows, dW, r0 > 0 ? 1 : 0, live, stream));
    }
  }
  if (want_loss) {
    Timed t(T_OTHER, stream, tm);
    CKL_TRY(launch_finalize(kl, N, scal, out_loss, stream));
  }
  // CKL_DEBUG=1: wait for the call and report cached ids outside [0, V) or
  // repeated within a row (the kernels leave them out, so nothing outside the
  // buffers was touched, but the results are not those of the definition)
  if (debug_checks()) {
    unsigned flags = 0;
    CKL_TRY(hipMemcpyAsync(&flags, err, sizeof(flags), hipMemcpyDeviceToHost, stream));
    CKL_TRY(hipStreamSynchronize(stream));
    if (flags != 0) return CKL_EINVAL;
  }
  return CKL_OK;
}

inline bool dtype_ok(int dtype) { return dtype == CKL_DTYPE_BF16 || dtype == CKL_DTYPE_F32; }
// Workgroups of 256 threads in one launch dimension, at most (exclusive).
constexpr int64_t kMaxBlocks256 = (int64_t)1 << 24;
// Rows of a sampling call, at most (exclusive): a workgroup of 1024 threads each.
constexpr int64_t kMaxSampleRows = (int64_t)1 << 22;

int embed_shape(int64_t N, int64_t d, int64_t V) {
  if (N < 0 || d <= 0 || V <= 0) return CKL_EINVAL;
  if (d % 8 != 0 || d > (int64_t)1 << 20 || V > (int64_t)1 << 26 || N >= (int64_t)1 << 26) return CKL_EUNSUPPORTED;
  return CKL_OK;
}

// ------------------------------------------------------------------ log-probabilities
// Arguments that the calls on logits share.
int logprob_shape(int dtype, const void* logits, int64_t N, int64_t V, int64_t ld, const int32_t* ids, int64_t T) {
  if (!dtype_ok(dtype) || N < 0 || V <= 0 || ld < 0 || T < 0) return CKL_EINVAL;
  if (V > (int64_t)1 << 26 || N >= kMaxSampleRows || T > kMaxK) return CKL_EUNSUPPORTED;
  if (!aligned(logits, dtype == CKL_DTYPE_BF16 ? 2 : 4) || !aligned(ids, 4)) return CKL_EINVAL;
  if (N > 0 && (!logits || (T > 0 && !ids))) return CKL_EINVAL;
  return CKL_OK;
}

// Device workspace of a call on hidden states with chunks of C rows.
struct HeadLayout {
  int64_t C = 0, pblk = 0;
  int n_slices = 0;
  HeadTiling tiling{TILE_256, TILE_256, 0};  // forward: the contraction's, and its slices of a row
  HeadSplit split{TILE_256, 0};              // backward: dH's
  uint64_t live_off = 0, hc_off = 0, vidx_off = 0, pos_off = 0, part_off = 0, parta_off = 0, g_off = 0, coef_off = 0, slab_off = 0, dw_off = 0, total = 0;
};

HeadLayout head_layout(bool backward, int64_t N, int64_t d, int64_t V, int64_t C, size_t esz, bool dw_sum) {
  HeadLayout L;
  L.C = C;
  L.pblk = tile_row_stride(V);
  uint64_t off = 0;
  const auto take = [&off](uint64_t bytes) {
    const uint64_t at = off;
    off += align256(bytes);
    return at;
  };
  L.live_off = take(4);
  L.hc_off = take((uint64_t)C * d * esz);
  L.vidx_off = take((uint64_t)C * 4);
  L.pos_off = take((uint64_t)C * 4);
  if (!backward) {
    L.tiling = head_logits_tiling(esz == 2 ? DT_BF16 : DT_F32, C, V, d);
    L.n_slices = head_slices(L.tiling, V);
    L.part_off = take((uint64_t)C * L.n_slices * 8);
    L.parta_off = take((uint64_t)C * L.n_slices * 4);
  } else {
    L.split = head_dh_split(esz == 2 ? DT_BF16 : DT_F32, C, d, V);
    L.g_off = take((uint64_t)((C + 63) / 64) * L.pblk * esz);
    L.coef_off = take((uint64_t)C * 16);
    L.slab_off = take((uint64_t)L.split.splits * C * d * 4);
    if (dw_sum && C < N) L.dw_off = take((uint64_t)V * d * 4);  // a bf16 dW's sums over chunks
  }
  L.total = off;
  return L;
}

int head_plan(bool backward, int dtype, int dw_dtype, int64_t N, int64_t d, int64_t V, int64_t chunk, uint64_t budget,
              HeadLayout* out) {
  if (!dtype_ok(dtype) || N < 0 || d <= 0 || V <= 0 || chunk < 0) return CKL_EINVAL;
  if (backward && (!dtype_ok(dw_dtype) || (dw_dtype == CKL_DTYPE_BF16 && dtype != CKL_DTYPE_BF16))) return CKL_EINVAL;
  if (d % 8 != 0 || V > (int64_t)1 << 26 || N > (int64_t)1 << 26 || d > (int64_t)1 << 20) return CKL_EUNSUPPORTED;
  *out = HeadLayout{};
  if (N == 0) return CKL_OK;
  budget = budget_from_env(budget);
  const size_t esz = dtype == CKL_DTYPE_BF16 ? 2 : 4;
  const bool sum = backward && dw_dtype == CKL_DTYPE_BF16;
  // rows per chunk at most: below 2^24 tiles of 64 x 64, the smallest, of 256 threads each
  const int64_t most_tiles = (((int64_t)1 << 24) - 1) / ((V + 63) / 64);
  const int64_t most = most_tiles >= kMaxChunk / 64 ? kMaxChunk : most_tiles / 4 * 256;
  if (chunk > 0) {
    const int64_t C = chunk < N ? chunk : N;
    if (C > most) return CKL_EUNSUPPORTED;
    const HeadLayout L = head_layout(backward, N, d, V, C, esz, sum);
    if (L.total > budget) return CKL_EBUDGET;
    *out = L;
    return CKL_OK;
  }
  // the fewest chunks of a multiple of 256 rows (or all rows) that fit
  int64_t C = N < most ? N : most;
  while (true) {
    const HeadLayout L = head_layout(backward, N, d, V, C, esz, sum);
    if (L.total <= budget) {
      *out = L;
      return CKL_OK;
    }
    if (C <= kRowStep) return CKL_EBUDGET;
    // even chunks, one more than now (N / 256 steps at most; far fewer, as C falls with 1 / chunks)
    const int64_t next = roundup((N + (N + C - 1) / C) / ((N + C - 1) / C + 1), kRowStep);
    C = next < C ? next : (C - 1) / kRowStep * kRowStep;
  }
}

// One call on hidden states: the shared chunk loop.  `grad` null: forward.
struct HeadCall {
  Dtype dt;
  size_t esz;
  const uint8_t* mask;
  char* ws;
};
struct Chunk {
  const void* Hc;
  const int *vidx, *pos, *live;
};
hipError_t head_chunk(const HeadCall& c, const HeadLayout& L, const void* H, int64_t d, int64_t r0, int64_t rows,
                      float* zero_out, Chunk* out, hipStream_t s) {
  *out = Chunk{(const char*)H + (size_t)r0 * d * c.esz, nullptr, nullptr, nullptr};
  if (!c.mask) return hipSuccess;
  int* live = (int*)(c.ws + L.live_off);
  int* vidx = (int*)(c.ws + L.vidx_off);
  int* pos = (int*)(c.ws + L.pos_off);
  const hipError_t e = launch_compact(c.dt, c.mask + r0, rows, L.C, out->Hc, d, nullptr, nullptr, 0, vidx, pos, live,
                                      zero_out, nullptr, c.ws + L.hc_off, nullptr, nullptr, s);
  *out = Chunk{c.ws + L.hc_off, vidx, pos, live};
  return e;
}

// A caller's dropout settings as the kernels take them; NULL drops nothing.
int drop_of(const ckl_drop* how, Drop* out) {
  *out = Drop{0, 0, nullptr, 0u, 1.f};
  if (!how) return CKL_OK;
  if (!(how->p >= 0.0 && how->p <= 1.0) || !aligned(how->offset_dev, 8)) return CKL_EINVAL;  // NaN fails too
  out->seed = how->seed;
  out->offset = how->offset;
  out->at = how->offset_dev;
  out->border = (uint32_t)(how->p * 65536.0 + 0.5);
  out->keep = out->border < 65536u ? (float)(65536.0 / (double)(65536u - out->border)) : 0.f;
  return CKL_OK;
}

int norm_shape(int64_t N, int64_t d) {
  if (N < 0 || d <= 0) return CKL_EINVAL;
  if (d % 8 != 0 || d > kMaxNormWidth || N > (int64_t)1 << 31) return CKL_EUNSUPPORTED;
  return CKL_OK;
}

// The part of the kernels' arguments that both directions share.
int norm_args(int dtype, const void* y, const void* r, const ckl_norm* how, int64_t N, int64_t d, NormArgs* p) {
  if (!how || !(how->eps >= 0.f) || (how->gate_rows != 0 && how->gate_rows != 1)) return CKL_EINVAL;
  const uintptr_t el = dtype == CKL_DTYPE_BF16 ? 2 : 4;
  if (!aligned(y, el) || !aligned(r, el) || !aligned(how->w_post, el) || !aligned(how->w_pre, el) ||
      !aligned(how->gate, el))
    return CKL_EINVAL;
  *p = NormArgs{};
  const int st = drop_of(how->drop, &p->drop);
  if (st != CKL_OK) return st;
  p->y = y;
  p->r = r;
  p->w_post = how->w_post;
  p->w_pre = how->w_pre;
  p->gate = how->gate;
  p->gate_rows = how->gate_rows != 0;
  p->scale = how->scale;
  p->eps = how->eps;
  p->N = N;
  p->d = d;
  return CKL_OK;
}

inline Dtype to_dt(int dtype) { return dtype == CKL_DTYPE_BF16 ? DT_BF16 : DT_F32; }

}  // namespace

extern "C" {

int ckl_fwd_bwd(const void* H, const void* W, const int32_t* topk_idx, const float* topk_logit,
                const uint8_t* mask, int64_t N, int64_t d, int64_t V, int64_t K, int64_t chunk, float* out_loss,
                void* dH, float* dW, hipStream_t stream) {
  try {
    return run_impl(PASS_FUSED, DT_BF16, H, W, topk_idx, topk_logit, mask, nullptr, nullptr, N, d, V, K, chunk,
                    out_loss, dH, dW, nullptr, nullptr, stream);
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_fwd_bwd_f32(const float* H, const float* W, const int32_t* topk_idx, const float* topk_logit,
                    const uint8_t* mask, int64_t N, int64_t d, int64_t V, int64_t K, int64_t chunk,
                    float* out_loss, float* dH, float* dW, hipStream_t stream) {
  try {
    return run_impl(PASS_FUSED, DT_F32, H, W, topk_idx, topk_logit, mask, nullptr, nullptr, N, d, V, K, chunk,
                    out_loss, dH, dW, nullptr, nullptr, stream);
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_fwd_bwd_ex(int dtype, const void* H, const void* W, const int32_t* topk_idx, const float* topk_logit,
                   const uint8_t* mask, int64_t N, int64_t d, int64_t V, int64_t K, int64_t chunk, float* out_loss,
                   void* dH, float* dW, float* row_kl, float* row_lse, hipStream_t stream) {
  if (!dtype_ok(dtype)) return CKL_EINVAL;
  try {
    return run_impl(PASS_FUSED, to_dt(dtype), H, W, topk_idx, topk_logit, mask, nullptr, nullptr, N, d, V, K, chunk,
                    out_loss, dH, dW, row_kl, row_lse, stream);
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_fwd_bwd_noalloc(int dtype, const void* H, const void* W, const int32_t* topk_idx,
                        const float* topk_logit, const uint8_t* mask, int64_t N, int64_t d, int64_t V, int64_t K,
                        int64_t chunk, float* out_loss, void* dH, float* dW, float* row_kl, float* row_lse,
                        hipStream_t stream) {
  if (!dtype_ok(dtype)) return CKL_EINVAL;
  try {
    return run_impl(PASS_FUSED, to_dt(dtype), H, W, topk_idx, topk_logit, mask, nullptr, nullptr, N, d, V, K, chunk,
                    out_loss, dH, dW, row_kl, row_lse, stream, true);
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_fwd(int dtype, const void* H, const void* W, const int32_t* topk_idx, const float* topk_logit,
            const uint8_t* mask, int64_t N, int64_t d, int64_t V, int64_t K, int64_t chunk, float* out_loss,
            float* row_lse, float* row_kl, hipStream_t stream) {
  if (!dtype_ok(dtype)) return CKL_EINVAL;
  try {
    return run_impl(PASS_FWD, to_dt(dtype), H, W, topk_idx, topk_logit, mask, nullptr, nullptr, N, d, V, K, chunk,
                    out_loss, nullptr, nullptr, row_kl, row_lse, stream);
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_bwd(int dtype, const void* H, const void* W, const int32_t* topk_idx, const float* topk_logit,
            const uint8_t* mask, const float* row_lse, const float* grad_loss, int64_t N, int64_t d, int64_t V,
            int64_t K, int64_t chunk, void* dH, float* dW, hipStream_t stream) {
  if (!dtype_ok(dtype)) return CKL_EINVAL;
  try {
    return run_impl(PASS_BWD, to_dt(dtype), H, W, topk_idx, topk_logit, mask, row_lse, grad_loss, N, d, V, K, chunk,
                    nullptr, dH, dW, nullptr, nullptr, stream);
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_topk(int dtype, const void* logits, int64_t N, int64_t V, int64_t K, int32_t* ids_out, float* vals_out,
             hipStream_t stream) {
  if (!dtype_ok(dtype)) return CKL_EINVAL;
  const size_t esz = dtype == CKL_DTYPE_BF16 ? 2 : 4;
  if (N < 0 || V <= 0 || K <= 0 || K > V) return CKL_EINVAL;
  if (N == 0) return K > kMaxK ? CKL_EUNSUPPORTED : CKL_OK;  // no rows: nothing to write
  if (!logits || !ids_out || !vals_out) return CKL_EINVAL;
  if (!aligned(logits, esz) || !aligned(ids_out, 4) || !aligned(vals_out, 4)) return CKL_EINVAL;
  if (K > kMaxK || V > 0x7FFFFFFFll || N > (int64_t)(0xFFFFFFFFull / 512)) return CKL_EUNSUPPORTED;
  try {
    Timed t(T_TOPK, stream);
    CKL_TRY(launch_topk(to_dt(dtype), logits, N, V, K, ids_out, vals_out, stream));
    return CKL_OK;
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_embed(int dtype, const int32_t* ids, const void* W, float scale, int64_t N, int64_t d, int64_t V, void* out,
              hipStream_t stream) {
  if (!dtype_ok(dtype)) return CKL_EINVAL;
  const int st = embed_shape(N, d, V);
  if (st != CKL_OK || N == 0) return st;
  if (!ids || !W || !out) return CKL_EINVAL;
  if (!aligned(ids, 4) || !aligned(W, 16) || !aligned(out, 16)) return CKL_EINVAL;
  if (embed_blocks(to_dt(dtype), N, d) >= kMaxBlocks256) return CKL_EUNSUPPORTED;
  try {
    Timed t(T_EMBED, stream);
    CKL_TRY(launch_embed(to_dt(dtype), ids, W, scale, N, d, V, out, stream));
    return CKL_OK;
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_embed_bwd_workspace(int64_t N, int64_t d, int64_t V, uint64_t* bytes_out) {
  if (!bytes_out) return CKL_EINVAL;
  const int st = embed_shape(N, d, V);
  if (st != CKL_OK) return st;
  *bytes_out = embed_bwd_workspace(N, d, V);
  return CKL_OK;
}

int ckl_embed_bwd(int dtype, const int32_t* ids, const void* dY, float scale, int64_t N, int64_t d, int64_t V,
                  int accumulate, float* dW, void* workspace, uint64_t workspace_bytes, hipStream_t stream) {
  if (!dtype_ok(dtype)) return CKL_EINVAL;
  const int st = embed_shape(N, d, V);
  if (st != CKL_OK) return st;
  if (!dW || !aligned(dW, 16)) return CKL_EINVAL;
  try {
    if (N == 0) {  // no positions: a zero gradient, or nothing to add
      if (!accumulate) CKL_TRY(launch_fill_f32(dW, V * d, 0.f, stream));
      return CKL_OK;
    }
    if (!ids || !dY || !workspace) return CKL_EINVAL;
    if (!aligned(ids, 4) || !aligned(dY, 16) || !aligned(workspace, 256)) return CKL_EINVAL;
    if (workspace_bytes < embed_bwd_workspace(N, d, V)) return CKL_EINVAL;
    if (embed_bwd_blocks(to_dt(dtype), N, d, V) >= kMaxBlocks256) return CKL_EUNSUPPORTED;
    Timed t(T_EMBED, stream);
    CKL_TRY(launch_embed_bwd(to_dt(dtype), ids, dY, scale, N, d, V, accumulate != 0, dW, workspace, stream));
    return CKL_OK;
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_sample_workspace(int dtype, int64_t N, int64_t V, uint64_t* bytes_out) {
  if (!dtype_ok(dtype) || !bytes_out || N < 0 || V <= 0) return CKL_EINVAL;
  if (V > (int64_t)1 << 26 || N >= kMaxSampleRows) return CKL_EUNSUPPORTED;
  *bytes_out = N > 0 ? sample_workspace(to_dt(dtype), N, V) : 0;
  return CKL_OK;
}

int ckl_sample(int dtype, const void* logits, int64_t N, int64_t V, int64_t row_stride, const float* u,
               const ckl_sampling* how, int32_t* ids_out, float* logp_out, void* workspace,
               uint64_t workspace_bytes, hipStream_t stream) {
  if (!dtype_ok(dtype)) return CKL_EINVAL;
  if (N < 0 || V <= 0 || row_stride < 0) return CKL_EINVAL;
  SampleParams p{1.0, 0, 1.0, 0.0, nullptr, nullptr, nullptr, nullptr};
  if (how) {
    p = SampleParams{how->temperature, how->top_k,  how->top_p, how->min_p,
                     how->temperatures, how->top_ks, how->top_ps, how->min_ps};
    // written so that NaN fails
    if (!p.temperatures && !(p.temperature >= 0.0)) return CKL_EINVAL;
    if (!p.top_ks && p.top_k < 0) return CKL_EINVAL;
    if (!p.top_ps && !(p.top_p >= 0.0 && p.top_p <= 1.0)) return CKL_EINVAL;
    if (!p.min_ps && !(p.min_p >= 0.0 && p.min_p <= 1.0)) return CKL_EINVAL;
    if (!aligned(p.temperatures, 4) || !aligned(p.top_ks, 4) || !aligned(p.top_ps, 4) || !aligned(p.min_ps, 4))
      return CKL_EINVAL;
  }
  if (V > (int64_t)1 << 26 || N >= kMaxSampleRows) return CKL_EUNSUPPORTED;
  if (N == 0) return CKL_OK;
  if (!logits || !u || !ids_out) return CKL_EINVAL;
  if (!aligned(logits, dtype == CKL_DTYPE_BF16 ? 2 : 4) || !aligned(u, 4) || !aligned(ids_out, 4) ||
      !aligned(logp_out, 4))
    return CKL_EINVAL;
  const uint64_t need = sample_workspace(to_dt(dtype), N, V);
  if (workspace && (!aligned(workspace, 256) || workspace_bytes < need)) return CKL_EINVAL;
  try {
    Timed t(T_SAMPLE, stream);
    CKL_TRY(launch_sample(to_dt(dtype), logits, N, V, row_stride, u, p, ids_out, logp_out, need ? workspace : nullptr,
                          stream));
    return CKL_OK;
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_quantize_fp8(int dtype, const void* x, int64_t R, int64_t C, int64_t block_rows, uint8_t* q_out,
                     float* scales_out, hipStream_t stream) {
  if (!dtype_ok(dtype)) return CKL_EINVAL;
  if (R < 0 || C <= 0 || (block_rows != 1 && block_rows != 128)) return CKL_EINVAL;
  if (C % 16 != 0 || C > (int64_t)1 << 20 || R > (int64_t)1 << 26) return CKL_EUNSUPPORTED;
  const int64_t blocks = (C + 127) / 128 * (block_rows == 1 ? (R + 15) / 16 : (R + 127) / 128);
  if (blocks >= kMaxBlocks256) return CKL_EUNSUPPORTED;
  if (R == 0) return CKL_OK;
  if (!x || !q_out || !scales_out) return CKL_EINVAL;
  if (!aligned(x, 16) || !aligned(q_out, 16) || !aligned(scales_out, 4)) return CKL_EINVAL;
  try {
    Timed t(T_FP8, stream);
    CKL_TRY(launch_quantize_fp8(to_dt(dtype), x, R, C, block_rows == 1, q_out, scales_out, stream));
    return CKL_OK;
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_matmul_fp8(int out_dtype, const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, int64_t M,
                   int64_t V, int64_t d, void* out, hipStream_t stream) {
  if (!dtype_ok(out_dtype)) return CKL_EINVAL;
  if (M < 0 || V <= 0 || d <= 0) return CKL_EINVAL;
  if (d % 16 != 0 || d > (int64_t)1 << 20 || V > (int64_t)1 << 26 || M > (int64_t)1 << 26) return CKL_EUNSUPPORTED;
  // tiles of any size the product takes, by the smallest
  if ((V + 63) / 64 * ((M + 63) / 64) >= (int64_t)1 << 26) return CKL_EUNSUPPORTED;
  if (M == 0) return CKL_OK;
  if (!xq || !xs || !wq || !ws || !out) return CKL_EINVAL;
  if (!aligned(xq, 16) || !aligned(wq, 16) || !aligned(xs, 4) || !aligned(ws, 4) ||
      !aligned(out, out_dtype == CKL_DTYPE_BF16 ? 2 : 4))
    return CKL_EINVAL;
  try {
    Timed t(T_FP8, stream);
    CKL_TRY(launch_matmul_fp8(to_dt(out_dtype), xq, xs, wq, ws, M, V, d, out, stream));
    return CKL_OK;
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_logprobs_workspace(int64_t N, int64_t V, int64_t top, uint64_t* bytes_out) {
  if (!bytes_out || N < 0 || V <= 0 || top < 0 || top > V) return CKL_EINVAL;
  if (V > (int64_t)1 << 26 || N >= kMaxSampleRows || top > kMaxTop) return CKL_EUNSUPPORTED;
  *bytes_out = align256(logprob_workspace(N, V, (int)top));
  return CKL_OK;
}

int ckl_logprobs(int dtype, const void* logits, int64_t N, int64_t V, int64_t row_stride, const int32_t* ids, int64_t T,
                 const uint8_t* mask, int64_t top, float* logp, float* entropy, float* stats, int32_t* top_ids,
                 float* top_logp, void* workspace, uint64_t workspace_bytes, hipStream_t stream) {
  const int st = logprob_shape(dtype, logits, N, V, row_stride, ids, T);
  if (st != CKL_OK) return st;
  if (top < 0 || top > V) return CKL_EINVAL;
  if (top > kMaxTop) return CKL_EUNSUPPORTED;
  if (!aligned(logp, 4) || !aligned(entropy, 4) || !aligned(stats, 4) || !aligned(top_ids, 4) || !aligned(top_logp, 4))
    return CKL_EINVAL;
  if (N == 0) return CKL_OK;
  if ((T > 0 && !logp) || !entropy || !stats || (top > 0 && (!top_ids || !top_logp))) return CKL_EINVAL;
  const uint64_t need = logprob_workspace(N, V, (int)top);
  if (workspace && (!aligned(workspace, 256) || workspace_bytes < need)) return CKL_EINVAL;
  LogprobArgs p{};
  p.x = logits;
  p.N = N;
  p.V = V;
  p.ld = row_stride;
  p.ids = ids;
  p.T = (int)T;
  p.top = (int)top;
  p.mask = mask;
  p.logp = logp;
  p.entropy = entropy;
  p.stats = stats;
  p.top_ids = top_ids;
  p.top_logp = top_logp;
  try {
    Timed t(T_OTHER, stream);
    CKL_TRY(launch_logprob(to_dt(dtype), p, need ? workspace : nullptr, stream));
    return CKL_OK;
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_logprobs_bwd(int dtype, const void* logits, int64_t N, int64_t V, int64_t row_stride, const int32_t* ids,
                     int64_t T, const uint8_t* mask, const float* stats, const float* entropy, const float* dlogp,
                     const float* dentropy, void* dlogits, int64_t out_stride, hipStream_t stream) {
  const int st = logprob_shape(dtype, logits, N, V, row_stride, ids, T);
  if (st != CKL_OK) return st;
  if (out_stride < V) return CKL_EINVAL;
  if (!aligned(stats, 4) || !aligned(entropy, 4) || !aligned(dlogp, 4) || !aligned(dentropy, 4) ||
      !aligned(dlogits, dtype == CKL_DTYPE_BF16 ? 2 : 4))
    return CKL_EINVAL;
  if (logprob_grad_blocks(N, V) >= kMaxBlocks256) return CKL_EUNSUPPORTED;
  if (N == 0) return CKL_OK;
  if (!stats || !dlogits || (T > 0 && !dlogp) || (dentropy && !entropy)) return CKL_EINVAL;
  if (dlogits == logits && N > 1 && out_stride != row_stride) return CKL_EINVAL;
  LogprobGradArgs p{};
  p.x = logits;
  p.N = N;
  p.V = V;
  p.ld = row_stride;
  p.ldo = out_stride;
  p.ids = ids;
  p.T = (int)T;
  p.mask = mask;
  p.stats = stats;
  p.entropy = entropy;
  p.dlogp = dlogp;
  p.dentropy = dentropy;
  p.out = dlogits;
  try {
    Timed t(T_OTHER, stream);
    CKL_TRY(launch_logprob_grad(to_dt(dtype), p, stream));
    return CKL_OK;
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_head_logprobs_plan(int backward, int dtype, int dw_dtype, int64_t N, int64_t d, int64_t V, int64_t chunk,
                           uint64_t budget_bytes, int64_t* chunk_out, uint64_t* workspace_bytes_out) {
  if (backward != 0 && backward != 1) return CKL_EINVAL;
  try {
    HeadLayout L;
    const int st = head_plan(backward != 0, dtype, dw_dtype, N, d, V, chunk, budget_bytes, &L);
    if (st != CKL_OK) return st;
    if (chunk_out) *chunk_out = L.C;
    if (workspace_bytes_out) *workspace_bytes_out = L.total;
    return CKL_OK;
  } catch (...) {
    return CKL_EINVAL;
  }
}

int ckl_head_logprobs(int dtype, const void* H, const void* W, const int32_t* ids, const uint8_t* mask, int64_t N,
                      int64_t d, int64_t V, int64_t T, int64_t chunk, float* logp, float* entropy, float* stats,
                      void* workspace, uint64_t workspace_bytes, hipStream_t stream) {
  try {
    HeadLayout L;
    const int st = head_plan(false, dtype, 0, N, d, V, chunk, 0, &L);
    if (st != CKL_OK) return st;
    if (T < 0) return CKL_EINVAL;
    if (T > kMaxK || N * T > (int64_t)1 << 26) return CKL_EUNSUPPORTED;
    if (!aligned(H, 16) || !aligned(W, 16) || !aligned(ids, 4) || !aligned(logp, 4) || !aligned(entropy, 4) ||
        !aligned(stats, 4) || !aligned(workspace, 256))
      return CKL_EINVAL;
    if (N == 0) return CKL_OK;
    if (!H || !W || (T > 0 && (!ids || !logp)) || !entropy || !stats || !workspace || workspace_bytes < L.total)
      return CKL_EINVAL;
    char* ws = (char*)workspace;
    const HeadCall c{to_dt(dtype), dtype == CKL_DTYPE_BF16 ? (size_t)2 : (size_t)4, mask, ws};
    const HeadArgs p{H, W, N, d, V, ids, (int)T, mask, logp, entropy, stats};
    float2* part = (float2*)(ws + L.part_off);
    float* part_a = (float*)(ws + L.parta_off);
    TraceRange range("ckl head logprobs N=%lld d=%lld V=%lld T=%lld chunk=%lld", (long long)N, (long long)d, (long long)V,
                     (long long)T, (long long)L.C);
    Timed t(T_OTHER, stream);
    for (int64_t r0 = 0; r0 < N; r0 += L.C) {
      const int64_t rows = N - r0 < L.C ? N - r0 : L.C;
      Chunk k;
      CKL_TRY(head_chunk(c, L, H, d, r0, rows, entropy + r0, &k, stream));
      CKL_TRY(launch_head_stats(c.dt, L.tiling, p, k.Hc, rows, part, part_a, L.n_slices, k.live, stream));
      CKL_TRY(launch_head_rows(c.dt, p, r0, rows, part, part_a, L.n_slices, k.pos, stream));
    }
    return CKL_OK;
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_head_logprobs_bwd(int dtype, const void* H, const void* W, const int32_t* ids, const uint8_t* mask, int64_t N,
                          int64_t d, int64_t V, int64_t T, int64_t chunk, const float* logp, const float* entropy,
                          const float* stats, const float* dlogp, const float* dentropy, void* dH, int dw_dtype,
                          int accumulate, void* dW, void* workspace, uint64_t workspace_bytes, hipStream_t stream) {
  try {
    HeadLayout L;
    const int st = head_plan(true, dtype, dw_dtype, N, d, V, chunk, 0, &L);
    if (st != CKL_OK) return st;
    if (T < 0 || (accumulate != 0 && accumulate != 1) || (accumulate && dw_dtype != CKL_DTYPE_F32)) return CKL_EINVAL;
    if (T > kMaxK || N * T > (int64_t)1 << 26) return CKL_EUNSUPPORTED;
    if (!aligned(H, 16) || !aligned(W, 16) || !aligned(ids, 4) || !aligned(logp, 4) || !aligned(entropy, 4) ||
        !aligned(stats, 4) || !aligned(dlogp, 4) || !aligned(dentropy, 4) || !aligned(dH, 16) || !aligned(dW, 16) ||
        !aligned(workspace, 256))
      return CKL_EINVAL;
    if (!dW) return CKL_EINVAL;
    const bool round = dw_dtype == CKL_DTYPE_BF16;
    if (N == 0) {  // V d is a multiple of 8: a bf16 dW is whole 32-bit words
      if (!accumulate) CKL_TRY(launch_fill_f32((float*)dW, round ? V * d / 2 : V * d, 0.f, stream));
      return CKL_OK;
    }
    if (!H || !W || !stats || !dH || (T > 0 && (!ids || !logp || !dlogp)) || (dentropy && !entropy) || !workspace ||
        workspace_bytes < L.total)
      return CKL_EINVAL;
    char* ws = (char*)workspace;
    const HeadCall c{to_dt(dtype), dtype == CKL_DTYPE_BF16 ? (size_t)2 : (size_t)4, mask, ws};
    const HeadGradArgs p{N, d, V, ids, (int)T, logp, stats, entropy, dlogp, dentropy};
    void* G = ws + L.g_off;
    float4* coef = (float4*)(ws + L.coef_off);
    float* slab = (float*)(ws + L.slab_off);
    float* sums = round ? (L.C < N ? (float*)(ws + L.dw_off) : nullptr) : (float*)dW;
    TraceRange range("ckl head logprobs backward N=%lld d=%lld V=%lld T=%lld chunk=%lld", (long long)N, (long long)d,
                     (long long)V, (long long)T, (long long)L.C);
    Timed t(T_OTHER, stream);
    for (int64_t r0 = 0; r0 < N; r0 += L.C) {
      const int64_t rows = N - r0 < L.C ? N - r0 : L.C;
      Chunk k;
      // the compaction writes a zero per masked row somewhere: the coefficients' place, which holds nothing yet
      CKL_TRY(head_chunk(c, L, H, d, r0, rows, (float*)coef, &k, stream));
      CKL_TRY(launch_head_grad(c.dt, p, W, k.Hc, r0, rows, k.vidx, k.live, coef, G, L.pblk, stream));
      HeadSplit h = head_dh_split(c.dt, rows, d, V);
      const int64_t cap = (int64_t)L.split.splits * L.C / rows;  // slab capacity in splits of this chunk
      if (h.splits > cap) h.splits = dh_fit_splits(c.dt, V, (int)cap);
      CKL_TRY(launch_head_dh(c.dt, h, G, L.pblk, W, V, d, rows, slab, k.live, stream));
      CKL_TRY(launch_dh_reduce(c.dt, slab, h.splits, rows, d, k.pos, (char*)dH + (size_t)r0 * d * c.esz, stream));
      const bool last = round && r0 + rows >= N;
      CKL_TRY(launch_head_dw(c.dt, G, L.pblk, k.Hc, V, d, rows, last && r0 > 0 ? sums : nullptr, sums,
                             r0 > 0 || accumulate ? 1 : 0, last ? dW : nullptr, k.live, stream));
    }
    return CKL_OK;
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_dropout(int dtype, const void* x, int64_t n, const ckl_drop* how, void* out, hipStream_t stream) {
  if (!dtype_ok(dtype) || n < 0 || !how) return CKL_EINVAL;
  Drop r;
  const int st = drop_of(how, &r);
  if (st != CKL_OK) return st;
  if (n >= (int64_t)1 << 37 || dropout_blocks(n) >= kMaxBlocks256) return CKL_EUNSUPPORTED;
  if (n == 0) return CKL_OK;
  const uintptr_t el = dtype == CKL_DTYPE_BF16 ? 2 : 4;
  if (!x || !out || !aligned(x, el) || !aligned(out, el)) return CKL_EINVAL;
  try {
    Timed t(T_OTHER, stream);
    CKL_TRY(launch_dropout(to_dt(dtype), x, n, r, out, stream));
    return CKL_OK;
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_add_norm(int dtype, const void* y, const void* r, const ckl_norm* how, int64_t N, int64_t d, void* r_out,
                 void* x, float* stats, hipStream_t stream) {
  if (!dtype_ok(dtype)) return CKL_EINVAL;
  int st = norm_shape(N, d);
  if (st != CKL_OK) return st;
  NormArgs p;
  st = norm_args(dtype, y, r, how, N, d, &p);
  if (st != CKL_OK) return st;
  const uintptr_t el = dtype == CKL_DTYPE_BF16 ? 2 : 4;
  if (!aligned(r_out, el) || !aligned(x, el) || !aligned(stats, 4)) return CKL_EINVAL;
  if (N == 0) return CKL_OK;
  if (!y || !r || !r_out || r_out == x || (p.w_pre != nullptr) != (x != nullptr)) return CKL_EINVAL;
  p.r_out = r_out;
  p.x = x;
  p.stats = stats;
  try {
    Timed t(T_OTHER, stream);
    CKL_TRY(launch_add_norm(to_dt(dtype), p, stream));
    return CKL_OK;
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_add_norm_bwd_workspace(int64_t N, int64_t d, int sums, uint64_t* bytes_out) {
  if (!bytes_out || sums < 0 || sums > 3) return CKL_EINVAL;
  const int st = norm_shape(N, d);
  if (st != CKL_OK) return st;
  *bytes_out = align256(add_norm_bwd_workspace(N, d, sums));
  return CKL_OK;
}

int ckl_add_norm_bwd(int dtype, const void* y, const void* r, const ckl_norm* how, int64_t N, int64_t d,
                     const float* stats, const void* dx, const void* dr_in, void* dy, void* dr, float* dw_post,
                     float* dw_pre, void* dgate, void* workspace, uint64_t workspace_bytes, hipStream_t stream) {
  if (!dtype_ok(dtype)) return CKL_EINVAL;
  int st = norm_shape(N, d);
  if (st != CKL_OK) return st;
  NormArgs p;
  st = norm_args(dtype, y, r, how, N, d, &p);
  if (st != CKL_OK) return st;
  const uintptr_t el = dtype == CKL_DTYPE_BF16 ? 2 : 4;
  const bool sums_gate = p.gate != nullptr && !p.gate_rows;
  if ((p.w_post != nullptr) != (dw_post != nullptr) || (p.w_pre != nullptr) != (dw_pre != nullptr)) return CKL_EINVAL;
  // without positions only the sums over them have something to hold
  if ((N > 0 || sums_gate) && (p.gate != nullptr) != (dgate != nullptr)) return CKL_EINVAL;
  if (!aligned(stats, 4) || !aligned(dx, el) || !aligned(dr_in, el) || !aligned(dy, el) || !aligned(dr, el) ||
      !aligned(dw_post, 4) || !aligned(dw_pre, 4) || !aligned(dgate, sums_gate ? 4 : el) || !aligned(workspace, 256))
    return CKL_EINVAL;
  NormGrads q{};
  const int n_sums = (dw_post != nullptr) + (dw_pre != nullptr) + (sums_gate ? 1 : 0);
  try {
    if (N == 0) {
      if (dw_post) CKL_TRY(launch_fill_f32(dw_post, d, 0.f, stream));
      if (dw_pre) CKL_TRY(launch_fill_f32(dw_pre, d, 0.f, stream));
      if (sums_gate) CKL_TRY(launch_fill_f32((float*)dgate, d, 0.f, stream));
      return CKL_OK;
    }
    if (!y || !r || !stats || !dy || !dr || (!dx && !dr_in) || (dx && !p.w_pre)) return CKL_EINVAL;
    if (dy == dr || dgate == dy || dgate == dr) return CKL_EINVAL;  // dgate may be null, these are not
    if (n_sums && (!workspace || workspace_bytes < add_norm_bwd_workspace(N, d, n_sums))) return CKL_EINVAL;
    p.stats_in = stats;
    q.dx = dx;
    q.dr_in = dr_in;
    q.dy = dy;
    q.dr = dr;
    q.dw_post = dw_post;
    q.dw_pre = dw_pre;
    q.dgate = dgate;
    q.part = (float*)workspace;
    Timed t(T_OTHER, stream);
    CKL_TRY(launch_add_norm_bwd(to_dt(dtype), p, q, stream));
    return CKL_OK;
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_plan_pass(int pass, int64_t N, int64_t d, int64_t V, int64_t K, int dtype, int64_t chunk,
                  uint64_t budget_bytes, int64_t* chunk_out, uint64_t* workspace_bytes_out) {
  if (!dtype_ok(dtype)) return CKL_EINVAL;
  if (pass != CKL_PASS_FUSED && pass != CKL_PASS_FWD && pass != CKL_PASS_BWD) return CKL_EINVAL;
  try {
    Layout L;
    const int st = plan_impl((Pass)pass, N, d, V, K, chunk, budget_bytes, dtype == CKL_DTYPE_BF16 ? 2 : 4, &L);
    if (st != CKL_OK) return st;
    if (chunk_out) *chunk_out = L.C;
    if (workspace_bytes_out) *workspace_bytes_out = L.total;
    return CKL_OK;
  } catch (...) {
    return CKL_EINVAL;
  }
}

int ckl_plan(int64_t N, int64_t d, int64_t V, int64_t K, int dtype, uint64_t budget_bytes, int64_t* chunk_out,
             uint64_t* workspace_bytes_out) {
  return ckl_plan_pass(CKL_PASS_FUSED, N, d, V, K, dtype, 0, budget_bytes, chunk_out, workspace_bytes_out);
}

void ckl_release_workspace(void) {
  std::lock_guard<std::mutex> lk(g_ws_mu);
  for (auto& kv : g_ws) {
    if (kv.second.ptr) {
      int cur = 0;
      (void)hipGetDevice(&cur);
      (void)hipSetDevice(kv.first.dev);
      (void)hipDeviceSynchronize();
      (void)hipFree(kv.second.ptr);
      (void)hipSetDevice(cur);
    }
  }
  g_ws.clear();
}

uint64_t ckl_workspace_bytes_held(void) {
  std::lock_guard<std::mutex> lk(g_ws_mu);
  uint64_t t = 0;
  for (auto& kv : g_ws) t += kv.second.bytes;
  return t;
}

const char* ckl_strerror(int status) {
  switch (status) {
    case CKL_OK: return "ok";
    case CKL_EINVAL: return "invalid argument";
    case CKL_ENOMEM: return "device workspace allocation failed";
    case CKL_EBUDGET: return "no chunk size fits the workspace budget";
    case CKL_EHIP: return "HIP runtime error";
    case CKL_EUNSUPPORTED: return "unsupported shape";
    default: return "unknown status";
  }
}

int ckl_debug_rows(const float* Z, const int32_t* idx, const float* tlogit, const uint8_t* mask, int64_t R,
                   int64_t V, int64_t K, float scale, int g_bf16, float* zg_out, int32_t* scatter_ids_out,
                   void* G_out, float* kl_out, float* lse_out, hipStream_t stream) {
  try {
    if (!Z || !idx || !tlogit || !zg_out || !scatter_ids_out || !G_out || !kl_out || !lse_out) return CKL_EINVAL;
    if (R <= 0 || V <= 0 || K <= 0 || K > V) return CKL_EINVAL;
    if (K > kMaxK) return CKL_EUNSUPPORTED;
    if (R > (int64_t)1 << 20 || V > (int64_t)1 << 26) return CKL_EUNSUPPORTED;
    const Dtype gdt = g_bf16 ? DT_BF16 : DT_F32;
    const size_t esz = g_bf16 ? 2 : 4;
    const int64_t pblk = tile_row_stride(V);
    const int n_slices = (int)((V + 127) / 128);
    const int64_t cpad = roundup(R, 256);
    const uint64_t pb = align256((uint64_t)((R + 63) / 64) * pblk * esz);
    const uint64_t qb = align256((uint64_t)R * n_slices * 8);
    const uint64_t sb = align256((uint64_t)R * K * 4);
    const uint64_t bb = align256((uint64_t)id_table_pairs(V) * cpad * 32);
    const uint64_t cb = align256((uint64_t)id_table_pairs(V) * cpad * 4);
    int dev = 0;
    CKL_TRY(hipGetDevice(&dev));
    void* ws = nullptr;
    int st = get_workspace(dev, stream, pb + qb + 3 * sb + bb + cb, &ws);
    if (st != CKL_OK) return st;
    char* wsb = (char*)ws;
    void* P = wsb;
    float2* part = (float2*)(wsb + pb);
    float* scat = (float*)(wsb + pb + qb);
    int32_t* rank = (int32_t*)(wsb + pb + qb + sb);
    float* zs = (float*)(wsb + pb + qb + 2 * sb);
    void* bits = wsb + pb + qb + 3 * sb;
    void* pre = wsb + pb + qb + 3 * sb + bb;
    // the id tables the chunk loop builds, and the logits at the cached ids
    // copied from Z as the logits contraction copies them from its accumulators
    CKL_TRY(launch_id_tables(idx, (int)K, R, V, nullptr, bits, pre, cpad, rank, nullptr, stream));
    CKL_TRY(launch_zs_from_z(Z, V, idx, rank, R, (int)K, zs, stream));
    CKL_TRY(launch_partials_from_z(gdt, Z, V, R, V, part, n_slices, P, pblk, stream));
    RowArgs a{};
    a.P = P;
    a.pblk = pblk;
    a.part = part;
    a.n_slices = n_slices;
    a.ids = idx;
    a.tlogit = tlogit;
    a.mask = mask;
    a.scal = nullptr;
    a.scale_value = scale;
    a.V = V;
    a.K = (int)K;
    a.rows = R;
    a.scat = scat;
    a.kl_out = kl_out;
    a.lse_out = lse_out;
    a.rank = rank;
    a.zs = zs;
    a.zg_dbg = zg_out;
    a.sid_dbg = scatter_ids_out;
    CKL_TRY(launch_row_stats(gdt, a, stream));
    CKL_TRY(launch_dense(gdt, a, stream));
    CKL_TRY(launch_scatter(gdt, a, stream));
    CKL_TRY(launch_untile(gdt, P, pblk, R, V, G_out, stream));
    CKL_TRY(hipStreamSynchronize(stream));
    return CKL_OK;
  } catch (...) {
    return CKL_EHIP;
  }
}

int ckl_timing_enable(int on) {
  g_tm.on = on != 0;
  g_tm.recs.clear();
  return CKL_OK;
}

int ckl_timing_query(int kind, double* total_ms, int64_t* launches) {
  if (kind < 0 || kind >= T_KINDS || !total_ms || !launches) return CKL_EINVAL;
  double t = 0.0;
  int64_t n = 0;
  for (auto& r : g_tm.recs) {
    if (r.first != kind) continue;
    auto& ev = g_tm.pool[r.second];
    if (hipEventSynchronize(ev.second) != hipSuccess) return CKL_EHIP;
    float ms = 0.f;
    if (hipEventElapsedTime(&ms, ev.first, ev.second) != hipSuccess) return CKL_EHIP;
    t += ms;
    ++n;
  }
  *total_ms = t;
  *launches = n;
  return CKL_OK;
}

}  // extern "C"
