// Sampling a token per row of logits with temperature, top-k, top-p and min-p
// from a given random number.
//
// The tokens of a row are ordered by logit descending, equal logits by id
// ascending (the order of the top-K writer).  With e_j = exp((l_j - l_max) / T)
//   K = the first k tokens,
//   P = the shortest prefix whose mass reaches p mass(K),
//   M = the prefix with e_j >= min_p,
// and S the mass of the shortest of the three, the token is the first of the
// order whose cumulative mass exceeds u S, and logp = log(e_token / S).
//
// A token changes where its border moves, so masses and borders are held to
// about 1e-14 of the total: exponentials in fp64, sums in 64-bit integers (in
// any order the same) and fp64.
//
// One workgroup per row, bound by reading the row:
//  1. the largest logit of the row, with each thread's chunk maxima kept;
//  2a. 1 <= k <= 512: the k-th largest of the threads' maxima is a bound that
//     at least k tokens reach; only the chunks that reach it are read again,
//     the tokens found are sorted in LDS and everything else happens there;
//  2b. otherwise a histogram of the row's mass over 4096 bins, 1/64 octave of
//     e each (64 octaves: what lies below weighs less than 2^-64 a token).
//     Within a bin the masses e / (upper edge) lie in (2^-1/64, 1], so a short
//     polynomial gives them and 64-bit integers sum them with one relative
//     rounding.  Each border (k, then p, then u) falls into one bin, whose
//     tokens are collected and sorted in LDS; a bin with more tokens than fit
//     there is narrowed by 8 bits of the key at a time first, and where only
//     equal logits are left the border is a count, and the token is found by
//     its rank in id order.
#include <hip/hip_runtime.h>

#include "launch.hpp"

namespace ckl {

namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 4096;
constexpr int kPerThread = kBins / kThreads;
constexpr int kCap = 2048;      // tokens held in LDS
constexpr int kFastK = 512;     // largest k of the collected path
constexpr int kTopBits = 13;    // key bits of the histogram of the threads' maxima
constexpr int kSub = 256;       // digits of a narrowing pass
static_assert((1 << kTopBits) * 4 <= kBins * 8, "the maxima's histogram lives in the mass histogram");

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// Order-preserving unsigned key of a logit (-0 as +0); bf16 logits keep 16 bits.
template <typename T>
struct Key;
template <>
struct Key<__bf16> {
  static constexpr int kBits = 16;
  __device__ static inline uint32_t of(float v) {
    uint32_t b = __builtin_bit_cast(uint32_t, v) >> 16;
    if (b == 0x8000u) b = 0;
    return (b & 0x8000u) ? (~b & 0xFFFFu) : (b | 0x8000u);
  }
  __device__ static inline float value(uint32_t k) {
    const uint32_t b = (k & 0x8000u) ? (k & 0x7FFFu) : (~k & 0xFFFFu);
    return __builtin_bit_cast(float, b << 16);
  }
};
template <>
struct Key<float> {
  static constexpr int kBits = 32;
  __device__ static inline uint32_t of(float v) {
    uint32_t b = __builtin_bit_cast(uint32_t, v);
    if (b == 0x80000000u) b = 0;
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  }
  __device__ static inline float value(uint32_t k) {
    const uint32_t b = (k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k;
    return __builtin_bit_cast(float, b);
  }
};

// (key, id) packed so that a larger number comes earlier in the order.
__device__ inline uint64_t pack(uint32_t key, uint32_t id) { return ((uint64_t)key << 32) | (0xFFFFFFFFu - id); }
__device__ inline uint32_t unpack_id(uint64_t c) { return 0xFFFFFFFFu - (uint32_t)c; }

// A row as 16-byte chunks of its aligned memory: chunk c holds the elements
// c kN - off .. + kN - 1, off = the elements between the aligned address and
// the row's first one.  The first and the last chunk may reach outside the
// row and are put together from element loads, the others are one load.
template <typename T>
struct Row {
  static constexpr int kN = 16 / (int)sizeof(T);
  const T* x;
  const u32x4_t* base;
  int64_t V;
  int off;
  uint32_t chunks;
  __device__ inline Row(const T* row, int64_t v) : x(row), V(v) {
    off = (int)(((uintptr_t)row & 15) / sizeof(T));
    base = (const u32x4_t*)((uintptr_t)row & ~(uintptr_t)15);
    chunks = (uint32_t)((v + off + kN - 1) / kN);
  }
  __device__ inline bool edge(uint32_t c) const {
    return (c == 0 && off != 0) || (c == chunks - 1 && (V + off) % kN != 0);
  }
  // the chunk's values; outside the row -inf
  __device__ inline void load(uint32_t c, float* f) const {
    if (edge(c)) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int64_t e = (int64_t)c * kN + i - off;
        f[i] = (e >= 0 && e < V) ? (float)x[e] : -INFINITY;
      }
      return;
    }
    unpack(base[c], f);
  }
  __device__ static inline void unpack(const u32x4_t& v, float* f) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = v[i];
        f[2 * i] = __builtin_bit_cast(float, w << 16);
        f[2 * i + 1] = __builtin_bit_cast(float, w & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = v[i];
        f[i] = __builtin_bit_cast(float, w);
      }
    }
  }
  __device__ inline int64_t id(uint32_t c, int i) const { return (int64_t)c * kN + i - off; }
};

// Every value of the row as fn(value, id): the chunks of a thread in turn,
// four loads in flight.
template <typename T, typename F>
__device__ inline void for_each(const Row<T>& row, F&& fn) {
  constexpr int kN = Row<T>::kN;
  constexpr int U = 4;
  for (uint32_t c0 = threadIdx.x; c0 < row.chunks; c0 += U * kThreads) {
    u32x4_t v[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const uint32_t c = c0 + j * kThreads;
      if (c < row.chunks && !row.edge(c)) v[j] = row.base[c];
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const uint32_t c = c0 + j * kThreads;
      if (c >= row.chunks) break;
      float f[kN];
      if (row.edge(c))
        row.load(c, f);
      else
        Row<T>::unpack(v[j], f);
#pragma unroll
      for (int i = 0; i < kN; ++i) fn(f[i], row.id(c, i));
    }
  }
}

// The masses of one row.  y = -64 log2(e) of a logit; a bin is floor(y).
struct Scale {
  double mx, c, fix;  // c = 64 log2(e) / T; fix = 2^shift of the integer masses
  bool inf;           // the largest logit is +inf: equal ones weigh 1, all others nothing
  __device__ inline double y(float l) const {
    if (inf) return l == INFINITY ? 0.0 : (double)INFINITY;
    // -inf (and NaN, by the comparison below being false) weighs nothing
    return l > -INFINITY ? (mx - (double)l) * c : (double)INFINITY;
  }
};

// 2^(-f / 64) for f in [0, 1): the exponential series, off by at most
// (ln 2 / 64)^6 / 720 = 2.2e-15.
__device__ inline double pow_frac(double f) {
  const double t = f * -0.010830424696249145;  // -ln 2 / 64
  double r = 1.0 / 120.0;
  r = __builtin_fma(r, t, 1.0 / 24.0);
  r = __builtin_fma(r, t, 1.0 / 6.0);
  r = __builtin_fma(r, t, 0.5);
  r = __builtin_fma(r, t, 1.0);
  return __builtin_fma(r, t, 1.0);
}
__device__ inline double bin_top(int b) { return exp2(-(double)b / 64.0); }
// e of a logit whose y is below kBins, else 0
__device__ inline double mass_of(double y) {
  if (!(y < (double)kBins)) return 0.0;
  const double b = floor(y);
  return bin_top((int)b) * pow_frac(y - b);
}

struct Shared {
  uint64_t mass[kBins];       // integer masses relative to each bin's upper edge
  uint32_t count[kBins];      // tokens per bin (kept while k limits)
  uint64_t cand[kCap];        // collected (key, id)
  uint64_t sub_mass[kSub];    // a narrowing pass
  uint32_t sub_count[kSub];
  double red_d[kWaves];
  uint32_t red_u[kWaves];
  float red_f[kWaves];
  uint64_t edge_mass;         // mass of the tokens of min_p's bin that reach it
  uint32_t n_cand;
  uint32_t pick;
  double pick_mass;           // mass above the chosen bin or digit
  uint32_t pick_count;        // tokens above it
  double got_mass;
};

__device__ inline float block_max(float v, Shared& sh) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh.red_f[threadIdx.x >> 6] = v;
  __syncthreads();
  float m = sh.red_f[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) m = fmaxf(m, sh.red_f[i]);
  return m;
}

// Sum of v over the threads before this one, and over all of them: one fixed
// order, and a thread's sum plus its value is the next thread's sum exactly.
__device__ inline double block_prefix(double v, Shared& sh, double* before) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  double x = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const double y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 63) sh.red_d[w] = x;
  __syncthreads();
  double base = 0.0, all = 0.0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (i == w) base = all;
    all += sh.red_d[i];
  }
  const double prev = __shfl_up(x, 1);
  *before = lane == 0 ? base : base + prev;
  return all;
}
__device__ inline uint32_t block_prefix(uint32_t v, Shared& sh, uint32_t* before) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 63) sh.red_u[w] = x;
  __syncthreads();
  uint32_t base = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (i == w) base = all;
    all += sh.red_u[i];
  }
  *before = base + x - v;
  return all;
}

// Sort cand[0, n) descending.  The packed pairs are distinct, so up to one a
// thread its place is the number of larger ones; beyond that a bitonic sort.
__device__ inline void sort_cand(Shared& sh, int n) {
  uint64_t* a = sh.cand;
  if (n <= kThreads) {
    uint64_t c = 0;
    int place = 0;
    if ((int)threadIdx.x < n) {
      c = a[threadIdx.x];
      for (int i = 0; i < n; ++i) place += a[i] > c;
    }
    __syncthreads();
    if ((int)threadIdx.x < n) a[place] = c;
    __syncthreads();
    return;
  }
  int p2 = 1;
  while (p2 < n) p2 <<= 1;
  for (int i = n + threadIdx.x; i < p2; i += kThreads) a[i] = 0;  // below every real pair
  __syncthreads();
  for (int k = 2; k <= p2; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = threadIdx.x; i < p2; i += kThreads) {
        const int l = i ^ j;
        if (l > i) {
          const uint64_t x = a[i], y = a[l];
          if ((i & k) == 0 ? (x < y) : (x > y)) {
            a[i] = y;
            a[l] = x;
          }
        }
      }
      __syncthreads();
    }
  }
}

enum Border : int { BY_COUNT = 0, BY_MASS = 1, BY_MASS_OVER = 2 };  // the k-th token; mass >= target; mass > target

// Whether a prefix of `count` tokens and mass `mass` has reached the border.
__device__ inline bool reached(int kind, uint32_t count, double mass, uint32_t k, double target) {
  return kind == BY_COUNT ? count >= k : kind == BY_MASS ? mass >= target : mass > target;
}

// In the sorted cand[0, n): the first token at which the border is reached,
// `above` / `above_n` being what lies before the list; the last one if
// rounding leaves none.  Returns its place; *mass = the mass up to and with it.
template <typename T>
__device__ inline int pick_in_list(Shared& sh, int n, const Scale& sc, int kind, uint32_t k, double target,
                                   double above, uint32_t above_n, double* mass) {
  constexpr int kEach = kCap / kThreads;
  double e[kEach], mine = 0.0;
  const int b = threadIdx.x * kEach;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    e[i] = b + i < n ? mass_of(sc.y(Key<T>::value((uint32_t)(sh.cand[b + i] >> 32)))) : 0.0;
    mine += e[i];
  }
  double before = 0.0;
  block_prefix(mine, sh, &before);
  if (threadIdx.x == 0) sh.pick = 0xFFFFFFFFu;
  __syncthreads();
  double run = above + before;
  int at = -1;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    run += e[i];
    if (at < 0 && b + i < n && reached(kind, above_n + (uint32_t)(b + i + 1), run, k, target)) at = b + i;
  }
  if (at >= 0) atomicMin(&sh.pick, (uint32_t)at);
  __syncthreads();
  const int j = sh.pick < (uint32_t)n ? (int)sh.pick : n - 1;
  run = above + before;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    run += e[i];
    if (b + i == j) sh.got_mass = run;
  }
  __syncthreads();
  *mass = sh.got_mass;
  return j;
}

// Where a border lies: the mass of the prefix that ends there, and the last
// token of that prefix.
struct Found {
  double mass;
  float logit;
  int64_t id;
};

template <typename T>
__device__ Found find_border(const Row<T>& row, Shared& sh, const Scale& sc, int kind, uint32_t k, double target,
                             bool want_id) {
  const int tid = threadIdx.x;
  // 1. the bin: thread t holds the bins [kPerThread t, kPerThread (t + 1))
  double m[kPerThread], mine = 0.0, before = 0.0;
  uint32_t cmine = 0, cbefore = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * kPerThread + i;
    const uint64_t q = sh.mass[b];
    m[i] = q ? (double)q / sc.fix * bin_top(b) : 0.0;
    mine += m[i];
    cmine += sh.count[b];
  }
  block_prefix(mine, sh, &before);
  if (kind == BY_COUNT) block_prefix(cmine, sh, &cbefore);
  if (tid == 0) sh.pick = 0xFFFFFFFFu;
  __syncthreads();
  // the first bin at whose end the border is reached, else the last with mass
  int at = -1, last = -1;
  double run = before;
  uint32_t crun = cbefore;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * kPerThread + i;
    run += m[i];
    crun += kind == BY_COUNT ? sh.count[b] : 0;
    if (sh.mass[b] != 0) {
      last = b;
      if (at < 0 && reached(kind, crun, run, k, target)) at = b;
    }
  }
  if (at >= 0) atomicMin(&sh.pick, (uint32_t)at);
  __syncthreads();
  if (sh.pick == 0xFFFFFFFFu) {
    __syncthreads();
    if (tid == 0) sh.n_cand = 0;
    __syncthreads();
    if (last >= 0) atomicMax(&sh.n_cand, (uint32_t)last);
    __syncthreads();
    if (tid == 0) sh.pick = sh.n_cand;
    __syncthreads();
  }
  const int bin = (int)sh.pick;
  if (bin / kPerThread == tid) {
    double r = before;
    uint32_t c = cbefore;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      if (tid * kPerThread + i < bin) {
        r += m[i];
        c += kind == BY_COUNT ? sh.count[tid * kPerThread + i] : 0;
      }
    }
    sh.pick_mass = r;
    sh.pick_count = c;
  }
  __syncthreads();
  double above = sh.pick_mass;
  uint32_t above_n = sh.pick_count;
  const double top = bin_top(bin), y0 = (double)bin, y1 = (double)(bin + 1);
  // a float interval around the bin's logits: a cheap first test of each value
  // (c may be 0 or tiny: the interval is then the whole line)
  float lo = -INFINITY, hi = INFINITY;
  if (!sc.inf && sc.c > 0.0) {
    const double a = sc.mx - y1 / sc.c, b = sc.mx - y0 / sc.c;
    const double slack = 1e-9 * fabs(sc.mx) + 1e-30;  // far above the rounding of a, b and y
    lo = (float)(a - 1e-5 * fabs(a) - slack);
    hi = (float)(b + 1e-5 * fabs(b) + slack);
  }
  auto in_bin = [&](float l) {
    if (!(l >= lo && l <= hi)) return false;
    const double y = sc.y(l);
    return y >= y0 && y < y1;
  };

  // 2. the bin's tokens, narrowed by key digits until they fit
  uint32_t prefix = 0, prefix_mask = 0;
  int digits_left = Key<T>::kBits;
  for (;;) {
    __syncthreads();
    if (tid == 0) sh.n_cand = 0;
    __syncthreads();
    for_each(row, [&](float l, int64_t id) {
      if (in_bin(l)) {
        const uint32_t key = Key<T>::of(l);
        if ((key & prefix_mask) == prefix && id >= 0 && id < row.V) {
          const uint32_t slot = atomicAdd(&sh.n_cand, 1u);
          if (slot < (uint32_t)kCap) sh.cand[slot] = pack(key, (uint32_t)id);
        }
      }
    });
    __syncthreads();
    const uint32_t n = sh.n_cand;
    if (n <= (uint32_t)kCap) {
      sort_cand(sh, (int)n);
      double mass = 0.0;
      const int j = pick_in_list<T>(sh, (int)n, sc, kind, k, target, above, above_n, &mass);
      const uint64_t c = sh.cand[j];
      return Found{mass, Key<T>::value((uint32_t)(c >> 32)), (int64_t)unpack_id(c)};
    }
    if (digits_left == 0) break;
    // by the next 8 bits of the key, the largest digit first
    digits_left -= 8;
    __syncthreads();
    for (int i = tid; i < kSub; i += kThreads) {
      sh.sub_mass[i] = 0;
      sh.sub_count[i] = 0;
    }
    __syncthreads();
    for_each(row, [&](float l, int64_t id) {
      if (in_bin(l)) {
        const uint32_t key = Key<T>::of(l);
        if ((key & prefix_mask) == prefix && id >= 0 && id < row.V) {
          const double y = sc.y(l);
          const uint32_t dg = 255u - ((key >> digits_left) & 255u);
          atomicAdd((unsigned long long*)&sh.sub_mass[dg], (unsigned long long)(pow_frac(y - y0) * sc.fix + 0.5));
          atomicAdd(&sh.sub_count[dg], 1u);
        }
      }
    });
    __syncthreads();
    const double dm = tid < kSub && sh.sub_count[tid] ? (double)sh.sub_mass[tid] / sc.fix * top : 0.0;
    const uint32_t dc = tid < kSub ? sh.sub_count[tid] : 0;
    double db = 0.0;
    uint32_t cb = 0;
    block_prefix(dm, sh, &db);
    block_prefix(dc, sh, &cb);
    if (tid == 0) {
      sh.pick = 0xFFFFFFFFu;
      sh.n_cand = 0;
    }
    __syncthreads();
    if (dc && reached(kind, above_n + cb + dc, above + db + dm, k, target)) atomicMin(&sh.pick, (uint32_t)tid);
    if (dc) atomicMax(&sh.n_cand, (uint32_t)tid);
    __syncthreads();
    const uint32_t dg = sh.pick == 0xFFFFFFFFu ? sh.n_cand : sh.pick;
    if ((uint32_t)tid == dg) {
      sh.pick_mass = above + db;
      sh.pick_count = above_n + cb;
    }
    __syncthreads();
    above = sh.pick_mass;
    above_n = sh.pick_count;
    prefix |= (255u - dg) << digits_left;
    prefix_mask |= 255u << digits_left;
  }

  // 3. more equal logits than fit: each weighs e, and the border is a count of
  // them (at least 1, at most n)
  const uint32_t n = sh.n_cand;
  const float l = Key<T>::value(prefix);
  const double e = mass_of(sc.y(l));
  uint32_t r = 1;
  if (kind == BY_COUNT) {
    r = k > above_n ? k - above_n : 1;
  } else {
    // the smallest r in [1, n] with above + r e >= (or >) target, n if none
    uint32_t lo_r = 1, hi_r = n;
    while (lo_r < hi_r) {
      const uint32_t mid = lo_r + (hi_r - lo_r) / 2;
      if (reached(kind, 0, above + (double)mid * e, 0, target))
        hi_r = mid;
      else
        lo_r = mid + 1;
    }
    r = lo_r;
  }
  if (r > n) r = n;
  Found f{above + (double)r * e, l, -1};
  if (!want_id) return f;
  // the r-th of them in id order
  uint32_t seen = 0;
  for (int64_t base = 0; base < row.V; base += kThreads) {
    const int64_t id = base + tid;
    const bool eq = id < row.V && Key<T>::of((float)row.x[id]) == prefix;
    uint32_t rank = 0;
    const uint32_t total = block_prefix(eq ? 1u : 0u, sh, &rank);
    if (eq && seen + rank + 1 == r) sh.pick = (uint32_t)id;
    seen += total;
    if (seen >= r) break;  // uniform: every thread has the same total
  }
  __syncthreads();
  f.id = (int64_t)sh.pick;
  return f;
}

struct SampleArgs {
  const void* x;
  int64_t ld;
  int64_t V;
  const float* u;
  SampleParams p;
  int fix_bits;
  int32_t* ids;
  float* logp;
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) sample_kernel(SampleArgs a) {
  __shared__ Shared sh;
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x;
  const Row<T> row((const T*)a.x + r * a.ld, a.V);
  constexpr int kN = Row<T>::kN;

  // the row's settings; a temperature that is not above zero is greedy
  double T_ = a.p.temperatures ? (double)a.p.temperatures[r] : a.p.temperature;
  int64_t k64 = a.p.top_ks ? (int64_t)a.p.top_ks[r] : a.p.top_k;
  const double p = a.p.top_ps ? (double)a.p.top_ps[r] : a.p.top_p;
  double min_p = a.p.min_ps ? (double)a.p.min_ps[r] : a.p.min_p;
  if (!(T_ > 0.0)) {
    T_ = 1.0;
    k64 = 1;
  }
  T_ = fmax(T_, 1e-200);  // keeps 1 / T finite; only equal logits share the mass long before
  const bool limit = k64 > 0 && k64 < a.V;
  const uint32_t k = (uint32_t)(limit ? k64 : a.V);
  if (!(min_p > 0.0)) min_p = 0.0;
  if (min_p > 1.0) min_p = 1.0;
  double u = (double)a.u[r];
  if (!(u > 0.0)) u = 0.0;
  const double u_max = 1.0 - 0x1p-24;  // the largest fp32 below 1
  if (u > u_max) u = u_max;

  // 1. the largest logit; each thread's largest, and those of its chunks
  float mv = -INFINITY;
  for_each(row, [&](float l, int64_t) { mv = fmaxf(mv, l); });
  const float mx = block_max(mv, sh);
  if (mx == -INFINITY) {  // nothing to sample
    if (tid == 0) {
      a.ids[r] = -1;
      if (a.logp) a.logp[r] = -INFINITY;
    }
    return;
  }
  Scale sc;
  sc.inf = mx == INFINITY;
  sc.mx = (double)mx;
  sc.c = 92.332482616893656877 / T_;  // 64 log2(e)
  sc.fix = (double)(1ull << a.fix_bits);

  // 2a. few tokens: those that reach the k-th largest of the threads' maxima
  if (k <= (uint32_t)kFastK) {
    uint32_t* hist = (uint32_t*)sh.mass;
    constexpr int kHist = 1 << kTopBits, kShift = Key<T>::kBits - kTopBits, kPer = kHist / kThreads;
    for (int i = tid; i < kHist; i += kThreads) hist[i] = 0;
    if (tid == 0) {
      sh.n_cand = 0;
      sh.pick = 0;
    }
    __syncthreads();
    if (mv > -INFINITY) atomicAdd(&hist[Key<T>::of(mv) >> kShift], 1u);
    __syncthreads();
    // thread t holds the bins from the top: kHist - kPer (t + 1) ..
    uint32_t mine = 0, above = 0;
#pragma unroll
    for (int b = 0; b < kPer; ++b) mine += hist[kHist - 1 - (kPer * tid + b)];
    block_prefix(mine, sh, &above);
    if (above < k && above + mine >= k) {
      uint32_t c = above;
      for (int b = 0; b < kPer; ++b) {
        const int at = kHist - 1 - (kPer * tid + b);
        c += hist[at];
        if (c >= k) {
          sh.pick = (uint32_t)at << kShift;
          break;
        }
      }
    }
    __syncthreads();
    const uint32_t t0 = sh.pick;
    const float v0 = t0 <= Key<T>::of(-INFINITY) ? -INFINITY : Key<T>::value(t0);
    for_each(row, [&](float l, int64_t id) {
      if (l >= v0 && l > -INFINITY) {
        const uint32_t slot = atomicAdd(&sh.n_cand, 1u);
        if (slot < (uint32_t)kCap) sh.cand[slot] = pack(Key<T>::of(l), (uint32_t)id);
      }
    });
    __syncthreads();
    const uint32_t held = sh.n_cand;
    if (held <= (uint32_t)kCap) {
      sort_cand(sh, (int)held);
      const int n = (int)(held < k ? held : k);
      double S = 0.0, m = 0.0;
      // mass of the first n; then the p and min_p borders within them
      pick_in_list<T>(sh, n, sc, BY_COUNT, (uint32_t)n, 0.0, 0.0, 0, &S);
      const double Sk = S;
      if (p < 1.0) {
        pick_in_list<T>(sh, n, sc, BY_MASS, 0, p * Sk, 0.0, 0, &m);
        S = fmin(S, m);
      }
      if (min_p > 0.0) {
        // the prefix with e >= min_p: its length is a count of the list
        uint32_t c = 0, b = 0;
        for (int i = tid; i < n; i += kThreads)
          c += mass_of(sc.y(Key<T>::value((uint32_t)(sh.cand[i] >> 32)))) >= min_p;
        const uint32_t len = block_prefix(c, sh, &b);
        pick_in_list<T>(sh, n, sc, BY_COUNT, len > 0 ? len : 1, 0.0, 0.0, 0, &m);
        S = fmin(S, m);
      }
      const int j = pick_in_list<T>(sh, n, sc, BY_MASS_OVER, 0, u * S, 0.0, 0, &m);
      if (tid == 0) {
        const uint64_t c = sh.cand[j];
        a.ids[r] = (int32_t)unpack_id(c);
        if (a.logp) a.logp[r] = (float)log(mass_of(sc.y(Key<T>::value((uint32_t)(c >> 32)))) / S);
      }
      return;
    }
    __syncthreads();
  }

  // 2b. the row's mass over bins
  for (int i = tid; i < kBins; i += kThreads) {
    sh.mass[i] = 0;
    sh.count[i] = 0;
  }
  if (tid == 0) sh.edge_mass = 0;
  __syncthreads();
  // min_p's border: y <= y_min; its bin's share is summed on the side
  const double y_min = min_p > 0.0 ? -64.0 * log2(min_p) : (double)INFINITY;
  const int bin_min = y_min < (double)kBins ? (int)y_min : kBins;
  for_each(row, [&](float l, int64_t) {
    const double y = sc.y(l);
    if (y < (double)kBins) {
      const double b = floor(y);
      const int bin = (int)b;
      // round to an integer by adding 2^52: the low bits of the sum are it
      const double q = __builtin_fma(pow_frac(y - b), sc.fix, 0x1p52);
      const unsigned long long qi = (unsigned long long)__builtin_bit_cast(uint64_t, q) & 0xFFFFFFFFFFFFFull;
      atomicAdd((unsigned long long*)&sh.mass[bin], qi);
      if (limit) atomicAdd(&sh.count[bin], 1u);
      if (bin == bin_min && y <= y_min) atomicAdd((unsigned long long*)&sh.edge_mass, qi);
    }
  });
  __syncthreads();
  // masses of the whole row and of the tokens that reach min_p
  double S = 0.0, s_min = 0.0;
  {
    double all = 0.0, likely = 0.0, dummy;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int b = tid * kPerThread + i;
      const double m = sh.mass[b] ? (double)sh.mass[b] / sc.fix * bin_top(b) : 0.0;
      all += m;
      if (b < bin_min) likely += m;
      if (b == bin_min) likely += (double)sh.edge_mass / sc.fix * bin_top(b);
    }
    S = block_prefix(all, sh, &dummy);
    s_min = min_p > 0.0 ? block_prefix(likely, sh, &dummy) : S;
  }
  if (limit) S = find_border(row, sh, sc, BY_COUNT, k, 0.0, false).mass;
  if (p < 1.0) S = fmin(S, find_border(row, sh, sc, BY_MASS, 0, p * S, false).mass);
  S = fmin(S, s_min);
  const Found f = find_border(row, sh, sc, BY_MASS_OVER, 0, u * S, true);
  if (tid == 0) {
    a.ids[r] = (int32_t)f.id;
    if (a.logp) a.logp[r] = (float)log(mass_of(sc.y(f.logit)) / S);
  }
}

}  // namespace

hipError_t launch_sample(Dtype dt, const void* x, int64_t N, int64_t V, int64_t ld, const float* u,
                         const SampleParams& p, int32_t* ids, float* logp, hipStream_t s) {
  SampleArgs a{};
  a.x = x;
  a.ld = ld;
  a.V = V;
  a.u = u;
  a.p = p;
  int lg = 0;
  while (((int64_t)1 << lg) < V) ++lg;
  a.fix_bits = 62 - lg < 51 ? 62 - lg : 51;  // V masses of at most 2^fix_bits stay below 2^63
  a.ids = ids;
  a.logp = logp;
  if (dt == DT_BF16)
    hipLaunchKernelGGL(sample_kernel<__bf16>, dim3((unsigned)N), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL(sample_kernel<float>, dim3((unsigned)N), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace ckl
