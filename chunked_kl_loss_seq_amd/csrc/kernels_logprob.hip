// Log-probabilities of given tokens, entropy and the most likely alternatives of
// rows of logits, in one pass over a row, and their gradient.
//
// With M = max z, S = sum exp(z - M), A = sum exp(z - M) (z - M):
//   log p_j = (z_j - M) - log S       entropy = log S - A / S
// M and log S are kept apart ("stats"): their sum, the log-normaliser, loses the
// low bits of log S where |M| is large (a row masked with the type's lowest
// value).  The gradient of sum_t w_t log p_{id_t} + u entropy is
//   dz_j = sum_{t: id_t = j} w_t - p_j (sum_t w_t + u (log p_j + entropy)).
//
// A thread keeps its own reference m, at most 8 below its largest logit so far,
// its sums relative to m, and the largest logit: a new maximum costs a rescaling
// only when it is 8 above the reference.  -inf logits weigh nothing (z - m is
// held at -1000, whose exponential is 0, so that 0 x -inf never arises); NaN
// passes through to the row's results.
//
// Alternatives: a thread keeps the largest logit of each half of its share.  The
// K-th largest of those (or of the maxima of 64 groups of threads), cut to 16 bits,
// is a bound that at least K logits reach.  The halves whose maximum reaches it are
// read again, each by several lanes at once, and what reaches it is collected; up
// to 128 are placed by the number of larger (logit, lower id) pairs, more are
// sorted.  Where more than 1,024 reach the bound (equal logits, or fp32 ones under a
// common offset, whose keys differ in their lower 16 bits alone), a binary search over
// the pairs narrows it first, a pass over the row a step.  All of it is inlined: as
// calls, which the compiler made of what two kernels share, the registers saved around
// them cost 20 to 50 us of every case with alternatives below.
//
// Bound by reading the logits.  Measured (MI355X):
//  1,024 x 201,088 bf16: 72 us, 5.7 TB/s (with 100 given tokens a row 74); 20
//    alternatives 75 us, 128 110 us, 400 154 us.  fp32 140 us, with 20 148 us.
//  3,000 x 40,001 bf16, 20 alternatives: 51 us for 46 without.
//  The search: 1,024 x 201,088 fp32 normal logits about 300, top 1 / 20 / 128 / 400, 381 /
//    937 / 1,046 / 1,283 us (about 0: 144 / 148 / 193 / 266); about 5,000, 1,400 to 1,900;
//    bf16 about 300, where they take a dozen values, 130 / 132 / 137 / 7,800 us.
//  2,048 x 128,256 bf16 forward and gradient, a tenth of the rows masked: 284 us,
//    5.2 TB/s of 1.47 GB.
//  1 x 201,088 bf16, 20 alternatives: 7.7 us for the slices and 4.6 for joining them.
#include <hip/hip_runtime.h>
#include <math.h>

#include "row_io.hpp"

namespace ckl {

namespace {

typedef unsigned long long u64;

constexpr float kLog2 = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e38f;
constexpr float kFar = -1000.f;  // exp(kFar) is 0 in fp32
constexpr int kList = 1024;      // pairs held in LDS
constexpr int kGroups = 64;
// Up to this many alternatives the bound comes from the groups' maxima (2,048 x 128,256
// bf16, 20: 139 us and 140 with the threads' own; 48: 167 and 155, the coarser bound
// lets more through).
constexpr int kGroupTop = 24;
constexpr int kWideTop = 128;    // beyond, 256 threads' maxima are too few for a bound

__device__ inline float exp_fast(float t) { return __builtin_amdgcn_exp2f(t * kLog2); }
// the larger of t and kFar; NaN stays NaN
__device__ inline float not_far(float t) { return __builtin_elementwise_maximum(t, kFar); }

// Order-preserving key of a logit (-0 as +0); 0 for -inf and NaN, which are never alternatives.
__device__ inline uint32_t key_of(float z) {
  if (!(z > -INFINITY)) return 0u;
  const uint32_t u = __builtin_bit_cast(uint32_t, z + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ inline float key_value(uint32_t k) {
  return __builtin_bit_cast(float, (k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// (logit, lower id) pairs: larger comes first
__device__ inline u64 pair_of(uint32_t key, int64_t id) { return ((u64)key << 32) | (u64)(0xFFFFFFFFu - (uint32_t)id); }
__device__ inline int32_t pair_id(u64 p) { return (int32_t)(0xFFFFFFFFu - (uint32_t)p); }

// ------------------------------------------------------------------ sums of a run of logits
struct Sums {
  float m = kLowest;      // reference
  float mx = -INFINITY;   // largest logit (NaN left out)
  float s = 0.f, a = 0.f;
  __device__ inline void move(float to) {  // the reference becomes `to` >= m
    const float dm = fmaxf(m - to, kFar), k = exp_fast(dm);
    a = __builtin_fmaf(s, dm, a) * k;
    s *= k;
    m = to;
  }
  __device__ inline void add8(const float (&z)[8]) {
    const float c = fmaxf(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])), fmaxf(fmaxf(z[4], z[5]), fmaxf(z[6], z[7])));
    mx = fmaxf(mx, c);
    if (c > m + 8.f) move(c);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = not_far(z[e] - m), x = exp_fast(t);
      s += x;
      a = __builtin_fmaf(x, t, a);
    }
  }
};

// (M, S, A) of all threads of the workgroup, in every thread.
template <int NT>
__device__ inline void block_sums(Sums& v, float* red) {
  float M = wave_max(v.mx);
  const int w = threadIdx.x >> 6;
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) red[w] = M;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) M = fmaxf(M, red[i]);
  }
  v.mx = M;
  v.move(fmaxf(M, kLowest));
  v.s = lanes_sum(v.s, 64);
  v.a = lanes_sum(v.a, 64);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) {
      red[16 + w] = v.s;
      red[32 + w] = v.a;
    }
    __syncthreads();
    v.s = v.a = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) {
      v.s += red[16 + i];
      v.a += red[32 + i];
    }
  }
}

// What a row's sums give.  A row whose logits are all -inf has no distribution:
// entropy 0, log-probabilities -inf.
struct RowResult {
  float m, logs, entropy;
  bool none;
  __device__ inline RowResult(const Sums& v) {
    none = v.s == 0.f;
    m = none ? -INFINITY : fmaxf(v.mx, kLowest);
    logs = none ? 0.f : logf(v.s);
    const float h = logs - v.a / v.s;
    entropy = none || h < 0.f ? 0.f : h;
  }
  __device__ inline float logp(float z) const { return none ? -INFINITY : (z - m) - logs; }
};

// ------------------------------------------------------------------ alternatives
template <int NT>
struct TopLds {
  u64 list[kList], other[kList];
  uint32_t keys[2 * NT];
  int n, count[2];
  uint32_t bound;
};

// By one wave: the largest 16-bit prefix that at least K of n <= 1,024 keys reach, as
// a key (0 if fewer than K keys are above 0).
template <typename F>
__device__ __forceinline__ uint32_t prefix_bound(F key, int n, int K) {
  const int lane = threadIdx.x & 63;
  uint32_t v[kList / 64];
#pragma unroll
  for (int i = 0; i < kList / 64; ++i) v[i] = lane + 64 * i < n ? key(lane + 64 * i) >> 16 : 0u;
  uint32_t best = 0;
  for (int b = 15; b >= 0; --b) {
    const uint32_t next = best | (1u << b);
    int c = 0;
#pragma unroll
    for (int i = 0; i < kList / 64; ++i)
      if (64 * i < n) c += __builtin_popcountll(__ballot(v[i] >= next));
    if (c >= K) best = next;
  }
  return best << 16;
}

// The number of larger pairs in the list (kList long; entries past n may hold anything).
__device__ __forceinline__ int rank_in(const u64* list, int n, u64 pair) {
  int rank = 0;
  for (int j = 0; j < n; j += 8) {
    u64 o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = list[j + i];
#pragma unroll
    for (int i = 0; i < 8; ++i) rank += j + i < n && o[i] > pair;
  }
  return rank;
}

// The K largest of n <= kList pairs in `list` (all of them if there are fewer), in
// order; `other` is scratch.  Returns where they are.  The workgroup comes here
// together, and goes on with the result in sight of all.
template <int NT>
__device__ __forceinline__ const u64* order_top(u64* list, u64* other, int& n, int K, int* count, uint32_t* bound) {
  const int t = threadIdx.x;
  if (n > 128 && n > 2 * K) {  // fewer first: those that reach the K-th largest's prefix
    if (t < 64) {
      const uint32_t b = prefix_bound([&](int i) { return (uint32_t)(list[i] >> 32); }, n, K);
      if (t == 0) {
        *bound = b;
        *count = 0;
      }
    }
    __syncthreads();
    const uint32_t b = *bound;
    for (int i = t; i < n; i += NT) {
      const u64 pair = list[i];
      if ((uint32_t)(pair >> 32) >= b) other[atomicAdd(count, 1)] = pair;
    }
    __syncthreads();
    n = *count;
    u64* const swap = list;
    list = other;
    other = swap;
  }
  if (n <= 128) {  // each pair's place is the number of larger ones
    for (int i = t; i < n; i += NT) {
      const u64 pair = list[i];
      other[rank_in(list, n, pair)] = pair;
    }
    __syncthreads();
    return other;
  }
  int m = 256;
  while (m < n) m <<= 1;
  for (int i = n + t; i < m; i += NT) list[i] = 0;
  __syncthreads();
  for (int k = 2; k <= m; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int i = t; i < m / 2; i += NT) {
        const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
        const u64 x = list[lo], y = list[hi];
        if ((lo & k) == 0 ? x < y : x > y) {
          list[lo] = y;
          list[hi] = x;
        }
      }
      __syncthreads();
    }
  return list;
}

// Number of (key, id) pairs at or above `from` among the elements [lo, hi) of a row.
template <typename T, int NT>
__device__ __forceinline__ int count_from(const T* row, int64_t lo, int64_t hi, u64 from, TopLds<NT>& sh, int turn) {
  if (threadIdx.x == 0) sh.count[turn] = 0;
  __syncthreads();
  int c = 0;
  for (int64_t i = lo + threadIdx.x; i < hi; i += NT) {
    const uint32_t k = key_of((float)row[i]);
    c += k != 0u && pair_of(k, i) >= from;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) c += __shfl_xor(c, o);
  if ((threadIdx.x & 63) == 0) atomicAdd(&sh.count[turn], c);
  __syncthreads();
  return sh.count[turn];
}

// A thread takes the vectors t + k NT of a run of n8; k < first_half(n8) are its first half.
template <int NT>
__device__ inline int64_t first_half(int64_t n8) {
  const int64_t h = (n8 + NT - 1) / NT / 2;
  return h >= 8 ? h / 4 * 4 : h > 0 ? h : 1;  // whole turns of the scan
}

// Collects into sh.list at least the K largest pairs of the row's elements
// [lo, hi) (all of them if there are fewer), at most kList; mx0 and mx1 are the
// largest of the two halves of the elements that this thread took, M the row's.
template <typename T, int NT>
__device__ __forceinline__ int collect_top(const T* row, int64_t lo, int64_t hi, float mx0, float mx1, float M, int K,
                                  TopLds<NT>& sh) {
  const int t = threadIdx.x;
  const uint32_t key0 = key_of(mx0), key1 = key_of(mx1);
  if (t == 0) {
    sh.n = sh.count[0] = 0;
    sh.bound = 0u;
  }
  if (K <= kGroupTop && NT > 64) {
    uint32_t g = key0 > key1 ? key0 : key1;
#pragma unroll
    for (int o = 1; o < NT / kGroups; o <<= 1) {
      const uint32_t h = (uint32_t)__shfl_xor((int)g, o);
      g = g > h ? g : h;
    }
    if (t % (NT / kGroups) == 0) sh.keys[t / (NT / kGroups)] = g;
    __syncthreads();
    if (t < 64) {
      // the largest 16-bit prefix that K of the maxima reach (0 if there are fewer)
      const uint32_t v = sh.keys[t] >> 16;
      uint32_t best = 0;
#pragma unroll
      for (int b = 15; b >= 0; --b) {
        const uint32_t next = best | (1u << b);
        if (__builtin_popcountll(__ballot(v >= next)) >= K) best = next;
      }
      if (t == 0) sh.bound = best << 16;
    }
  } else if (K <= NT) {
    sh.keys[t] = key0;
    sh.keys[NT + t] = key1;
    __syncthreads();
    if (t < 64) {
      const uint32_t b = prefix_bound([&](int i) { return sh.keys[i]; }, 2 * NT, K);
      if (t == 0) sh.bound = b;
    }
  }
  __syncthreads();
  const uint32_t bound = sh.bound > 1u ? sh.bound : 1u;
  // The halves that hold such a maximum; g lanes (a power of two) read each one's logits again.
  if (key0 >= bound) sh.keys[atomicAdd(&sh.count[0], 1)] = (uint32_t)t;
  if (key1 >= bound) sh.keys[atomicAdd(&sh.count[0], 1)] = (uint32_t)(NT + t);
  __syncthreads();
  const int owners = sh.count[0];
  const float least = bound > 1u ? key_value(bound) : kLowest;  // NaN and -inf do not reach it
  const auto take = [&](float z, int64_t id) {
    if (z >= least) {
      const int i = atomicAdd(&sh.n, 1);
      if (i < kList) sh.list[i] = pair_of(key_of(z), id);
    }
  };
  const int64_t n8 = (hi - lo) / 8, half = first_half<NT>(n8), rest = (n8 + NT - 1) / NT - half;
  const int64_t most = rest > half ? rest : half;
  int g = 1;
  while (g < 64 && g < most) g <<= 1;
  const int teams = NT / g;
  constexpr int U = sizeof(T) == 2 ? 4 : 2;  // vectors under way
  for (int o = t / g; o < owners && n8 > 0; o += U * teams)
    for (int64_t j = t & (g - 1); j < most; j += g) {
      Eight<T> v[U];
      int64_t at[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t q = o + u * teams < owners ? sh.keys[o + u * teams] : 2 * NT;
        at[u] = q < NT && j < half ? q + j * NT : q >= NT && q < 2 * NT ? q - NT + (half + j) * NT : n8;
        v[u].load(row + lo + 8 * (at[u] < n8 ? at[u] : 0));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (at[u] >= n8) continue;
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = v[u].get(e);
        if (fmaxf(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])), fmaxf(fmaxf(z[4], z[5]), fmaxf(z[6], z[7]))) >= least) {
#pragma unroll
          for (int e = 0; e < 8; ++e) take(z[e], lo + 8 * at[u] + e);
        }
      }
    }
  if (lo + 8 * n8 + t < hi) take((float)row[lo + 8 * n8 + t], lo + 8 * n8 + t);
  __syncthreads();
  int n = sh.n;
  if (n <= kList) return n;
  // At least K pairs lie at or above `from`, fewer than K above `top`.
  u64 from = pair_of(bound, hi - 1), top = pair_of(key_of(M), lo);
  int turn = 0;
  while (n > kList) {
    const u64 mid = from + (top - from + 1) / 2;
    const int c = count_from<T, NT>(row, lo, hi, mid, sh, turn);
    turn ^= 1;
    if (c >= K) {
      from = mid;
      n = c;
    } else {
      top = mid - 1;
    }
  }
  __syncthreads();
  if (t == 0) sh.n = 0;
  __syncthreads();
  for (int64_t i = lo + t; i < hi; i += NT) {
    const uint32_t k = key_of((float)row[i]);
    if (k != 0u && pair_of(k, i) >= from) sh.list[atomicAdd(&sh.n, 1)] = pair_of(k, i);
  }
  __syncthreads();
  return sh.n;
}

// ------------------------------------------------------------------ forward
// The sums of the row's elements [lo, hi), this thread's share: vectors of 8 in turn.
template <typename T, int NT>
__device__ __forceinline__ void scan(const T* row, int64_t lo, int64_t hi, Sums& v) {
  constexpr int U = 4;  // vectors in flight
  const int64_t n8 = (hi - lo) / 8;
  const T* p = row + lo;
  int64_t i = threadIdx.x;
  for (; i + (U - 1) * NT < n8; i += U * NT) {
    Eight<T> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u].load(p + 8 * (i + u * NT));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = x[u].get(e);
      v.add8(z);
    }
  }
  for (; i < n8; i += NT) {
    Eight<T> x;
    x.load(p + 8 * i);
    float z[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = x.get(e);
    v.add8(z);
  }
  const int rest = (int)((hi - lo) - 8 * n8);
  if (rest && threadIdx.x == n8 % NT) {
    float z[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = e < rest ? (float)p[8 * n8 + e] : -INFINITY;
    v.add8(z);
  }
}

// The same, with the largest logit of each half of the thread's share for the alternatives.
template <typename T, int NT, bool TOP>
__device__ __forceinline__ void scan_halves(const T* row, int64_t lo, int64_t hi, Sums& v, float& mx0, float& mx1) {
  if constexpr (TOP) {
    int64_t mid = lo + 8 * NT * first_half<NT>((hi - lo) / 8);
    if (mid > hi) mid = hi;
    scan<T, NT>(row, lo, mid, v);
    mx0 = v.mx;
    v.mx = -INFINITY;
    scan<T, NT>(row, mid, hi, v);
    mx1 = v.mx;
    v.mx = fmaxf(mx0, mx1);
  } else {
    scan<T, NT>(row, lo, hi, v);
  }
}

__device__ inline bool masked(const LogprobArgs& p, int64_t row) { return p.mask != nullptr && p.mask[row] == 0; }

// Everything of a masked row: zeros, ids -1.
__device__ inline void write_masked(const LogprobArgs& p, int64_t row, int t, int nt) {
  for (int i = t; i < p.T; i += nt) p.logp[row * p.T + i] = 0.f;
  for (int i = t; i < p.top; i += nt) {
    p.top_ids[row * p.top + i] = -1;
    p.top_logp[row * p.top + i] = 0.f;
  }
  if (t == 0) p.entropy[row] = p.stats[row] = p.stats[p.N + row] = 0.f;
}

template <typename T>
__device__ inline void write_row(const LogprobArgs& p, int64_t row, const RowResult& r, int t, int nt) {
  const T* x = (const T*)p.x + row * p.ld;
  for (int i = t; i < p.T; i += nt) {
    const int32_t id = p.ids[row * p.T + i];
    p.logp[row * p.T + i] = id >= 0 && id < p.V ? r.logp((float)x[id]) : 0.f;
  }
  if (t == 0) {
    p.entropy[row] = r.entropy;
    p.stats[row] = r.m;
    p.stats[p.N + row] = r.logs;
  }
}

// A row's alternatives from its n largest pairs in order; -1 where there are no more.
__device__ inline void write_top(const LogprobArgs& p, int64_t row, const u64* sorted, int n, const RowResult& r, int t,
                                 int nt) {
  for (int i = t; i < p.top; i += nt) {
    const u64 pair = i < n ? sorted[i] : 0;
    p.top_ids[row * p.top + i] = i < n ? pair_id(pair) : -1;
    p.top_logp[row * p.top + i] = i < n ? r.logp(key_value((uint32_t)(pair >> 32))) : -INFINITY;
  }
}

// (two workgroups of 1,024 threads a compute unit: 64 registers a lane)
template <typename T, int NT, bool TOP>
__global__ void __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(8))) logprob_kernel(LogprobArgs p) {
  __shared__ float red[48];
  const int64_t row = blockIdx.x;
  const int t = threadIdx.x;
  if (masked(p, row)) {
    write_masked(p, row, t, NT);
    return;
  }
  const T* x = (const T*)p.x + row * p.ld;
  Sums v;
  float mx0 = -INFINITY, mx1 = -INFINITY;
  scan_halves<T, NT, TOP>(x, 0, p.V, v, mx0, mx1);
  block_sums<NT>(v, red);
  const RowResult r(v);
  write_row<T>(p, row, r, t, NT);
  if constexpr (TOP) {
    __shared__ TopLds<NT> sh;
    int n = collect_top<T, NT>(x, 0, p.V, mx0, mx1, v.mx, p.top, sh);
    const u64* sorted = order_top<NT>(sh.list, sh.other, n, p.top, &sh.count[0], &sh.bound);
    write_top(p, row, sorted, n, r, t, NT);
  }
}

// A slice of a row (few rows): its sums, and its `top` largest pairs in order.
template <typename T, int NT, bool TOP>
__global__ void __launch_bounds__(NT) __attribute__((amdgpu_waves_per_eu(8))) logprob_slice_kernel(LogprobArgs p) {
  __shared__ float red[48];
  const int64_t row = blockIdx.x / (unsigned)p.slices;
  const int sl = (int)(blockIdx.x % (unsigned)p.slices), t = threadIdx.x;
  if (masked(p, row)) return;
  const T* x = (const T*)p.x + row * p.ld;
  const int64_t lo = sl * p.per, hi = lo + p.per < p.V ? lo + p.per : p.V;
  Sums v;
  float mx0 = -INFINITY, mx1 = -INFINITY;
  scan_halves<T, NT, TOP>(x, lo, hi, v, mx0, mx1);
  block_sums<NT>(v, red);
  if (t == 0) p.part[blockIdx.x] = make_float4(v.mx, v.m, v.s, v.a);
  if constexpr (TOP) {
    __shared__ TopLds<NT> sh;
    u64* out = (u64*)p.pairs + (int64_t)blockIdx.x * p.top;
    int n = collect_top<T, NT>(x, lo, hi, mx0, mx1, v.mx, p.top, sh);
    const u64* sorted = order_top<NT>(sh.list, sh.other, n, p.top, &sh.count[0], &sh.bound);
    for (int i = t; i < p.top; i += NT) out[i] = i < n ? sorted[i] : 0;
  }
}

// Joins a row's slices (2 to 64, and at most kList pairs).
template <typename T, int NT>
__global__ void __launch_bounds__(NT) logprob_join_kernel(LogprobArgs p) {
  __shared__ u64 list[kList], other[kList];
  __shared__ u64 least;
  __shared__ float got[3];
  __shared__ int found, count;
  __shared__ uint32_t reach;
  const int64_t row = blockIdx.x;
  const int t = threadIdx.x;
  if (masked(p, row)) {
    write_masked(p, row, t, NT);
    return;
  }
  const u64* pairs = (const u64*)p.pairs + row * p.slices * p.top;
  if (t < 64) {
    Sums v;
    if (t < p.slices) {
      const float4 q = p.part[row * p.slices + t];
      v.mx = q.x;
      v.m = q.y;
      v.s = q.z;
      v.a = q.w;
    }
    if (p.top) {
      // Of the slices' q-th largest pairs, the r-th largest is a bound that q r >=
      // top pairs reach; q about 2 top / slices, so that r is about half the slices.
      const int q = (2 * p.top + p.slices - 1) / p.slices < p.top ? (2 * p.top + p.slices - 1) / p.slices : p.top;
      const int r = (p.top + q - 1) / q;
      const u64 v = t < p.slices ? pairs[t * p.top + q - 1] : 0;
      const uint32_t hi = (uint32_t)(v >> 32);
      uint32_t best = 0;
#pragma unroll
      for (int b = 31; b >= 0; --b) {
        const uint32_t next = best | (1u << b);
        if (__builtin_popcountll(__ballot(hi >= next)) >= r) best = next;
      }
      if (t == 0) least = (u64)best << 32 > 1 ? (u64)best << 32 : 1;
    }
    v.mx = wave_max(v.mx);
    v.move(fmaxf(v.mx, kLowest));
    v.s = lanes_sum(v.s, 64);
    v.a = lanes_sum(v.a, 64);
    if (t == 0) {
      got[0] = v.mx;
      got[1] = v.s;
      got[2] = v.a;
      found = 0;
    }
  }
  __syncthreads();
  Sums v;
  v.mx = got[0];
  v.s = got[1];
  v.a = got[2];
  const RowResult r(v);
  write_row<T>(p, row, r, t, NT);
  if (p.top == 0) return;
  const u64 bound = least;
  for (int i = t; i < p.slices * p.top; i += NT) {
    const u64 pair = pairs[i];
    if (pair >= bound) list[atomicAdd(&found, 1)] = pair;
  }
  __syncthreads();
  int n = found;
  const u64* sorted = order_top<NT>(list, other, n, p.top, &count, &reach);
  write_top(p, row, sorted, n, r, t, NT);
}

// ------------------------------------------------------------------ gradient
constexpr int kGradThreads = 256, kGradVec = 4;
constexpr int kGradRun = kGradThreads * kGradVec * 8;  // logits of a row per workgroup

__device__ inline bool in_row(int32_t id, int64_t V) { return id >= 0 && id < V; }

// -p (c + u l), l = log p
__device__ inline float grad_of(float z, float m, float logs, float c, float u) {
  const float l = not_far((z - m) - logs);
  return -exp_fast(l) * __builtin_fmaf(u, l, c);
}

template <typename T>
__global__ void __launch_bounds__(kGradThreads) logprob_grad_kernel(LogprobGradArgs p) {
  extern __shared__ int32_t lds[];  // T > 1: the row's ids, then their weights
  __shared__ float red[kGradThreads / 64];
  const unsigned runs = (unsigned)p.runs, at_row = blockIdx.x / runs;
  const int64_t row = at_row, lo = (int64_t)(blockIdx.x - at_row * runs) * kGradRun, hi = lo + kGradRun < p.V ? lo + kGradRun : p.V;
  const int t = threadIdx.x;
  const T* x = (const T*)p.x + row * p.ld;
  T* out = (T*)p.out + row * p.ldo;
  const float m = p.stats[row], logs = p.stats[p.N + row];
  const bool off = (p.mask != nullptr && p.mask[row] == 0) || m == -INFINITY;
  const float u = p.dentropy != nullptr && !off ? p.dentropy[row] : 0.f;
  float w = 0.f;  // the sum of the given tokens' weights
  int32_t mine[kMaxK / kGradThreads];
  float add[kMaxK / kGradThreads], zt[kMaxK / kGradThreads];
  int nm = 0;     // given ids of this run whose first mention is this thread's
  if (p.T == 1) {
    const int32_t id = p.ids[row];
    if (in_row(id, p.V) && !off) {
      w = p.dlogp[row];
      if (t == 0 && id >= lo && id < hi) {
        mine[0] = id;
        add[0] = w;
        zt[0] = (float)x[id];
        nm = 1;
      }
    }
  } else if (p.T > 1 && !off) {
    float* lw = (float*)(lds + p.T);
    for (int i = t; i < p.T; i += kGradThreads) {
      const int32_t id = p.ids[row * p.T + i];
      const bool in = in_row(id, p.V);
      lds[i] = in ? id : -1;
      lw[i] = in ? p.dlogp[row * p.T + i] : 0.f;
      w += lw[i];
    }
    w = lanes_sum(w, 64);
    if ((t & 63) == 0) red[t >> 6] = w;
    __syncthreads();
    w = 0.f;
#pragma unroll
    for (int i = 0; i < kGradThreads / 64; ++i) w += red[i];
    for (int q = 0; q < kMaxK / kGradThreads; ++q) {
      const int i = t + q * kGradThreads;
      if (i >= p.T) break;
      const int32_t id = lds[i];
      if (id < lo || id >= hi) continue;
      bool first = true;
      float sum = 0.f;
      for (int j = 0; j < p.T; ++j)
        if (lds[j] == id) {
          if (j < i) first = false;
          sum += lw[j];
        }
      if (!first) continue;
      mine[nm] = id;
      add[nm] = sum;
      zt[nm++] = (float)x[id];
    }
  }
  // the logits at given ids are read before the run is written (out may be x)
  if (p.T > 0) __syncthreads();
  const float c = __builtin_fmaf(u, p.entropy != nullptr && !off ? p.entropy[row] : 0.f, w);
  if (lo + kGradRun <= p.V) {
    Eight<T> v[kGradVec];
#pragma unroll
    for (int i = 0; i < kGradVec; ++i)
      if (!off) v[i].load(x + lo + 8 * (t + i * kGradThreads));
#pragma unroll
    for (int i = 0; i < kGradVec; ++i) {
      float g[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = off ? 0.f : grad_of(v[i].get(e), m, logs, c, u);
      v[i].set(g);
      v[i].store(out + lo + 8 * (t + i * kGradThreads));
    }
  } else {
    for (int64_t at = lo + 8 * t; at < hi; at += 8 * kGradThreads) {
      if (at + 8 <= hi) {
        Eight<T> v;
        if (!off) v.load(x + at);
        float g[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = off ? 0.f : grad_of(v.get(e), m, logs, c, u);
        v.set(g);
        v.store(out + at);
      } else {
        for (int64_t j = at; j < hi; ++j) out[j] = (T)(off ? 0.f : grad_of((float)x[j], m, logs, c, u));
      }
    }
  }
  if (p.T == 0) return;
  __syncthreads();
  for (int q = 0; q < nm; ++q) out[mine[q]] = (T)(add[q] + grad_of(zt[q], m, logs, c, u));
}

template <typename T, int NT, bool TOP>
void logprob_rows(const LogprobArgs& p, hipStream_t s) {
  hipLaunchKernelGGL((logprob_kernel<T, NT, TOP>), dim3((unsigned)p.N), dim3(NT), 0, s, p);
}

template <typename T>
hipError_t logprob_of(const LogprobArgs& p, hipStream_t s) {
  if (p.slices > 1) {
    const dim3 grid((unsigned)(p.N * p.slices));
    if (p.top > kWideTop)
      hipLaunchKernelGGL((logprob_slice_kernel<T, 512, true>), grid, dim3(512), 0, s, p);
    else if (p.top)
      hipLaunchKernelGGL((logprob_slice_kernel<T, 256, true>), grid, dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((logprob_slice_kernel<T, 256, false>), grid, dim3(256), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((logprob_join_kernel<T, 256>), dim3((unsigned)p.N), dim3(256), 0, s, p);
    return hipGetLastError();
  }
  if (p.top == 0) {
    if (p.V <= 1024)
      logprob_rows<T, 64, false>(p, s);
    else if (p.V <= 8192)
      logprob_rows<T, 256, false>(p, s);
    else
      logprob_rows<T, 1024, false>(p, s);
  } else if (p.V <= 1024) {
    logprob_rows<T, 64, true>(p, s);
  } else if (p.V <= 8192 && p.top <= kWideTop) {
    logprob_rows<T, 256, true>(p, s);
  } else {
    logprob_rows<T, 512, true>(p, s);
  }
  return hipGetLastError();
}

}  // namespace

// Slices of a row: enough for four workgroups a compute unit, at least 2,048
// logits each, at most 64, and no more pairs than the join holds.
int logprob_slices(int64_t N, int64_t V, int top) {
  if (N <= 0 || N >= 256 || V < 8192) return 1;
  int64_t s = 1024 / N;
  if (s > 64) s = 64;
  if (s > V / 2048) s = V / 2048;
  if (top > 0 && s > kList / top) s = kList / top;
  return s > 1 ? (int)s : 1;
}

uint64_t logprob_workspace(int64_t N, int64_t V, int top) {
  const int s = logprob_slices(N, V, top);
  return s > 1 ? (uint64_t)N * s * (16 + 8 * (uint64_t)top) : 0;
}

hipError_t launch_logprob(Dtype dt, LogprobArgs p, void* ws, hipStream_t s) {
  p.slices = ws != nullptr ? logprob_slices(p.N, p.V, p.top) : 1;
  p.per = ((p.V + p.slices - 1) / p.slices + 7) / 8 * 8;
  if (p.slices > 1) p.slices = (int)((p.V + p.per - 1) / p.per);
  p.part = (float4*)ws;
  p.pairs = (char*)ws + (uint64_t)p.N * p.slices * 16;
  return dt == DT_BF16 ? logprob_of<__bf16>(p, s) : logprob_of<float>(p, s);
}

int64_t logprob_grad_blocks(int64_t N, int64_t V) { return N * ((V + kGradRun - 1) / kGradRun); }

hipError_t launch_logprob_grad(Dtype dt, LogprobGradArgs p, hipStream_t s) {
  p.runs = (p.V + kGradRun - 1) / kGradRun;
  const dim3 grid((unsigned)logprob_grad_blocks(p.N, p.V));
  const size_t lds = p.T > 1 ? (size_t)p.T * 8 : 0;
  if (dt == DT_BF16)
    hipLaunchKernelGGL((logprob_grad_kernel<__bf16>), grid, dim3(kGradThreads), lds, s, p);
  else
    hipLaunchKernelGGL((logprob_grad_kernel<float>), grid, dim3(kGradThreads), lds, s, p);
  return hipGetLastError();
}

}  // namespace ckl
