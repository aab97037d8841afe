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
// A token changes where its border moves, so exponentials are fp64 and sums 64-bit
// integers (in any order the same) and fp64.  The integers of the general path
// hold a token's mass to half a unit of 2^-min(51, 62 - ceil(log2 V)) of its bin's
// edge and equal logits round alike, so borders are held to V / 2^62 of the total
// (4e-14 at 201,088 tokens), plus 5e-15 of the exponentials.  Counted rows may
// leave out 1e-13 of it.
//
// The floor is reading a row once.  One workgroup of 1024 threads takes a row:
//  1. bf16 rows (count_kernel): a count of every value, one LDS add per logit,
//     from which all borders follow; then the drawn token, the n-th logit of
//     its value, is looked for in the third of the row that holds it.  N <= 64
//     rows of 32,768 logits and more are counted by several workgroups each
//     (count_slice_kernel, count_finish_kernel).
//  2. The general path (sample_kernel): fp32 rows, bf16 rows that counting
//     leaves (logits beyond +-256 that matter, and the like), and a few bf16
//     rows of which few tokens are wanted (direct_bf16).  First the largest
//     logit, then
//   a. 1 <= k <= 512: the k-th largest of the threads' maxima is a bound that
//     at least k tokens reach; the tokens that do are collected, sorted in LDS,
//     and one wave does everything else there;
//   b. otherwise a histogram of the row's mass over 4096 bins, 1/64 octave of
//     e each (64 octaves: what lies below weighs less than 2^-64 a token).
//     Within a bin the masses e / (upper edge) lie in (2^-1/64, 1], so a short
//     polynomial gives them and 64-bit integers sum them with one relative
//     rounding.  Each border (k, then p, then u) falls into one bin, whose
//     tokens are collected and sorted in LDS; a bin with more tokens than fit
//     there is narrowed by 8 bits of the key at a time first, and where only
//     equal logits are left the border is a count, and the token is found by
//     its rank in id order.
//
// Measured (MI355X):
//  1,024 x 201,088 bf16, no limit: 100 us, 4.1 TB/s of the logits (80 us for
//    the counting, the rest what follows a workgroup's last load; by the
//    histogram of 2b 890 us).
//  512 x 128,256 bf16, top-p: 42 us, 3.1 TB/s.
//  1 x 201,088 bf16, top-k 50: 18 us, latency: one compute unit reads the row.
//  61 x 32,000 fp32, limits of each row's own: 29 us, the rows without a top-k
//    in 2b, half of it fp64 arithmetic on the row's one compute unit (with
//    top-k 200: 16 us by 2a).
//  1,024 x 201,088 fp32, no limit: 436 us, 1.9 TB/s, bound by the 64-bit LDS
//    adds of 2b and the fp64 polynomial (with top-k 50, by 2a: 185 us).
//  A bf16 row that counting leaves to the general path keeps its compute unit
//    busy for 40 to 100 us more: 1,024 x 201,088 normal logits of deviation 1, 3
//    of which rows hold a nonzero one below 2^-24, take 192 us.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "launch.hpp"

namespace ckl {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 4096;
constexpr int kPerThread = kBins / kThreads;
constexpr int kCap = 2048;      // tokens held in LDS
constexpr int kFastK = 512;     // largest k of the collected path
constexpr int kTopBits = 13;    // key bits of the histogram of the threads' maxima
constexpr int kFlight = 4;      // 16-byte loads of a thread in flight
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

// The larger of two logits, NaN if either is.  (fmaxf would go on from what comes
// after a signalling NaN, and forget the largest before it.  Comparisons, which
// leave NaN out at once, made one row of 201,088 bf16 logits 26 us for 18.)
__device__ inline float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// A value that is the same in every lane, in scalar registers.
__device__ inline uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ inline float uniform(float v) { return __builtin_bit_cast(float, uniform(__builtin_bit_cast(uint32_t, v))); }
__device__ inline double uniform(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)uniform((uint32_t)(b >> 32)) << 32 | uniform((uint32_t)b));
}
// A lane's value, the lane being the same for all.
__device__ inline uint32_t of_lane(uint32_t v, int l) { return (uint32_t)__builtin_amdgcn_readlane((int)v, l); }
__device__ inline double of_lane(double v, int l) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)of_lane((uint32_t)(b >> 32), l) << 32 | of_lane((uint32_t)b, l));
}

// A row as its 16-byte aligned chunks, `nb` of them, with the fewer than kN
// elements before the first one and after the last one apart.
template <typename T>
struct Row {
  static constexpr int kN = 16 / (int)sizeof(T);
  const T* x;
  const u32x4_t* body;
  int64_t V;
  int head, tail;
  uint32_t nb;
  __device__ inline Row(const T* row, int64_t v) : x(row), V(v) {
    const int skip = (int)((0 - (uintptr_t)row) & 15) / (int)sizeof(T);
    head = skip < v ? skip : (int)v;
    nb = (uint32_t)((v - head) / kN);
    tail = (int)(v - head - (int64_t)nb * kN);
    body = (const u32x4_t*)(row + head);
  }
  __device__ inline int64_t body_id(uint32_t c) const { return head + (int64_t)c * kN; }
  __device__ inline int64_t tail_id() const { return body_id(nb); }
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
  // NaN where one of them is
  __device__ static inline float largest(const u32x4_t& v) {
    float f[kN];
    unpack(v, f);
#pragma unroll
    for (int i = 1; i < kN; ++i) f[0] = larger(f[0], f[i]);
    return f[0];
  }
};

// Every chunk of the row as chunk(words, index), the chunks of a thread in
// turn with kFlight loads in flight each (past the end the last chunk is loaded
// again and left out: a load under a condition would wait for the one before),
// and every element apart as one(element, id).
template <int kFlight, typename T, typename C, typename O>
__device__ inline void for_each_chunk(const Row<T>& row, C&& chunk, O&& one) {
  const uint32_t tid = threadIdx.x;
  for (uint32_t c0 = tid; c0 < row.nb; c0 += kFlight * kThreads) {
    u32x4_t v[kFlight];
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const uint32_t c = c0 + j * kThreads;
      v[j] = row.body[c < row.nb ? c : row.nb - 1];
    }
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const uint32_t c = c0 + j * kThreads;
      if (c < row.nb) chunk(v[j], c);
    }
  }
  if (tid < (uint32_t)row.head) one(row.x[tid], (int64_t)tid);
  if (tid < (uint32_t)row.tail) one(row.x[row.tail_id() + tid], row.tail_id() + tid);
}

// Every value of the row as fn(value, id).
template <typename T, typename F>
__device__ inline void for_each(const Row<T>& row, F&& fn) {
  for_each_chunk<kFlight>(
      row,
      [&](const u32x4_t& v, uint32_t c) {
        float f[Row<T>::kN];
        Row<T>::unpack(v, f);
#pragma unroll
        for (int i = 0; i < Row<T>::kN; ++i) fn(f[i], row.body_id(c) + i);
      },
      [&](T x, int64_t id) { fn((float)x, id); });
}

// The masses of one row.  y = -64 log2(e) of a logit, in fp64; its bin is the
// whole part of the same in fp32 (monotone in the logit and within 1e-3 of y,
// at a fifth of the cost), so that y - bin lies in [-1e-3, 1 + 1e-3].
struct Scale {
  double mx, c;        // c = 64 log2(e) / T
  double fix, inv_fix; // 2^shift of the integer masses, and its inverse
  float mxf, cf;
  bool inf;            // the largest logit is +inf: equal ones weigh 1, all others nothing
  bool wide;           // c or the logits' differences may leave fp32's range
  __device__ inline void set(float m, double over_t, int fix_bits) {
    inf = m == INFINITY;
    mx = (double)m;
    c = over_t;
    fix = (double)(1ull << fix_bits);
    inv_fix = 1.0 / fix;
    mxf = m;
    cf = (float)c;
    wide = !(c > 1e-30 && c < 1e30);
  }
  __device__ inline double y(float l) const {
    if (inf) return l == INFINITY ? 0.0 : (double)INFINITY;
    // -inf (and NaN, by the comparison below being false) weighs nothing
    return l > -INFINITY ? (mx - (double)l) * c : (double)INFINITY;
  }
  // a logit's place among the bins; kBins and more, or NaN, where it has none
  // (-inf and NaN never have one).  kPlain: neither inf nor wide.
  template <bool kPlain>
  __device__ inline float place(float l) const {
    if constexpr (kPlain) return (mxf - l) * cf;
    if (inf) return l == INFINITY ? 0.f : INFINITY;
    return (float)((mx - (double)l) * c);
  }
  // y - bin of a logit in that bin
  template <bool kPlain>
  __device__ inline double frac(float l, int bin) const {
    if (!kPlain && inf) return 0.0;
    return __builtin_fma(mx - (double)l, c, -(double)bin);
  }
  // fn(true_type) for plain rows, fn(false_type) for the others: the choice is
  // made once per pass over the row
  template <typename F>
  __device__ inline void either(F&& fn) const {
    if (!inf && !wide)
      fn(std::true_type{});
    else
      fn(std::false_type{});
  }
};

// 2^(-f / 64) for f in [-1e-3, 1 + 1e-3]: the polynomial of degree 4 through the
// Chebyshev points of [0, 1], its constant moved to 1 so that f = 0 is exact;
// off by at most 5e-15.
__device__ inline double pow_frac(double f) {
  double r = 5.701897951327709e-10;
  r = __builtin_fma(r, f, -2.1172866563406743e-07);
  r = __builtin_fma(r, f, 5.864904858456656e-05);
  r = __builtin_fma(r, f, -0.010830424696128419);
  return __builtin_fma(r, f, 1.0);
}

// Room for the block-wide reductions, and a table for mass_of.
struct Red {
  double d[kWaves];
  uint32_t u[kWaves];
  float f[kWaves];
  double pow64[64];  // 2^(-j / 64)
};
__device__ inline void fill_pow64(Red& red) {
  if (threadIdx.x < 64) red.pow64[threadIdx.x] = exp2(-(double)threadIdx.x / 64.0);
}
__device__ inline double bin_top(const Red& red, int b) { return ldexp(red.pow64[b & 63], -(b >> 6)); }
// e of a logit whose y is below kBins, else 0; here 2^(-f / 64) is its Taylor
// polynomial of degree 6 (off by 4e-18), as a product of such values follows
__device__ inline double mass_of(const Red& red, double y) {
  if (!(y < (double)kBins)) return 0.0;
  const double b = floor(y), f = (y - b) * -0.01083042469624914;  // ln 2 / 64
  double r = 1.0 / 720;
  r = __builtin_fma(r, f, 1.0 / 120);
  r = __builtin_fma(r, f, 1.0 / 24);
  r = __builtin_fma(r, f, 1.0 / 6);
  r = __builtin_fma(r, f, 0.5);
  r = __builtin_fma(r, f, 1.0);
  return bin_top(red, (int)b) * __builtin_fma(r, f, 1.0);
}

// A row's settings; in LDS, where they take no registers through the passes.
struct Settings {
  double p, min_p, u;
  double c;  // 64 log2(e) / T
  bool limit;
  uint32_t k;
};
struct Shared {
  Settings how;
  uint64_t mass[kBins];       // integer masses relative to each bin's upper edge, then (fp64) masses
  uint32_t count[kBins];      // tokens per bin (kept while k limits)
  uint64_t cand[kCap];        // collected (key, id)
  uint64_t sub_mass[kSub];    // a narrowing pass
  uint32_t sub_count[kSub];
  Red red;
  uint64_t edge_mass[3];      // mass of the tokens of min_p's bin and of its neighbours that reach it
  uint32_t n_cand;
  uint32_t pick;
  double pick_mass;           // mass above the chosen bin or digit
  uint32_t pick_count;        // tokens above it
  double got_mass;
};

__device__ inline float block_max(float v, Red& red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red.f[threadIdx.x >> 6] = v;
  __syncthreads();
  float m = red.f[0];
#pragma unroll
  for (int i = 1; i < kWaves; ++i) m = fmaxf(m, red.f[i]);
  return m;
}

// Inclusive sum over the lanes of a wave (lane order, one fixed order of
// additions): four steps within rows of 16 lanes, two across them.
template <int kCtrl, int kRows>
__device__ inline uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, kRows, 0xF, false);
}
template <int kCtrl, int kRows>
__device__ inline double dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = dpp<kCtrl, kRows>((uint32_t)b), hi = dpp<kCtrl, kRows>((uint32_t)(b >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
template <typename N>
__device__ inline N wave_scan(N x) {
  x += dpp<0x111, 0xF>(x);  // row_shr:1
  x += dpp<0x112, 0xF>(x);
  x += dpp<0x114, 0xF>(x);
  x += dpp<0x118, 0xF>(x);
  x += dpp<0x142, 0xA>(x);  // row_bcast:15 into rows 1 and 3
  x += dpp<0x143, 0xC>(x);  // row_bcast:31 into rows 2 and 3
  return x;
}

// Sum of v over the threads before this one (thread order), and over all of
// them, in one fixed order.
__device__ inline double block_prefix(double v, Red& red, double* before) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const double x = wave_scan(v);
  __syncthreads();
  if (lane == 63) red.d[w] = x;
  __syncthreads();
  double base = 0.0, all = 0.0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (i == w) base = all;
    all += red.d[i];
  }
  const double prev = __shfl_up(x, 1);
  *before = lane == 0 ? base : base + prev;
  return all;
}
__device__ inline uint32_t block_prefix(uint32_t v, Red& red, uint32_t* before) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const uint32_t x = wave_scan(v);
  __syncthreads();
  if (lane == 63) red.u[w] = x;
  __syncthreads();
  uint32_t base = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (i == w) base = all;
    all += red.u[i];
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
#pragma unroll 8
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

// *slot = the least v of the threads with `hit`, v growing with the thread: one
// atomic per wave (one per thread would pass through the LDS one by one).
__device__ inline void min_of_hits(bool hit, uint32_t v, uint32_t* slot) {
  const uint64_t m = __ballot(hit);
  if (hit && (threadIdx.x & 63) == __builtin_ctzll(m)) atomicMin(slot, v);
}
__device__ inline void max_of_hits(bool hit, uint32_t v, uint32_t* slot) {
  const uint64_t m = __ballot(hit);
  if (hit && (threadIdx.x & 63) == 63 - __builtin_clzll(m)) atomicMax(slot, v);
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
  constexpr int kEach = kCap / kThreads;  // tokens of a thread
  double e[kEach], mine = 0.0;
  const int b = threadIdx.x * kEach;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    e[i] = b + i < n ? mass_of(sh.red, sc.y(Key<T>::value((uint32_t)(sh.cand[b + i] >> 32)))) : 0.0;
    mine += e[i];
  }
  double before = 0.0;
  block_prefix(mine, sh.red, &before);
  if (threadIdx.x == 0) sh.pick = 0xFFFFFFFFu;
  __syncthreads();
  double run = above + before;
  int at = -1;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    run += e[i];
    if (at < 0 && b + i < n && reached(kind, above_n + (uint32_t)(b + i + 1), run, k, target)) at = b + i;
  }
  min_of_hits(at >= 0, (uint32_t)at, &sh.pick);
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

// Which values of a 16-byte chunk equal l (bit i: value i).
__device__ inline uint32_t equal_in(const u32x4_t& v, float l, float*) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = v[i];
    m |= (uint32_t)(__builtin_bit_cast(float, w) == l) << i;
  }
  return m;
}
__device__ inline uint32_t equal_in(const u32x4_t& v, float l, __bf16*) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = v[i];
    m |= (uint32_t)(__builtin_bit_cast(float, w << 16) == l) << (2 * i);
    m |= (uint32_t)(__builtin_bit_cast(float, w & 0xFFFF0000u) == l) << (2 * i + 1);
  }
  return m;
}
// Whether any may: no more for fp32; for bf16 one test for pairs (l's bits in
// both halves; 0 stands for either zero).
__device__ inline bool may_equal(const u32x4_t& v, float l, float* t) { return equal_in(v, l, t) != 0; }
__device__ inline bool may_equal(const u32x4_t& v, float l, __bf16*) {
  const uint32_t h = __builtin_bit_cast(uint32_t, l) >> 16;
  const uint32_t mask = l == 0.f ? 0x7FFF7FFFu : 0xFFFFFFFFu, want = l == 0.f ? 0u : h << 16 | h;
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 z = {0xFFFF, 0xFFFF};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = v[i];
    z = __builtin_elementwise_min(z, __builtin_bit_cast(u16x2, (w & mask) ^ want));
  }
  return z[0] == 0 || z[1] == 0;
}

// The id of the r-th token (1 <= r <= n) of the n of logit l in id order, in
// every thread.  A wave reads 64 chunks (a piece) at once, the workgroup 64
// pieces a round, from the row's nearer end (by r among n); the wave that holds
// the r-th finds it among its own.  room: kNthRoom words of LDS.
constexpr int kNthPieces = 64;
constexpr int kNthRoom = 2 * kNthPieces + 1;  // the pieces' counts of two rounds in turn, and the id
template <typename T>
__device__ __forceinline__ int64_t nth_equal(const Row<T>& row, uint32_t* room, float l, uint32_t r, uint32_t n) {
  constexpr int U = kNthPieces / kWaves;
  const uint32_t lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  // the r-th set bit of a mask of lanes
  auto nth_lane = [](uint64_t m, uint32_t n) {
    for (; n > 1; --n) m &= m - 1;
    return __builtin_ctzll(m);
  };
  // the lanes whose element of the n at `first` equals l
  auto equal_at = [&](int64_t first, int n) -> uint64_t {
    if (n == 0) return 0;
    const bool in = (int)lane < n;
    return __ballot(in && (float)row.x[first + (in ? (int)lane : 0)] == l);
  };
  const uint64_t head = equal_at(0, row.head), tail = equal_at(row.tail_id(), row.tail);
  const uint32_t nh = (uint32_t)__popcll(head), in_body = n - nh - (uint32_t)__popcll(tail);
  if (r <= nh) return nth_lane(head, r);
  r -= nh;
  if (r > in_body) return row.tail_id() + nth_lane(tail, r - in_body);
  const uint32_t pieces = (row.nb + 63) / 64;
  const bool back = r > in_body - r + 1;  // pieces in falling order: the r-th is the (in_body - r + 1)-th
  if (back) r = in_body - r + 1;
  __syncthreads();
  uint32_t* cnt = room;
  for (uint32_t done = 0; done < pieces; done += kNthPieces) {
    u32x4_t v[U];
    uint32_t c[U], m[U], upto[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const uint32_t o = done + j * kWaves + w;
      c[j] = (o >= pieces ? pieces : back ? pieces - 1 - o : o) * 64 + lane;
      v[j] = row.body[c[j] < row.nb ? c[j] : row.nb - 1];
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const bool may = c[j] < row.nb && may_equal(v[j], l, (T*)nullptr);
      m[j] = upto[j] = 0;
      if (__ballot(may) != 0) {
        m[j] = may ? equal_in(v[j], l, (T*)nullptr) : 0;
        upto[j] = wave_scan((uint32_t)__popc(m[j]));
      }
      if (lane == 63) cnt[j * kWaves + w] = upto[j];
    }
    __syncthreads();
    const uint32_t mine = cnt[lane], sum = wave_scan(mine);
    const uint64_t here = __ballot(sum - mine < r && sum >= r);
    if (here) {
      const int at = __builtin_ctzll(here);
      const uint32_t of = of_lane(mine, at);
      uint32_t in = r - (of_lane(sum, at) - of);
      if (back) in = of - in + 1;
      if ((uint32_t)at % kWaves == w) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
          if (at / kWaves != j) continue;
          uint32_t skip = in - 1 - (upto[j] - (uint32_t)__popc(m[j]));  // wraps where it lies in an earlier lane
          if (skip < (uint32_t)__popc(m[j])) {
            for (; skip > 0; --skip) m[j] &= m[j] - 1;
            room[2 * kNthPieces] = (uint32_t)row.body_id(c[j]) + (uint32_t)__builtin_ctz(m[j]);
          }
        }
      }
      __syncthreads();
      return (int64_t)uniform(room[2 * kNthPieces]);
    }
    r -= of_lane(sum, 63);
    cnt = cnt == room ? room + kNthPieces : room;
  }
  return -1;  // not reached: the row holds n such logits
}

// The smallest r in [1, n] for which above + r e reaches the target, n if none:
// how many of n equal logits a border takes.
__device__ inline uint32_t equal_taken(int kind, uint32_t n, uint32_t above_n, double above, double e, uint32_t k,
                                       double target) {
  if (kind == BY_COUNT) return k > above_n ? (k - above_n < n ? k - above_n : n) : 1;
  uint32_t lo = 1, hi = n;
  // the quotient, where the sums' rounding leaves it within one, spares most steps
  const double g = (target - above) / e;
  if (g > 2.0 && g < (double)n - 2.0) {
    const uint32_t a = (uint32_t)g - 1;
    if (!reached(kind, 0, above + (double)a * e, 0, target)) lo = a + 1;
    if (reached(kind, 0, above + (double)(a + 3) * e, 0, target)) hi = a + 3;
  }
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (reached(kind, 0, above + (double)mid * e, 0, target))
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// Where a border lies: the mass of the prefix that ends there, and the last
// token of that prefix.
struct Found {
  double mass;
  float logit;
  int64_t id;
};

// before, cbefore: mass and (for BY_COUNT) tokens of the bins of earlier threads.
template <typename T>
__device__ __forceinline__ Found find_border(const Row<T>& row, Shared& sh, const Scale& sc, int kind, uint32_t k,
                                             double target, double before, uint32_t cbefore, bool want_id) {
  const int tid = threadIdx.x;
  // 1. the bin: thread t holds the bins [kPerThread t, kPerThread (t + 1))
  const double* mass = (const double*)sh.mass;
  if (tid == 0) sh.pick = 0xFFFFFFFFu;
  __syncthreads();
  // the first bin at whose end the border is reached, else the last with mass
  int at = -1, last = -1;
  double run = before;
  uint32_t crun = cbefore;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = tid * kPerThread + i;
    run += mass[b];
    crun += kind == BY_COUNT ? sh.count[b] : 0;
    if (mass[b] != 0.0) {
      last = b;
      if (at < 0 && reached(kind, crun, run, k, target)) at = b;
    }
  }
  min_of_hits(at >= 0, (uint32_t)at, &sh.pick);
  __syncthreads();
  if (sh.pick == 0xFFFFFFFFu) {
    __syncthreads();
    if (tid == 0) sh.n_cand = 0;
    __syncthreads();
    max_of_hits(last >= 0, (uint32_t)last, &sh.n_cand);
    __syncthreads();
    if (tid == 0) sh.pick = sh.n_cand;
    __syncthreads();
  }
  const int bin = (int)uniform(sh.pick);
  if (bin / kPerThread == tid) {
    double r = before;
    uint32_t c = cbefore;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      if (tid * kPerThread + i < bin) {
        r += mass[tid * kPerThread + i];
        c += kind == BY_COUNT ? sh.count[tid * kPerThread + i] : 0;
      }
    }
    sh.pick_mass = r;
    sh.pick_count = c;
  }
  __syncthreads();
  double above = uniform(sh.pick_mass);
  uint32_t above_n = uniform(sh.pick_count);
  const double top = uniform(bin_top(sh.red, bin));
  const float p0 = (float)bin, p1 = (float)(bin + 1);
  // 2. the bin's tokens, narrowed by key digits until they fit
  uint32_t prefix = 0, prefix_mask = 0;
  int digits_left = Key<T>::kBits;
  for (;;) {
    __syncthreads();
    if (tid == 0) sh.n_cand = 0;
    __syncthreads();
    sc.either([&](auto plain) {
      for_each(row, [&](float l, int64_t id) {
        const float place = sc.template place<plain.value>(l);
        if (place >= p0 && place < p1) {
          const uint32_t key = Key<T>::of(l);
          if ((key & prefix_mask) == prefix) {
            const uint32_t slot = atomicAdd(&sh.n_cand, 1u);
            if (slot < (uint32_t)kCap) sh.cand[slot] = pack(key, (uint32_t)id);
          }
        }
      });
    });
    __syncthreads();
    const uint32_t n = uniform(sh.n_cand);
    if (n == 1) {  // the usual case of a short row
      const uint64_t c = sh.cand[0];
      const float l = uniform(Key<T>::value((uint32_t)(c >> 32)));
      return Found{above + mass_of(sh.red, sc.y(l)), l, (int64_t)unpack_id(c)};
    }
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
    sc.either([&](auto plain) {
      for_each(row, [&](float l, int64_t) {
        const float place = sc.template place<plain.value>(l);
        if (place >= p0 && place < p1) {
          const uint32_t key = Key<T>::of(l);
          if ((key & prefix_mask) == prefix) {
            const uint32_t dg = 255u - ((key >> digits_left) & 255u);
            atomicAdd((unsigned long long*)&sh.sub_mass[dg],
                      (unsigned long long)(pow_frac(sc.template frac<plain.value>(l, bin)) * sc.fix + 0.5));
            atomicAdd(&sh.sub_count[dg], 1u);
          }
        }
      });
    });
    __syncthreads();
    const double dm = tid < kSub && sh.sub_count[tid] ? (double)sh.sub_mass[tid] * sc.inv_fix * top : 0.0;
    const uint32_t dc = tid < kSub ? sh.sub_count[tid] : 0;
    double db = 0.0;
    uint32_t cb = 0;
    block_prefix(dm, sh.red, &db);
    block_prefix(dc, sh.red, &cb);
    if (tid == 0) {
      sh.pick = 0xFFFFFFFFu;
      sh.n_cand = 0;
    }
    __syncthreads();
    min_of_hits(dc && reached(kind, above_n + cb + dc, above + db + dm, k, target), (uint32_t)tid, &sh.pick);
    max_of_hits(dc != 0, (uint32_t)tid, &sh.n_cand);
    __syncthreads();
    const uint32_t dg = uniform(sh.pick == 0xFFFFFFFFu ? sh.n_cand : sh.pick);
    if ((uint32_t)tid == dg) {
      sh.pick_mass = above + db;
      sh.pick_count = above_n + cb;
    }
    __syncthreads();
    above = uniform(sh.pick_mass);
    above_n = uniform(sh.pick_count);
    prefix |= (255u - dg) << digits_left;
    prefix_mask |= 255u << digits_left;
  }

  // 3. more equal logits than fit: each weighs e, and the border is a count of
  // them (at least 1, at most n)
  const uint32_t n = sh.n_cand;
  const float l = Key<T>::value(prefix);
  const double e = mass_of(sh.red, sc.y(l));
  const uint32_t r = equal_taken(kind, n, above_n, above, e, k, target);
  Found f{above + (double)r * e, l, -1};
  if (!want_id) return f;
  f.id = nth_equal(row, (uint32_t*)sh.cand, l, r, n);
  return f;
}

// ---------------------------------------------------------------- bf16 rows
// bf16 logits have few distinct values, so a row is its count of every value:
// one pass with a 32-bit LDS add per logit, no exponential and no maximum
// before it, and each border is exact from count x e of the values in order.
// Counted one by one are the magnitudes in [2^-24, 2^8) of either sign; 0 and
// smaller ones are one count, larger ones another, so that a logit's place is
// eight packed 16-bit operations for two logits, without a branch.  Where
// logits beyond +-256 matter, or nonzero ones below 2^-24 do (by 1e-13 of the
// mass, because a border falls among them, min_p's too, or because the largest
// logit is one of them), the row is left to the general path (id kLeft).
//
// The counting itself keeps up with the memory (1,024 rows of 201,088: 80 us,
// 5.2 TB/s; without the LDS adds 77), so what follows it is kept short: a
// thread takes 8 adjacent values of one octave, equally spaced, whose e are a
// geometric series (two exponentials for eight), and one wave alone looks into
// the thread that a border falls to.
constexpr int32_t kLeft = -2;
struct Counted {
  static constexpr int kLo = (127 - 24) << 7, kHi = (127 + 8) << 7;  // magnitude bits
  static constexpr int kW = kHi - kLo;
  static constexpr int kPer = 8;  // values of a thread: the positive ones from the largest down, then the negative ones
  static_assert(2 * kW == kPer * kThreads && 128 % kPer == 0, "a thread's values lie in one octave");
  // counts of one sign: 0 = below 2^-24, 1 + (bits - kLo), kW + 1 = from 2^8 on
  // (also infinities and NaN); the negative ones follow the positive ones
  static constexpr int kSign = kW + 4;
  static constexpr int kCounts = 2 * kSign;
  static constexpr int kZeroThread = kThreads / 2 - 1;  // 0 comes after this thread's values, as place kPer
  static_assert(kCounts * 4 < 65536, "byte offsets fit 16 bits");
  // place i of thread t
  __device__ static inline float value(int t, int i) {
    if (i >= kPer) return 0.f;
    const int s = t * kPer + i;
    const uint32_t b = s < kW ? (uint32_t)(kHi - 1 - s) : 0x8000u | (uint32_t)(s - kW + kLo);
    return __builtin_bit_cast(float, b << 16);
  }
  __device__ static inline uint32_t word(const uint32_t* cnt, int t, int i) {
    const int s = t * kPer + i;
    return i < kPer ? s < kW ? cnt[kW - s] : cnt[kSign + 1 + s - kW] : cnt[0];
  }
};
struct CountShared {
  Settings how;
  u32x4_t words[(Counted::kCounts + 7) / 4];
  Red red;
  uint32_t first;    // the first place with a count
  uint32_t last;     // the last thread with mass
  uint32_t pick[3];  // the thread a border falls to
  double got[3];     // the mass up to and with the border's token, its own mass,
  double got_e[3];
  uint32_t got_at[3], got_r[3], got_n[3];  // its place, which of the equal ones it is, and how many there are
  uint32_t got_parts[3];
  // the counts, so that a thread's values are whole 16-byte words
  __device__ inline uint32_t* cnt() { return (uint32_t*)words + 3; }
};
static_assert(kNthRoom <= Counted::kCounts, "the search takes the counts' place");

// Rows of fewer than 2^18 logits: a count takes the low 18 bits of its word, and
// above them two fields of 7 bits count its logits in the row's first and in
// its second third, which later tells the third that holds the n-th of fewer
// than 128 equal logits (with more of them the fields overflow, harmlessly).
constexpr int kPartShift = 18, kPartBits = 7;
struct Thirds {
  bool on;
  uint32_t b1, b2;  // the second and the last third's first chunks
  __device__ inline Thirds(const Row<__bf16>& row, bool use) {
    b1 = row.nb / 3 / kThreads * kThreads;  // a round of chunks lies in one third
    b2 = 2 * b1;
    on = use && b1 > 0;
  }
  __device__ inline uint32_t mask() const { return on ? (1u << kPartShift) - 1 : 0xFFFFFFFFu; }
  __device__ inline uint32_t step(uint32_t c) const {
    const uint32_t s = c < b1 ? 1u + (1u << kPartShift) : c < b2 ? 1u + (1u << (kPartShift + kPartBits)) : 1u;
    return on ? s : 1u;
  }
};

// Two logits (the halves of w) counted.
__device__ inline void count_pair(uint32_t w, char* cnt, uint32_t step) {
  typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  const i16x2 lo = {(int16_t)(Counted::kLo - 1), (int16_t)(Counted::kLo - 1)}, zero = {0, 0};
  const i16x2 top = {(int16_t)(Counted::kW + 1), (int16_t)(Counted::kW + 1)};
  const i16x2 sign = {(int16_t)Counted::kSign, (int16_t)Counted::kSign}, fifteen = {15, 15};
  i16x2 at = __builtin_bit_cast(i16x2, w & 0x7FFF7FFFu) - lo;
  at = __builtin_elementwise_max(__builtin_elementwise_min(at, top), zero);
  at += (__builtin_bit_cast(i16x2, w) >> fifteen) & sign;
  const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_bit_cast(u16x2, at) << (u16x2){2, 2});
  atomicAdd((uint32_t*)(cnt + (b & 0xFFFFu)), step);
  atomicAdd((uint32_t*)(cnt + (b >> 16)), step);
}
__device__ inline void count_one(uint32_t h, uint32_t* cnt, uint32_t step) {
  int at = (int)(h & 0x7FFFu) - (Counted::kLo - 1);
  at = at < 0 ? 0 : at > Counted::kW + 1 ? Counted::kW + 1 : at;
  atomicAdd(&cnt[at + (h & 0x8000u ? Counted::kSign : 0)], step);
}

__device__ inline void count_row(const Row<__bf16>& row, uint32_t* cnt, const Thirds& parts) {
  for_each_chunk<8>(
      row,
      [&](const u32x4_t& v, uint32_t c) {
        const uint32_t step = parts.step(c);
#pragma unroll
        for (int i = 0; i < 4; ++i) count_pair(v[i], (char*)cnt, step);
      },
      [&](__bf16 x, int64_t id) {
        count_one(__builtin_bit_cast(uint16_t, x), cnt, parts.step(id < row.head ? 0 : row.nb));
      });
}

// Whether the row holds a nonzero logit that is counted as 0.
__device__ inline bool has_tiny(const Row<__bf16>& row) {
  const float least = __builtin_bit_cast(float, (uint32_t)Counted::kLo << 16);  // 2^-24
  bool tiny = false;
  for_each(row, [&](float l, int64_t) { tiny |= l != 0.f && fabsf(l) < least; });
  return __syncthreads_or(tiny);
}

// A drawn token: the r-th (r >= 1) of the row's n logits of this value, its
// mass e and the mass S it was drawn from.
struct Drawn {
  float logit;
  uint32_t r, n, parts;  // parts: the fields of n's thirds
  double e, S;
};

// The draw from the counts in sh.  False: the row is one for the general path.
__device__ __forceinline__ bool pick_counted(const Row<__bf16>& row, CountShared& sh, uint32_t mask, Drawn* out) {
  const int tid = threadIdx.x, lane = tid & 63;
  constexpr int kPer = Counted::kPer, kPlaces = kPer + 1;
  const uint32_t* cnt = sh.cnt();
  if (tid == 0) {
    sh.first = 0xFFFFFFFFu;
    sh.last = 0;
    for (int i = 0; i < 3; ++i) sh.pick[i] = 0xFFFFFFFFu;
  }
  if ((cnt[Counted::kW + 1] & mask) != 0) return false;  // 256 and more, +inf or NaN
  const bool low = (cnt[Counted::kSign + Counted::kW + 1] & mask) != 0;  // -256 and less, -inf or NaN
  const uint32_t zeros = uniform((cnt[0] & mask) + (cnt[Counted::kSign] & mask));
  uint32_t n[kPer], mine = tid == Counted::kZeroThread ? zeros : 0;
  {
    const int s = tid * kPer;
    const bool neg = s >= Counted::kW;
    const int at = neg ? Counted::kSign + 1 + s - Counted::kW : Counted::kW - s - kPer + 1;
    const u32x4_t a = ((const u32x4_t*)(cnt + at))[0], b = ((const u32x4_t*)(cnt + at))[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      n[i] = (neg ? a[i] : b[3 - i]) & mask;
      n[4 + i] = (neg ? b[i] : a[3 - i]) & mask;
    }
  }
  int first = kPer;
#pragma unroll
  for (int i = kPer - 1; i >= 0; --i) {
    mine += n[i];
    if (n[i]) first = i;
  }
  __syncthreads();
  const uint64_t any = __ballot(mine != 0);
  min_of_hits(mine != 0, (uint32_t)(tid * kPlaces + first), &sh.first);
  __syncthreads();
  const uint32_t top = uniform(sh.first);
  if (top == 0xFFFFFFFFu) return false;
  Scale sc;
  sc.set(Counted::value((int)(top / kPlaces), (int)(top % kPlaces)), uniform(sh.how.c), 0);
  if (low && sc.y(-256.f) < (double)kBins) return false;
  const double e0 = uniform(mass_of(sh.red, sc.y(0.f)));  // of 0, where the row has it
  const double min_p = uniform(sh.how.min_p);
  // Nonzero logits below 2^-24 are taken as 0, and weigh between the e of -2^-24
  // and of 2^-24 (which may be far apart: T may be smaller still).  They show by
  // that much mass, where min_p's border lies between the two, and where 0 is the
  // largest logit, as every e is relative to that.
  bool tiny_counts = zeros && top % kPlaces == kPer;
  double spread = 0.0;
  if (zeros && !tiny_counts) {
    const double w = 0x1p-24 * sc.c, y0 = sc.y(0.f);
    const double hi = uniform(mass_of(sh.red, fmax(y0 - w, 0.0))), lo = uniform(mass_of(sh.red, y0 + w));
    spread = uniform((double)zeros * (hi - lo));
    tiny_counts = lo < min_p && min_p <= hi;
  }
  double sum = 0.0, likely = 0.0, before = 0.0, dummy;
  uint32_t cbefore = 0;
  if (any) {  // else every place of the wave is empty
    // from the thread's first value that occurs (those above it may lie above
    // the largest logit, where e would overflow), each e is q of the one before
    const float v = Counted::value(tid, first);
    const uint32_t octave = __builtin_bit_cast(uint32_t, v) & 0x7F800000u;
    const float step = __builtin_bit_cast(float, octave - (7u << 23));
    double y = sc.y(v);
    const double dy = first < kPer ? (double)step * sc.c : 0.0, q = mass_of(sh.red, dy);
    double e = mine ? mass_of(sh.red, y) : 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const double m = (double)n[i] * e;
      sum += m;
      if (e >= min_p) likely += m;
      if (i >= first) {
        y += dy;
        e = y < (double)kBins ? e * q : 0.0;
      }
    }
    if (tid == Counted::kZeroThread && zeros) {
      sum += (double)zeros * e0;
      if (e0 >= min_p) likely += (double)zeros * e0;
    }
  }
  double S = uniform(block_prefix(sum, sh.red, &before));
  const bool limit = sh.how.limit;
  if (limit) block_prefix(mine, sh.red, &cbefore);
  const double s_min = min_p > 0.0 ? uniform(block_prefix(likely, sh.red, &dummy)) : S;
  tiny_counts |= spread > 1e-13 * S;

  // Borders: k, then p, then the draw.  Each falls to the first thread at the
  // end of whose values it is reached (the last with mass if rounding leaves
  // none); that thread's wave takes its places one per lane.
  max_of_hits(sum > 0.0, (uint32_t)tid, &sh.last);
  const double p = uniform(sh.how.p), u = uniform(sh.how.u);
  const uint32_t k = uniform(sh.how.k);
#pragma unroll 1
  for (int kind = limit ? BY_COUNT : p < 1.0 ? BY_MASS : BY_MASS_OVER;;) {
    if (kind == BY_MASS_OVER) S = fmin(S, s_min);
    const double target = kind == BY_MASS ? p * S : u * S;
    min_of_hits(sum > 0.0 && reached(kind, cbefore + mine, before + sum, k, target), (uint32_t)tid, &sh.pick[kind]);
    __syncthreads();
    const uint32_t hit = sh.pick[kind], at = uniform(hit != 0xFFFFFFFFu ? hit : sh.last);
    if (at >> 6 == (uint32_t)tid >> 6) {
      const double above0 = of_lane(before, (int)(at & 63));
      const uint32_t above_n0 = of_lane(cbefore, (int)(at & 63));
      const bool zero = lane == kPer && at == Counted::kZeroThread;
      uint32_t word = lane < kPer || zero ? Counted::word(cnt, (int)at, lane) : 0, ns = word & mask;
      word >>= kPartShift;
      if (zero) {
        ns = zeros;
        word += cnt[Counted::kSign] >> kPartShift;
      }
      const double e = ns ? mass_of(sh.red, sc.y(Counted::value((int)at, lane))) : 0.0;
      static_assert(kPlaces <= 16, "the places of a thread lie in one row of lanes");
      const double run = above0 + wave_scan((double)ns * e);
      const uint32_t crun = above_n0 + wave_scan(ns);
      const uint64_t there = __ballot(ns && e > 0.0 && reached(kind, crun, run, k, target));
      const uint64_t some = __ballot(ns && e > 0.0);
      const int l = there ? __builtin_ctzll(there) : 63 - __builtin_clzll(some | 1ull);
      const uint32_t nl = of_lane(ns, l), before_n = of_lane(crun, l) - nl;
      const double el = of_lane(e, l), above = l > 0 ? of_lane(run, l - 1) : above0;
      const uint32_t r = nl ? equal_taken(kind, nl, before_n, above, el, k, target) : 0;
      if (lane == 0) {
        sh.got[kind] = above + (double)r * el;
        sh.got_e[kind] = el;
        sh.got_at[kind] = at * kPlaces + (uint32_t)l;
        sh.got_r[kind] = r;
        sh.got_n[kind] = nl;
      }
      if (lane == l) sh.got_parts[kind] = word;
    }
    __syncthreads();
    tiny_counts |= sh.got_at[kind] % kPlaces == kPer;
    if (sh.got_r[kind] == 0) return false;  // nothing with mass there
    if (kind == BY_MASS_OVER) break;
    S = fmin(S, uniform(sh.got[kind]));
    kind = kind == BY_COUNT && p < 1.0 ? BY_MASS : BY_MASS_OVER;
  }
  if (tiny_counts && has_tiny(row)) return false;
  const uint32_t at = uniform(sh.got_at[BY_MASS_OVER]);
  out->logit = Counted::value((int)(at / kPlaces), (int)(at % kPlaces));
  out->r = uniform(sh.got_r[BY_MASS_OVER]);
  out->n = uniform(sh.got_n[BY_MASS_OVER]);
  out->parts = uniform(sh.got_parts[BY_MASS_OVER]);
  out->e = uniform(sh.got_e[BY_MASS_OVER]);
  out->S = S;
  return true;
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
  // direct: no counting kernel runs first
  // split rows (slices > 1): logits per slice, and the slices' counts
  bool direct;
  int slices;
  int64_t slice_len;
  uint16_t* tables;
};
constexpr int kSlicesMax = 16;

// The row's settings; a temperature that is not above zero is greedy.
__device__ inline Settings row_settings(const SampleArgs& a, int64_t r) {
  Settings s;
  double T = a.p.temperatures ? (double)a.p.temperatures[r] : a.p.temperature;
  int64_t k = a.p.top_ks ? (int64_t)a.p.top_ks[r] : a.p.top_k;
  s.p = a.p.top_ps ? (double)a.p.top_ps[r] : a.p.top_p;
  s.min_p = a.p.min_ps ? (double)a.p.min_ps[r] : a.p.min_p;
  if (!(T > 0.0)) {
    T = 1.0;
    k = 1;
  }
  T = fmax(T, 1e-200);  // keeps 1 / T finite; only equal logits share the mass long before
  s.c = 92.332482616893656877 / T;
  s.limit = k > 0 && k < a.V;
  s.k = (uint32_t)(s.limit ? k : a.V);
  if (!(s.min_p > 0.0)) s.min_p = 0.0;
  if (s.min_p > 1.0) s.min_p = 1.0;
  s.u = (double)a.u[r];
  if (!(s.u > 0.0)) s.u = 0.0;
  const double u_max = 1.0 - 0x1p-24;  // the largest fp32 below 1
  if (s.u > u_max) s.u = u_max;
  return s;
}

__device__ inline void clear_counts(CountShared& sh) {
  for (int i = threadIdx.x; i < (int)(sizeof(sh.words) / 16); i += kThreads) sh.words[i] = u32x4_t{0, 0, 0, 0};
}
// The row's answer: token id, of mass e among S.
__device__ inline void put(const SampleArgs& a, int64_t r, int64_t id, double e, double S) {
  if (threadIdx.x == 0) {
    a.ids[r] = (int32_t)id;
    if (a.logp) a.logp[r] = (float)log(e / S);
  }
}

__global__ void __launch_bounds__(kThreads, 8) count_kernel(SampleArgs a) {
  __shared__ CountShared sh;
  const int64_t r = blockIdx.x;
  const Row<__bf16> row((const __bf16*)a.x + r * a.ld, a.V);
  if (threadIdx.x == 0) sh.how = row_settings(a, r);
  clear_counts(sh);
  fill_pow64(sh.red);
  __syncthreads();
  const Thirds parts(row, a.V < (1 << kPartShift));
  count_row(row, sh.cnt(), parts);
  __syncthreads();
  Drawn t{};
  int64_t id = kLeft;
  if (pick_counted(row, sh, parts.mask(), &t)) {
    int64_t b = 0, e = a.V;
    if (parts.on && t.n < 1u << kPartBits) {
      const uint32_t n1 = t.parts & ((1u << kPartBits) - 1), n2 = t.parts >> kPartBits;
      if (t.r <= n1) {
        t.n = n1;
        e = row.body_id(parts.b1);
      } else if (t.r - n1 <= n2) {
        t.r -= n1;
        t.n = n2;
        b = row.body_id(parts.b1);
        e = row.body_id(parts.b2);
      } else {
        t.r -= n1 + n2;
        t.n -= n1 + n2;
        b = row.body_id(parts.b2);
      }
    }
    id = b + nth_equal(Row<__bf16>(row.x + b, e - b), sh.cnt(), t.logit, t.r, t.n);
  }
  put(a, r, id, t.e, t.S);
}

// Few long rows: `slices` workgroups count a row's slices, so that more of the
// chip reads it, and the finishing workgroup adds their counts (16 bits each)
// and looks for the token in its slice alone.
constexpr int64_t kSliceMax = 65535;  // logits: a count fits 16 bits
constexpr int kTable = (Counted::kCounts + 7) / 8 * 8;  // counts of a slice in the workspace
__device__ inline Row<__bf16> slice_of(const SampleArgs& a, int64_t r, int s) {
  const int64_t b = (int64_t)s * a.slice_len, left = a.V - b;
  return Row<__bf16>((const __bf16*)a.x + r * a.ld + b, left < a.slice_len ? left : a.slice_len);
}
__global__ void __launch_bounds__(kThreads, 8) count_slice_kernel(SampleArgs a) {
  __shared__ CountShared sh;
  const int64_t r = blockIdx.x / a.slices;
  const int s = (int)(blockIdx.x - r * a.slices);
  clear_counts(sh);
  __syncthreads();
  const Row<__bf16> row = slice_of(a, r, s);
  count_row(row, sh.cnt(), Thirds(row, false));
  __syncthreads();
  uint32_t* dst = (uint32_t*)(a.tables + (int64_t)blockIdx.x * kTable);
  for (int i = threadIdx.x; i < Counted::kCounts / 2; i += kThreads)
    dst[i] = sh.cnt()[2 * i] | sh.cnt()[2 * i + 1] << 16;
}
static_assert(Counted::kCounts % 2 == 0, "counts are stored in pairs");

__global__ void __launch_bounds__(kThreads, 8) count_finish_kernel(SampleArgs a) {
  __shared__ CountShared sh;
  __shared__ uint32_t there[kSlicesMax];
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x;
  if (tid == 0) sh.how = row_settings(a, r);
  const uint16_t* tables = a.tables + r * a.slices * kTable;
  fill_pow64(sh.red);
  for (int i = tid; i < Counted::kCounts / 2; i += kThreads) {
    uint32_t lo = 0, hi = 0;
#pragma unroll 4
    for (int s = 0; s < a.slices; ++s) {
      const uint32_t w = ((const uint32_t*)(tables + s * kTable))[i];
      lo += w & 0xFFFFu;
      hi += w >> 16;
    }
    sh.cnt()[2 * i] = lo;
    sh.cnt()[2 * i + 1] = hi;
  }
  __syncthreads();
  Drawn d{};
  int64_t id = kLeft;
  const Row<__bf16> row((const __bf16*)a.x + r * a.ld, a.V);
  if (pick_counted(row, sh, 0xFFFFFFFFu, &d)) {
    // the slice that holds the r-th such logit
    if (tid < a.slices) {
      const uint16_t* t = tables + tid * kTable;
      const uint32_t h = __builtin_bit_cast(uint32_t, d.logit) >> 16;
      const int at = (int)(h & 0x7FFFu) - (Counted::kLo - 1);
      there[tid] = d.logit == 0.f ? (uint32_t)t[0] + t[Counted::kSign] : t[at + (h & 0x8000u ? Counted::kSign : 0)];
    }
    __syncthreads();
    int s = 0;
    while (s + 1 < a.slices && d.r > there[s]) d.r -= there[s++];
    id = s * a.slice_len + nth_equal(slice_of(a, r, s), sh.cnt(), d.logit, d.r, there[s]);
  }
  put(a, r, id, d.e, d.S);
}

// The row's answer from its first n (at most kFastK) tokens, sorted in sh.cand,
// by one wave: each lane takes n / 64 adjacent ones.
template <typename T>
__device__ __forceinline__ void draw_from_list(const SampleArgs& a, int64_t r, const Shared& sh, int n, const Scale& sc,
                                               const Settings& how) {
  constexpr int kEach = kFastK / 64;
  const int lane = threadIdx.x & 63, each = (n + 63) / 64, b = lane * each;
  double e[kEach], mine = 0.0, likely = 0.0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    e[i] = i < each && b + i < n ? mass_of(sh.red, sc.y(Key<T>::value((uint32_t)(sh.cand[b + i] >> 32)))) : 0.0;
    mine += e[i];
    if (e[i] >= how.min_p) likely += e[i];
  }
  const double upto = wave_scan(mine), up = __shfl_up(upto, 1), before = lane ? up : 0.0;
  double S = of_lane(upto, 63);
  // the first token at which the border is reached, the last if rounding leaves
  // none, and the mass up to it
  int at = 0;
  auto border = [&](int kind, double target) {
    int mine_at = -1;
    double run = before, got = 0.0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      run += e[i];
      const bool last = b + i == n - 1;
      if (i < each && mine_at < 0 && b + i < n && (last || reached(kind, 0, run, 0, target))) {
        mine_at = b + i;
        got = run;
      }
    }
    const int l = __builtin_ctzll(__ballot(mine_at >= 0));
    at = (int)of_lane((uint32_t)mine_at, l);
    return of_lane(got, l);
  };
  // p is a share of the first k's mass; min_p keeps at least the first token
  const double s_min = how.min_p > 0.0 ? of_lane(wave_scan(likely), 63) : S;
  if (how.p < 1.0) S = border(BY_MASS, how.p * S);
  S = fmin(S, s_min);
  border(BY_MASS_OVER, how.u * S);
  const uint64_t c = sh.cand[at];
  if (lane == 0) {
    a.ids[r] = (int32_t)unpack_id(c);
    if (a.logp) a.logp[r] = (float)log(mass_of(sh.red, sc.y(Key<T>::value((uint32_t)(c >> 32)))) / S);
  }
}

// The general path: every row (direct), or those that the counting kernels left.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) sample_kernel(SampleArgs a) {
  __shared__ Shared sh;
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x;
  if (!a.direct && a.ids[r] != kLeft) return;
  const Row<T> row((const T*)a.x + r * a.ld, a.V);

  if (tid == 0) sh.how = row_settings(a, r);
  fill_pow64(sh.red);  // read after the next barrier

  // 1. the largest logit, and each thread's
  float mv = -INFINITY;
  for_each_chunk<8>(
      row, [&](const u32x4_t& v, uint32_t) { mv = larger(mv, Row<T>::largest(v)); },
      [&](T l, int64_t) { mv = larger(mv, (float)l); });
  if (mv != mv) {  // the thread met NaN: its largest by comparisons
    mv = -INFINITY;
    for_each(row, [&](float l, int64_t) { mv = l > mv ? l : mv; });
  }
  const float mx = uniform(block_max(mv, sh.red));
  if (mx == -INFINITY) {  // nothing to sample
    if (tid == 0) {
      a.ids[r] = -1;
      if (a.logp) a.logp[r] = -INFINITY;
    }
    return;
  }
  const Settings& how = sh.how;
  const uint32_t k = uniform(how.k);
  Scale sc;
  sc.set(mx, uniform(how.c), a.fix_bits);

  // 2a. few tokens: those that reach the k-th largest of the threads' maxima
  if (a.direct && k <= (uint32_t)kFastK) {
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
    block_prefix(mine, sh.red, &above);
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
    const uint32_t t0 = uniform(sh.pick);
    const float v0 = t0 <= Key<T>::of(-INFINITY) ? -INFINITY : Key<T>::value(t0);
    auto hold = [&](float l, int64_t id) {
      if (l >= v0 && l > -INFINITY) {
        const uint32_t slot = atomicAdd(&sh.n_cand, 1u);
        if (slot < (uint32_t)kCap) sh.cand[slot] = pack(Key<T>::of(l), (uint32_t)id);
      }
    };
    if (mv >= v0)  // among the logits of this thread
      for_each_chunk<kFlight>(
          row,
          [&](const u32x4_t& v, uint32_t c) {
            if (!(Row<T>::largest(v) < v0)) {  // also beside NaN
              float f[Row<T>::kN];
              Row<T>::unpack(v, f);
#pragma unroll
              for (int i = 0; i < Row<T>::kN; ++i) hold(f[i], row.body_id(c) + i);
            }
          },
          [&](T l, int64_t id) { hold((float)l, id); });
    __syncthreads();
    const uint32_t held = uniform(sh.n_cand);
    if (held <= (uint32_t)kCap) {
      sort_cand(sh, (int)held);
      if (tid < 64) draw_from_list<T>(a, r, sh, (int)(held < k ? held : k), sc, how);
      return;
    }
    __syncthreads();
  }

  // 2b. the row's mass over bins
  for (int i = tid; i < kBins; i += kThreads) {
    sh.mass[i] = 0;
    sh.count[i] = 0;
  }
  if (tid < 3) sh.edge_mass[tid] = 0;
  __syncthreads();
  // min_p's border: y <= y_min; the share of its bin and of the two beside it
  // (a bin is only within 1e-3 of y) is summed on the side
  const double p = uniform(how.p), min_p = uniform(how.min_p), u = uniform(how.u);
  const bool limit = uniform((uint32_t)how.limit) != 0;
  const double y_min = min_p > 0.0 ? -64.0 * log2(min_p) : (double)INFINITY;
  const int bin_min = y_min < (double)kBins ? (int)y_min : 2 * kBins;
  sc.either([&](auto plain) {
    for_each(row, [&](float l, int64_t) {
      const float place = sc.template place<plain.value>(l);
      if (place < (float)kBins) {
        const int bin = (int)place;
        // round to an integer by adding 2^52: the low bits of the sum are it
        const double q = __builtin_fma(pow_frac(sc.template frac<plain.value>(l, bin)), sc.fix, 0x1p52);
        const unsigned long long qi = (unsigned long long)__builtin_bit_cast(uint64_t, q) & 0xFFFFFFFFFFFFFull;
        atomicAdd((unsigned long long*)&sh.mass[bin], qi);
        if (limit) atomicAdd(&sh.count[bin], 1u);
        const uint32_t near = (uint32_t)(bin - bin_min + 1);
        if (near < 3u && sc.y(l) <= y_min) atomicAdd((unsigned long long*)&sh.edge_mass[near], qi);
      }
    });
  });
  __syncthreads();
  // masses of the bins, of the whole row and of the tokens that reach min_p
  double S = 0.0, s_min = 0.0, before = 0.0;
  uint32_t cbefore = 0;
  {
    double all = 0.0, likely = 0.0, dummy;
    uint32_t tokens = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int b = tid * kPerThread + i;
      const double unit = sc.inv_fix * bin_top(sh.red, b);
      const double m = (double)sh.mass[b] * unit;
      ((double*)sh.mass)[b] = m;
      all += m;
      tokens += sh.count[b];
      const uint32_t near = (uint32_t)(b - bin_min + 1);
      if (near < 3u)
        likely += (double)sh.edge_mass[near] * unit;
      else if (b < bin_min)
        likely += m;
    }
    S = uniform(block_prefix(all, sh.red, &before));
    if (limit) block_prefix(tokens, sh.red, &cbefore);
    s_min = min_p > 0.0 ? uniform(block_prefix(likely, sh.red, &dummy)) : S;
  }
  Found f;
#pragma unroll 1
  for (int kind = limit ? BY_COUNT : p < 1.0 ? BY_MASS : BY_MASS_OVER;;) {
    if (kind == BY_MASS_OVER) S = fmin(S, s_min);
    f = find_border(row, sh, sc, kind, k, kind == BY_MASS ? p * S : u * S, before, cbefore,
                    kind == BY_MASS_OVER);
    if (kind == BY_MASS_OVER) break;
    S = fmin(S, uniform(f.mass));
    kind = kind == BY_COUNT && p < 1.0 ? BY_MASS : BY_MASS_OVER;
  }
  if (tid == 0) {
    a.ids[r] = (int32_t)f.id;
    if (a.logp) a.logp[r] = (float)log(mass_of(sh.red, sc.y(f.logit)) / S);
  }
}

}  // namespace

namespace {
// Whether bf16 rows go to the general path at once: where each takes at most
// 128 tokens, its collected path needs less than counting's scan of 8,192
// counts, as long as no compute unit has a second row.  In us, that path and
// counting:
//   top_k     1 x 201,088   64 x 32,000   256 x 201,088   512 x 201,088
//     1          13   22        8   15         28   34         53   57
//   100          21   22       13   15         36   34         71   57
//   250          26   22       18   15         46   34         89   57
// A limit of each row's own cannot be read here.
constexpr int64_t kDirectK = 128, kDirectRows = 256;
bool direct_bf16(int64_t N, const SampleParams& p) {
  const bool few = !p.top_ks && !p.temperatures && ((p.top_k > 0 && p.top_k <= kDirectK) || p.temperature == 0.0);
  return few && N <= kDirectRows;
}

// Workgroups per bf16 row: more than one for few rows (at most a quarter of
// the 256 compute units busy) of at least 2 x 16,384 logits.  With top-p, one row
// of 201,088 logits takes 21 us so, 25 us by one workgroup; 64 rows 24 and 28.
int slices_of(Dtype dt, int64_t N, int64_t V) {
  if (dt != DT_BF16 || N > 64) return 1;
  int64_t s = V / 16384;
  if (s > 256 / N) s = 256 / N;
  if (s > kSlicesMax) s = kSlicesMax;
  return s < 2 || (V + s - 1) / s > kSliceMax - 64 ? 1 : (int)s;
}
}  // namespace
uint64_t sample_workspace(Dtype dt, int64_t N, int64_t V) {
  const int s = slices_of(dt, N, V);
  return s > 1 ? (uint64_t)N * s * kTable * sizeof(uint16_t) : 0;
}

hipError_t launch_sample(Dtype dt, const void* x, int64_t N, int64_t V, int64_t ld, const float* u,
                         const SampleParams& p, int32_t* ids, float* logp, void* ws, hipStream_t s) {
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
  a.direct = dt != DT_BF16 || direct_bf16(N, p);
  if (!a.direct) {
    a.slices = ws != nullptr ? slices_of(dt, N, V) : 1;
    hipError_t e;
    if (a.slices > 1) {
      a.slice_len = ((V + a.slices - 1) / a.slices + 63) / 64 * 64;
      a.slices = (int)((V + a.slice_len - 1) / a.slice_len);
      a.tables = (uint16_t*)ws;
      hipLaunchKernelGGL(count_slice_kernel, dim3((unsigned)(N * a.slices)), dim3(kThreads), 0, s, a);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      hipLaunchKernelGGL(count_finish_kernel, dim3((unsigned)N), dim3(kThreads), 0, s, a);
    } else {
      hipLaunchKernelGGL(count_kernel, dim3((unsigned)N), dim3(kThreads), 0, s, a);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (dt == DT_BF16)
    hipLaunchKernelGGL(sample_kernel<__bf16>, dim3((unsigned)N), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL(sample_kernel<float>, dim3((unsigned)N), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace ckl
