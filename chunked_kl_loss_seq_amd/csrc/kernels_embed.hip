// Token embedding: rows of the vocabulary table by id, scaled, and the
// gradient with respect to the table (the other end of the W [V, d] whose
// head gradient the loss computes; with tied weights both go to one dW).
//
//   out[n]  = scale W[ids[n]]                      (rounded once to W's type)
//   dW[v] (+)= scale sum_{n : ids[n] = v} dY[n]    (fp32, fixed order)
//
// An id outside [0, V) is a position without a token: its row of out is
// zeros, it adds nothing to dW, and nothing is read at it.
//
// The gradient sorts the positions by (id, position) and sums runs of equal
// ids, so no atomics touch the sums and the result depends on the inputs
// alone.  Text is skewed (one token can be a tenth of a batch) while most of
// a large vocabulary is absent, so neither a workgroup per token nor per
// position balances: the sorted list is cut into tiles of equal length
// whatever their tokens, a run inside one tile is written at once, and a run
// that crosses tiles leaves one partial row per tile, summed in tile order by
// a second kernel.  Rows without a token are written as zeros by other
// workgroups of the same launches, so every byte of dW is written once; those
// zeros bound the call for large vocabularies.
//
// Measured (MI355X, bf16):
//  lookup of 32,768 x 2,880: 52 us, 7.3 TB/s of rows read and written (repeated
//    rows come from the caches); of one row: 2 us on the device.
//  gradient of 32,768 x 2,880 of 201,088: 503-515 us, 4.9 TB/s (dY read, dW
//    written); the zeros alone, as a plain fill of dW, take 433 us (5.35 TB/s; a
//    fill of 1 GiB reaches 6.9).
//  gradient of 4,096 x 2,048 of 32,000: 54 us, 5.2 TB/s, of which rank 6, sum 31
//    with most of the zeros, join 15 with the rest.
#include <hip/hip_runtime.h>

#include "launch.hpp"

namespace ckl {

namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

// 16-byte chunk <-> fp32 values
template <typename T>
struct Chunk;
template <>
struct Chunk<__bf16> {
  static constexpr int kN = 8;
  __device__ static inline void unpack(const u32x4_t& v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = v[i];
      f[2 * i] = __builtin_bit_cast(float, w << 16);
      f[2 * i + 1] = __builtin_bit_cast(float, w & 0xFFFF0000u);
    }
  }
  __device__ static inline u32x4_t pack(const float* f) {
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint16_t lo = __builtin_bit_cast(uint16_t, (__bf16)f[2 * i]);
      const uint16_t hi = __builtin_bit_cast(uint16_t, (__bf16)f[2 * i + 1]);
      v[i] = (uint32_t)lo | ((uint32_t)hi << 16);
    }
    return v;
  }
};
template <>
struct Chunk<float> {
  static constexpr int kN = 4;
  __device__ static inline void unpack(const u32x4_t& v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = v[i];
      f[i] = __builtin_bit_cast(float, w);
    }
  }
  __device__ static inline u32x4_t pack(const float* f) {
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __builtin_bit_cast(uint32_t, f[i]);
    return v;
  }
};

// ---------------------------------------------------------------- lookup
// 2^lg lanes per row (at most a wave), each lane's chunks of the row loaded
// four at a time.  Bound by the rows written and, where tokens repeat little,
// the rows read.
template <typename T>
__global__ void __launch_bounds__(kThreads) embed_kernel(const int32_t* __restrict__ ids, const T* __restrict__ W,
                                                         float scale, int64_t N, int64_t V, int cpr, int lg,
                                                         T* __restrict__ out) {
  const int64_t n = (int64_t)blockIdx.x * (kThreads >> lg) + (threadIdx.x >> lg);
  if (n >= N) return;
  const int l = threadIdx.x & ((1 << lg) - 1), step = 1 << lg;
  const int64_t id = ids[n];
  u32x4_t* dst = (u32x4_t*)out + n * cpr;
  if (id < 0 || id >= V) {
    for (int c = l; c < cpr; c += step) dst[c] = u32x4_t{0, 0, 0, 0};
    return;
  }
  const u32x4_t* src = (const u32x4_t*)W + id * cpr;
  for (int c0 = l; c0 < cpr; c0 += 4 * step) {
    u32x4_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c0 + j * step < cpr) v[j] = src[c0 + j * step];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (c0 + j * step >= cpr) break;
      float f[Chunk<T>::kN];
      Chunk<T>::unpack(v[j], f);
#pragma unroll
      for (int i = 0; i < Chunk<T>::kN; ++i) f[i] *= scale;
      dst[c0 + j * step] = Chunk<T>::pack(f);
    }
  }
}

// ---------------------------------------------------------------- sort by (id, position)
// Key of a position: its id, or V (after every token) where it has none.
__device__ inline uint32_t key_of(const int32_t* ids, int64_t i, uint32_t V) {
  const uint32_t id = (uint32_t)ids[i];
  return id < V ? id : V;
}

// Sum of v over the threads before this one in a workgroup of kThreads.
__device__ inline uint32_t block_before(uint32_t v, uint32_t* wsum) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  if (lane == 63) wsum[w] = x;
  __syncthreads();
  uint32_t run = x - v;
  for (int i = 0; i < w; ++i) run += wsum[i];
  return run;
}

// Few positions: a position's place is the number of positions before it in
// (id, position) order, counted directly: one launch in place of the radix
// sort's four.  32 lanes share one position and the list passes through LDS
// (whole calls of 4,096 and 8,192 positions, d = 64, with 16, 32 and 64 lanes a
// position: 22, 20, 20 and 30, 29, 30 us; by the radix sort 8,192 x 2,048 takes 79
// us, so 72).
constexpr int kRankMax = 8192;
constexpr int kRankTile = 4096;
constexpr int kRankLanes = 32;
__global__ void __launch_bounds__(kThreads) rank_kernel(const int32_t* __restrict__ ids, int N, uint32_t V,
                                                        uint32_t* __restrict__ skey, uint32_t* __restrict__ spos) {
  __shared__ __attribute__((aligned(16))) uint32_t tile[kRankTile];
  const int i = blockIdx.x * (kThreads / kRankLanes) + threadIdx.x / kRankLanes, part = threadIdx.x % kRankLanes;
  const uint32_t key = i < N ? key_of(ids, i, V) : 0;
  int place = 0;
  for (int t0 = 0; t0 < N; t0 += kRankTile) {
    const int n = min(kRankTile, N - t0), n4 = (n + 3) & ~3;
    __syncthreads();
    uint32_t k[kRankTile / kThreads];  // loaded together: one after the other they took most of the launch
#pragma unroll
    for (int q = 0; q < kRankTile / kThreads; ++q) {
      const int j = q * kThreads + (int)threadIdx.x;
      k[q] = key_of(ids, t0 + (j < n ? j : n - 1), V);
    }
#pragma unroll
    for (int q = 0; q < kRankTile / kThreads; ++q) {
      const int j = q * kThreads + (int)threadIdx.x;
      tile[j] = j < n ? k[q] : 0xFFFFFFFFu;
    }
    __syncthreads();
#pragma unroll 8
    for (int j = 4 * part; j < n4; j += 4 * kRankLanes) {
      const u32x4_t k = *(const u32x4_t*)&tile[j];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t kq = k[q];
        place += kq < key + (t0 + j + q < i ? 1u : 0u) ? 1 : 0;  // an earlier equal key counts
      }
    }
  }
#pragma unroll
  for (int o = 1; o < kRankLanes; o <<= 1) place += __shfl_xor(place, o);
  if (i < N && part == 0) {
    skey[place] = key;
    spos[place] = (uint32_t)i;
  }
}

// Many positions: a stable radix sort of the keys, kDigit bits a pass (two
// passes up to 2^18 - 1 tokens).  Per pass: a histogram per tile, and a scatter
// in which each workgroup first adds up the tiles' histograms to its own
// places (an exclusive scan in (digit, tile) order) and each wave ranks its
// own stretch of the tile in order.  With more than kDirectTiles tiles those
// sums would outgrow the sort, and a scan kernel between the two makes them.
constexpr int kDigit = 9;
constexpr int kDigits = 1 << kDigit;
constexpr int kSortTile = 1024;
constexpr int kSortWaves = kThreads / 64;
constexpr int kRounds = kSortTile / kThreads;  // 64-element rounds per wave
constexpr int64_t kDirectTiles = 256;

// Element i of the pass: from the ids on the first pass (keys == null).
__device__ inline uint32_t pass_key(const int32_t* ids, const uint32_t* keys, int64_t i, uint32_t V) {
  return keys != nullptr ? keys[i] : key_of(ids, i, V);
}

// bits: null, or words to clear (a bit per token, set by the last scatter).
__global__ void __launch_bounds__(kThreads) sort_hist_kernel(const int32_t* __restrict__ ids,
                                                             const uint32_t* __restrict__ keys, int64_t N, uint32_t V,
                                                             int shift, int tiles, uint32_t* __restrict__ hist,
                                                             uint32_t* __restrict__ bits, int64_t words) {
  __shared__ uint32_t h[kDigits];
  for (int i = threadIdx.x; i < kDigits; i += kThreads) h[i] = 0;
  if (bits != nullptr)
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < words; i += (int64_t)tiles * kThreads)
      bits[i] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * kSortTile + threadIdx.x;
  uint32_t key[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = base + r * kThreads;
    key[r] = pass_key(ids, keys, i < N ? i : N - 1, V);
  }
#pragma unroll
  for (int r = 0; r < kRounds; ++r)
    if (base + r * kThreads < N) atomicAdd(&h[(key[r] >> shift) & (kDigits - 1)], 1u);
  __syncthreads();
  for (int i = threadIdx.x; i < kDigits; i += kThreads) hist[(int64_t)blockIdx.x * kDigits + i] = h[i];
}

// Exclusive scan of the histograms in (digit, tile) order in place, one
// workgroup: thread t takes two digits, all tiles.
static_assert(kDigits == 2 * kThreads, "two digits per thread");
__global__ void __launch_bounds__(kThreads) sort_scan_kernel(uint32_t* __restrict__ hist, int64_t tiles) {
  __shared__ uint32_t wsum[kThreads / 64];
  uint2* h = (uint2*)hist;
  uint32_t a = 0, b = 0;
#pragma unroll 8
  for (int64_t i = 0; i < tiles; ++i) {
    const uint2 c = h[i * kThreads + threadIdx.x];
    a += c.x;
    b += c.y;
  }
  uint32_t ra = block_before(a + b, wsum), rb = ra + a;
#pragma unroll 8
  for (int64_t i = 0; i < tiles; ++i) {
    const uint2 c = h[i * kThreads + threadIdx.x];
    h[i * kThreads + threadIdx.x] = make_uint2(ra, rb);
    ra += c.x;
    rb += c.y;
  }
}

// scanned: hist holds places (sort_scan_kernel) rather than counts.  bits: null,
// or (last pass) where the tokens that occur are marked.
__global__ void __launch_bounds__(kThreads) sort_scatter_kernel(const int32_t* __restrict__ ids,
                                                                const uint32_t* __restrict__ keys,
                                                                const uint32_t* __restrict__ pos, int64_t N,
                                                                uint32_t V, int shift, int tiles, bool scanned,
                                                                const uint32_t* __restrict__ hist,
                                                                uint32_t* __restrict__ keys_out,
                                                                uint32_t* __restrict__ pos_out,
                                                                uint32_t* __restrict__ bits) {
  __shared__ uint32_t cnt[kSortWaves][kDigits];
  __shared__ uint32_t wsum[kSortWaves];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < kSortWaves * kDigits; i += kThreads) (&cnt[0][0])[i] = 0;
  // wave w owns elements [64 kRounds w, 64 kRounds (w + 1)) of the tile, in order
  const int64_t base = (int64_t)blockIdx.x * kSortTile + (int64_t)w * 64 * kRounds;
  uint32_t key[kRounds], place[kRounds], rank[kRounds];
  bool marks[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = base + r * 64 + lane < N ? base + r * 64 + lane : N - 1;
    key[r] = pass_key(ids, keys, i, V);
    place[r] = pos != nullptr ? pos[i] : (uint32_t)i;
  }
  // the places of this tile's digits 2 t and 2 t + 1
  const uint2* h = (const uint2*)hist;
  uint32_t pa, pb;
  if (scanned) {
    const uint2 c = h[(int64_t)blockIdx.x * kThreads + threadIdx.x];
    pa = c.x;
    pb = c.y;
    __syncthreads();
  } else {
    uint32_t a = 0, b = 0, ea = 0, eb = 0;  // all tiles, earlier tiles
#pragma unroll 8
    for (int i = 0; i < tiles; ++i) {
      const uint2 c = h[i * kThreads + threadIdx.x];
      a += c.x;
      b += c.y;
      ea += i < (int)blockIdx.x ? c.x : 0;
      eb += i < (int)blockIdx.x ? c.y : 0;
    }
    const uint32_t run = block_before(a + b, wsum);  // has a barrier: the counters are clear
    pa = run + ea;
    pb = run + a + eb;
  }
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const bool in = base + r * 64 + lane < N;
    const uint32_t dg = (key[r] >> shift) & (kDigits - 1);
    uint64_t same = __ballot(in);
#pragma unroll
    for (int b = 0; b < kDigit; ++b) {
      const uint64_t m = __ballot((dg >> b) & 1u);
      same &= ((dg >> b) & 1u) ? m : ~m;
    }
    // the lanes of `same` hold this digit; earlier ones come first
    const uint32_t before =
        __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
    const uint32_t old = in ? cnt[w][dg] : 0;
    rank[r] = old + before;
    // The lower digits are in order, so lanes of one key are neighbours among
    // the lanes of `same`: the first of them marks the token.  (With a mark by
    // every position, a launch for 10,595 positions of 1,497 tokens took 36 us, not 13.)
    const uint64_t lower = same & ((1ull << lane) - 1);
    marks[r] = in;
    if (bits != nullptr) {
      const uint32_t other = __shfl(key[r], lower ? 63 - __builtin_clzll(lower) : lane);
      marks[r] = in && (lower == 0 || other != key[r]);
    }
    // one lane per digit moves the wave's counter on (LDS operations of one
    // wave are in order; the barriers keep the compiler from moving them)
    __builtin_amdgcn_wave_barrier();
    if (in && before == 0) cnt[w][dg] = old + (uint32_t)__popcll(same);
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  // counts of the earlier waves on top of the tile's places
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t run = q ? pb : pa;
#pragma unroll
    for (int i = 0; i < kSortWaves; ++i) {
      const uint32_t c = cnt[i][2 * threadIdx.x + q];
      cnt[i][2 * threadIdx.x + q] = run;
      run += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = base + r * 64 + lane;
    if (i < N) {
      const uint32_t at = cnt[w][(key[r] >> shift) & (kDigits - 1)] + rank[r];
      keys_out[at] = key[r];
      pos_out[at] = place[r];
      // the plain read spares a frequent token's word more atomics
      if (bits != nullptr && marks[r] && key[r] < V && ((bits[key[r] >> 5] >> (key[r] & 31)) & 1u) == 0)
        atomicOr(&bits[key[r] >> 5], 1u << (key[r] & 31));
    }
  }
}

// ---------------------------------------------------------------- sums of runs
// A wave takes one tile of `tlen` sorted positions and one slice of 64 chunks
// of the row (512 bf16 or 256 fp32 columns).  part[2 t] holds tile t's piece
// of the run that came in from tile t - 1, part[2 t + 1] its piece of the run
// that goes on into tile t + 1 (a tile inside one run has the first only).
constexpr int kTileMax = 64;
struct RunArgs {
  const uint32_t* skey;
  const uint32_t* spos;
  int64_t N;
  uint32_t V;
  int64_t d;
  int cpr;      // 16-byte chunks of a dY row
  int slices;   // slices of 64 chunks
  int tlen;     // sorted positions per tile
  int64_t tiles;
  float scale;
  int accumulate;
  float* dW;
  float* part;
  const uint32_t* bits;  // a bit per token that occurs, or null: looked up in skey
  int64_t sum_blocks;    // run_sum_kernel's workgroups that sum runs; its others write zeros
  int64_t join_blocks;   // run_join_kernel's that join them; its others write zeros
  int64_t zero_words;    // words of 32 tokens in all, and those of run_sum_kernel
  int64_t zero_first;
};

// dst[0 .. kN) = scale acc, or += for accumulate; a partial row is stored as it is.
template <int kN>
__device__ inline void store_row(float* dst, const float* acc, float scale, bool accumulate) {
#pragma unroll
  for (int q = 0; q < kN / 4; ++q) {
    f32x4_t v = {acc[4 * q] * scale, acc[4 * q + 1] * scale, acc[4 * q + 2] * scale, acc[4 * q + 3] * scale};
    if (accumulate) v += *(const f32x4_t*)(dst + 4 * q);
    *(f32x4_t*)(dst + 4 * q) = v;
  }
}

constexpr int kZeroRows = 32;  // table rows per zeroing workgroup: one word of bits

// Whether token v occurs in the sorted keys (few positions).
__device__ inline bool occurs(const uint32_t* skey, int64_t N, uint32_t v) {
  int64_t lo = 0, hi = N;  // the first key >= v lies in [lo, hi]
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (skey[mid] < v)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo < N && skey[lo] == v;
}

// Zeros in the rows of absent tokens among the kZeroRows of block b (of n),
// by all waves of the workgroup.  The blocks of one XCD (b % 8) take adjacent
// words (1.4 % less time at 201,088 x 2,880 than words in block order).
// present(word): a bit per token of the word that occurs.
template <typename P>
__device__ inline void zero_rows(const RunArgs& a, int64_t word0, int64_t n, int64_t b, P&& present_in) {
  const int64_t per = (n + 7) / 8, at = (b & 7) * per + (b >> 3);
  if ((b >> 3) >= per || at >= n) return;
  const int64_t word = word0 + at, v0 = word * kZeroRows;
  const int lane = threadIdx.x & 63, waves = blockDim.x / 64;
  const uint32_t present = present_in(word);
  const int64_t cols4 = a.d / 4;
  for (int r = threadIdx.x >> 6; r < kZeroRows; r += waves) {
    if (v0 + r >= a.V || ((present >> r) & 1u)) continue;
    f32x4_t* dst = (f32x4_t*)(a.dW + (v0 + r) * a.d);
    for (int64_t c = lane; c < cols4; c += 64) dst[c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
}
__device__ inline void zero_rows(const RunArgs& a, int64_t word0, int64_t n, int64_t b) {
  zero_rows(a, word0, n, b, [&](int64_t word) {
    const int lane = threadIdx.x & 63;
    return a.bits != nullptr
               ? a.bits[word]
               : (uint32_t)__ballot(lane < kZeroRows && occurs(a.skey, a.N, (uint32_t)(word * kZeroRows + lane)));
  });
}
// Blocks for n words: a whole number for each XCD.
inline int64_t zero_blocks(int64_t n) { return (n + 7) / 8 * 8; }

// At most kFewMax positions: one launch without a sort.  The workgroup of a
// position (and slice) whose id does not occur before it sums the rows of all
// its occurrences: a wave those among 64 positions in order, wave 0 then the
// waves' sums in order.  Against rank, sum and join, 256 positions take 6 us for
// 12 at 4,096 x 256 fp32 and 35 for 43 at 32,000 x 2,048 bf16 (the same token
// 256 times: 6 for 11 and 36 for 42).
constexpr int kFewMax = 256;
template <typename T>
__global__ void __launch_bounds__(kThreads) few_sum_kernel(RunArgs a, const int32_t* __restrict__ ids,
                                                           const T* __restrict__ dY) {
  constexpr int kN = Chunk<T>::kN;
  static_assert(kFewMax == kThreads, "a key per thread");
  __shared__ uint32_t keys[kFewMax];
  __shared__ float sums[kThreads / 64][64 * kN];
  const int lane = threadIdx.x & 63, N = (int)a.N;
  keys[threadIdx.x] = (int)threadIdx.x < N ? key_of(ids, threadIdx.x, a.V) : a.V;
  __syncthreads();
  if ((int64_t)blockIdx.x >= a.sum_blocks) {
    zero_rows(a, 0, a.zero_words, (int64_t)blockIdx.x - a.sum_blocks, [&](int64_t word) {
      uint32_t m = 0;
      for (int i = lane; i < N; i += 64) {
        const uint32_t at = keys[i] - (uint32_t)(word * kZeroRows);
        m |= at < (uint32_t)kZeroRows ? 1u << at : 0u;
      }
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) m |= __shfl_xor(m, o);
      return m;
    });
    return;
  }
  const int i = (int)(blockIdx.x / a.slices), slice = (int)(blockIdx.x - i * a.slices);
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t key = __builtin_amdgcn_readfirstlane(keys[i]);
  if (key >= a.V) return;
  for (int b = 0; b <= i; b += 64) {
    const uint64_t before = i - b < 64 ? (1ull << (i - b)) - 1 : ~0ull;
    if (__ballot(keys[b + lane] == key) & before) return;  // that position's workgroup sums it
  }
  const int c = slice * 64 + lane, cl = c < a.cpr ? c : a.cpr - 1;
  float acc[kN];
#pragma unroll
  for (int q = 0; q < kN; ++q) acc[q] = 0.f;
  const u32x4_t* src = (const u32x4_t*)dY;
  constexpr int U = 16;  // rows in flight
  uint64_t m = __ballot(keys[64 * w + lane] == key);
  while (m) {
    u32x4_t v[U];
    const int n = __popcll(m);
    int p = 0;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      p = m ? 64 * w + __builtin_ctzll(m) : p;
      m &= m - 1;
      v[j] = src[(int64_t)p * a.cpr + cl];
    }
#pragma unroll
    for (int j = 0; j < U; ++j) asm volatile("" : "+v"(v[j]));  // none is put off to its use
#pragma unroll
    for (int j = 0; j < U; ++j) {
      float f[kN];
      Chunk<T>::unpack(v[j], f);
#pragma unroll
      for (int q = 0; q < kN; ++q) acc[q] += j < n ? f[q] : 0.f;
    }
  }
#pragma unroll
  for (int q = 0; q < kN; ++q) sums[w][q * 64 + lane] = acc[q];
  __syncthreads();
  if (w > 0 || c >= a.cpr) return;
  for (int j = 1; j < kThreads / 64; ++j)
#pragma unroll
    for (int q = 0; q < kN; ++q) acc[q] += sums[j][q * 64 + lane];
  store_row<kN>(a.dW + (int64_t)key * a.d + (int64_t)c * kN, acc, a.scale, a.accumulate != 0);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) run_sum_kernel(RunArgs a, const T* __restrict__ dY, int groups) {
  constexpr int kN = Chunk<T>::kN;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // sums first: they wait for scattered reads, and the zeros' writes fill in
  // (alternating the two instead took 6 % longer)
  if ((int64_t)blockIdx.x >= a.sum_blocks) {
    zero_rows(a, 0, a.zero_first, (int64_t)blockIdx.x - a.sum_blocks);
    return;
  }
  const int64_t sum_block = blockIdx.x;
  const int64_t t = sum_block / groups;
  const int slice = (int)(sum_block - t * groups) * (kThreads / 64) + wave;
  if (slice >= a.slices) return;
  const int c = slice * 64 + lane;
  const bool on = c < a.cpr;
  const int cl = on ? c : a.cpr - 1;
  const int64_t b = t * a.tlen, e = b + a.tlen < a.N ? b + a.tlen : a.N;
  const uint32_t before = b > 0 ? a.skey[b - 1] : 0xFFFFFFFFu;
  const uint32_t after = e < a.N ? a.skey[e] : 0xFFFFFFFFu;
  // the tile's keys and positions, one a lane: read here at once, later by lane
  static_assert(kTileMax <= 64, "a lane per position of a tile");
  const int64_t mine = b + lane < e ? b + lane : e - 1;
  const uint32_t keys = a.skey[mine], places = a.spos[mine];
  uint32_t cur = __builtin_amdgcn_readlane(keys, 0);
  if (cur >= a.V) return;  // only positions without a token from here on
  const bool head = cur == before;
  bool first = true;  // the current run is the tile's first
  float acc[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) acc[i] = 0.f;
  const u32x4_t* src = (const u32x4_t*)dY;
  auto flush = [&](bool goes_on) {
    if (!on) return;
    if (first && head)
      store_row<kN>(a.part + (2 * t) * a.d + (int64_t)c * kN, acc, 1.f, false);
    else if (goes_on)
      store_row<kN>(a.part + (2 * t + 1) * a.d + (int64_t)c * kN, acc, 1.f, false);
    else
      store_row<kN>(a.dW + (int64_t)cur * a.d + (int64_t)c * kN, acc, a.scale, a.accumulate != 0);
  };
  // Rows in flight, loaded without conditions (lanes past the row take its last
  // chunk, positions without a token their own row, and neither is used): under
  // conditions each load waited, 4,096 x 2,048 of 32,000 70 us instead of 60.
  constexpr int U = 8;
  for (int64_t i0 = b; i0 < e; i0 += U) {
    u32x4_t v[U];
    uint32_t k[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = (int)((i0 + j < e ? i0 + j : e - 1) - b);
      k[j] = __builtin_amdgcn_readlane(keys, i);
      const uint32_t p = __builtin_amdgcn_readlane(places, i);
      v[j] = src[(int64_t)p * a.cpr + cl];
    }
#pragma unroll
    for (int j = 0; j < U; ++j) asm volatile("" : "+v"(v[j]));  // none is put off to its use
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (i0 + j >= e) break;
      if (k[j] != cur) {
        flush(false);
        if (k[j] >= a.V) return;
        cur = k[j];
        first = false;
#pragma unroll
        for (int i = 0; i < kN; ++i) acc[i] = 0.f;
      }
      float f[kN];
      Chunk<T>::unpack(v[j], f);
#pragma unroll
      for (int i = 0; i < kN; ++i) acc[i] += f[i];
    }
  }
  flush(after == cur);
}

// Runs that cross tiles: the workgroup of the tile where such a run starts (one
// per slice) sums its pieces.  Its waves take equal stretches of the tiles and
// wave 0 adds their sums in order.  Most of these workgroups find no run and
// the longest run takes 20 us, so a share of the zeros is left to this launch.
constexpr int kJoinWaves = 8;
template <int kN>
__global__ void __launch_bounds__(kJoinWaves * 64) run_join_kernel(RunArgs a) {
  __shared__ float sums[kJoinWaves][64 * kN];
  if ((int64_t)blockIdx.x >= a.join_blocks) {
    zero_rows(a, a.zero_first, a.zero_words - a.zero_first, (int64_t)blockIdx.x - a.join_blocks);
    return;
  }
  const int64_t t = blockIdx.x / a.slices;
  const int slice = (int)(blockIdx.x - t * a.slices);
  const int64_t e = (t + 1) * a.tlen;
  if (e >= a.N) return;
  const uint32_t key = a.skey[e - 1];
  if (key >= a.V || a.skey[e] != key) return;        // no run goes on
  if (t > 0 && a.skey[t * a.tlen - 1] == key) return;  // it started earlier
  // last tile of the run: the last whose first position still has the key
  int64_t lo = t + 1, hi = a.tiles - 1;
  while (lo < hi) {
    const int64_t mid = lo + (hi - lo + 1) / 2;
    if (a.skey[mid * a.tlen] == key)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t pieces = lo - t + 1;  // piece 0 is tile t's second partial, piece i tile (t + i)'s first
  const int64_t per = (pieces + kJoinWaves - 1) / kJoinWaves;
  const int64_t p0 = w * per, p1 = p0 + per < pieces ? p0 + per : pieces;
  const int c = slice * 64 + lane;
  const bool on = c < a.cpr;
  float acc[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) acc[i] = 0.f;
  if (on) {
#pragma unroll 8
    for (int64_t p = p0; p < p1; ++p) {
      const float* src = a.part + (p == 0 ? 2 * t + 1 : 2 * (t + p)) * a.d + (int64_t)c * kN;
#pragma unroll
      for (int q = 0; q < kN / 4; ++q) {
        const f32x4_t v = *(const f32x4_t*)(src + 4 * q);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[4 * q + i] += v[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) sums[w][i * 64 + lane] = acc[i];
  __syncthreads();
  if (w == 0 && on) {
    const int waves = (int)((pieces + per - 1) / per);
    for (int j = 1; j < waves; ++j)
#pragma unroll
      for (int i = 0; i < kN; ++i) acc[i] += sums[j][i * 64 + lane];
    store_row<kN>(a.dW + (int64_t)key * a.d + (int64_t)c * kN, acc, a.scale, a.accumulate != 0);
  }
}

inline uint64_t align256(uint64_t x) { return (x + 255) & ~uint64_t(255); }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Sorted positions per tile: short tiles while there are few positions (more
// waves in flight), long ones later (fewer partial rows).
inline int tile_len(int64_t N) { return N <= 8192 ? 16 : N <= 16384 ? 32 : kTileMax; }

struct BwdLayout {
  int64_t tiles = 0, sort_tiles = 0;
  int passes = 0;  // radix passes; 0 = counted ranks
  uint64_t key0 = 0, pos0 = 0, key1 = 0, pos1 = 0, hist = 0, bits = 0, part = 0, total = 0;
};

BwdLayout bwd_layout(int64_t N, int64_t d, int64_t V) {
  BwdLayout L;
  L.tiles = cdiv(N, tile_len(N));
  if (N > kRankMax) {
    int bits = 1;
    while (((int64_t)1 << bits) <= V) ++bits;  // keys are 0 .. V
    L.passes = (bits + kDigit - 1) / kDigit;
    L.sort_tiles = cdiv(N, kSortTile);
  }
  uint64_t off = 0;
  const uint64_t list = align256((uint64_t)N * 4);
  L.key0 = off, off += list;
  L.pos0 = off, off += list;
  if (L.passes) {
    L.key1 = off, off += list;
    L.pos1 = off, off += list;
    L.hist = off, off += align256((uint64_t)L.sort_tiles * kDigits * 4);
  }
  L.bits = off, off += align256((uint64_t)cdiv(V, 32) * 4);
  L.part = off, off += L.tiles > 1 ? align256((uint64_t)L.tiles * 2 * d * 4) : 0;
  L.total = off;
  return L;
}

template <typename T>
hipError_t launch_runs(RunArgs a, const int32_t* ids, const void* dY, hipStream_t s) {
  constexpr int kN = Chunk<T>::kN;
  a.cpr = (int)(a.d / kN);
  a.slices = (int)cdiv(a.cpr, 64);
  if (a.N <= kFewMax) {
    a.sum_blocks = a.N * a.slices;
    hipLaunchKernelGGL(few_sum_kernel<T>, dim3((unsigned)(a.sum_blocks + zero_blocks(a.zero_words))), dim3(kThreads), 0,
                       s, a, ids, (const T*)dY);
    return hipGetLastError();
  }
  const int groups = (int)cdiv(a.slices, kThreads / 64);
  a.sum_blocks = a.tiles * groups;
  a.join_blocks = (a.tiles - 1) * a.slices;
  a.zero_first = a.join_blocks > 0 ? a.zero_words - a.zero_words / 4 : a.zero_words;
  hipLaunchKernelGGL(run_sum_kernel<T>, dim3((unsigned)(a.sum_blocks + zero_blocks(a.zero_first))), dim3(kThreads), 0,
                     s, a, (const T*)dY, groups);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.join_blocks == 0) return e;
  hipLaunchKernelGGL(run_join_kernel<kN>, dim3((unsigned)(a.join_blocks + zero_blocks(a.zero_words - a.zero_first))),
                     dim3(kJoinWaves * 64), 0, s, a);
  return hipGetLastError();
}

}  // namespace

namespace {
// Lanes of a row, as their binary logarithm.
inline int embed_lanes(int cpr) {
  int lg = 0;
  while (lg < 6 && (1 << lg) < cpr) ++lg;
  return lg;
}
inline int row_chunks(Dtype dt, int64_t d) { return (int)(d / (dt == DT_BF16 ? 8 : 4)); }
}  // namespace

int64_t embed_blocks(Dtype dt, int64_t N, int64_t d) { return cdiv(N, kThreads >> embed_lanes(row_chunks(dt, d))); }

hipError_t launch_embed(Dtype dt, const int32_t* ids, const void* W, float scale, int64_t N, int64_t d, int64_t V,
                        void* out, hipStream_t s) {
  const int cpr = row_chunks(dt, d), lg = embed_lanes(cpr);
  const unsigned grid = (unsigned)embed_blocks(dt, N, d);
  if (dt == DT_BF16)
    hipLaunchKernelGGL(embed_kernel<__bf16>, dim3(grid), dim3(kThreads), 0, s, ids, (const __bf16*)W, scale, N, V, cpr,
                       lg, (__bf16*)out);
  else
    hipLaunchKernelGGL(embed_kernel<float>, dim3(grid), dim3(kThreads), 0, s, ids, (const float*)W, scale, N, V, cpr,
                       lg, (float*)out);
  return hipGetLastError();
}

uint64_t embed_bwd_workspace(int64_t N, int64_t d, int64_t V) { return N > 0 ? bwd_layout(N, d, V).total : 0; }

int64_t embed_bwd_blocks(Dtype dt, int64_t N, int64_t d, int64_t V) {
  const int64_t slices = cdiv(d / (dt == DT_BF16 ? 8 : 4), 64);
  const int64_t tiles = cdiv(N, tile_len(N));
  const int64_t words = cdiv(V, kZeroRows) + 8;
  const int64_t sum = tiles * cdiv(slices, kThreads / 64) + words;
  const int64_t join = ((tiles - 1) * slices + words) * (kJoinWaves * 64 / kThreads);  // of twice the threads
  return sum > join ? sum : join;
}

hipError_t launch_embed_bwd(Dtype dt, const int32_t* ids, const void* dY, float scale, int64_t N, int64_t d, int64_t V,
                            bool accumulate, float* dW, void* ws, hipStream_t s) {
  const BwdLayout L = bwd_layout(N, d, V);
  char* base = (char*)ws;
  uint32_t* skey = (uint32_t*)(base + L.key0);
  uint32_t* spos = (uint32_t*)(base + L.pos0);
  uint32_t* bits = nullptr;
  hipError_t e = hipSuccess;
#define EMBED_TRY()                            \
  if ((e = hipGetLastError()) != hipSuccess) return e
  if (N <= kFewMax) {
    // no sort
  } else if (L.passes == 0) {
    hipLaunchKernelGGL(rank_kernel, dim3((unsigned)cdiv(N, kThreads / kRankLanes)), dim3(kThreads), 0, s, ids, (int)N,
                       (uint32_t)V, skey, spos);
    EMBED_TRY();
  } else {
    // an accumulating call leaves the other rows alone and needs no bits
    if (!accumulate) bits = (uint32_t*)(base + L.bits);
    uint32_t* key1 = (uint32_t*)(base + L.key1);
    uint32_t* pos1 = (uint32_t*)(base + L.pos1);
    uint32_t* hist = (uint32_t*)(base + L.hist);
    const uint32_t *kin = nullptr, *pin = nullptr;  // the first pass reads the ids
    const dim3 grid((unsigned)L.sort_tiles);
    const int st = (int)L.sort_tiles;
    const bool scan = L.sort_tiles > kDirectTiles;
    for (int p = 0; p < L.passes; ++p) {
      // the last pass writes skey / spos
      uint32_t* kout = (L.passes - p) % 2 ? skey : key1;
      uint32_t* pout = (L.passes - p) % 2 ? spos : pos1;
      hipLaunchKernelGGL(sort_hist_kernel, grid, dim3(kThreads), 0, s, ids, kin, N, (uint32_t)V, p * kDigit, st, hist,
                         p == 0 ? bits : nullptr, cdiv(V, 32));
      EMBED_TRY();
      if (scan) {
        hipLaunchKernelGGL(sort_scan_kernel, dim3(1), dim3(kThreads), 0, s, hist, L.sort_tiles);
        EMBED_TRY();
      }
      hipLaunchKernelGGL(sort_scatter_kernel, grid, dim3(kThreads), 0, s, ids, kin, pin, N, (uint32_t)V, p * kDigit, st,
                         scan, hist, kout, pout, p == L.passes - 1 ? bits : nullptr);
      EMBED_TRY();
      kin = kout;
      pin = pout;
    }
  }
#undef EMBED_TRY
  RunArgs a{};
  a.skey = skey;
  a.spos = spos;
  a.N = N;
  a.V = (uint32_t)V;
  a.d = d;
  a.tlen = tile_len(N);
  a.tiles = L.tiles;
  a.scale = scale;
  a.accumulate = accumulate ? 1 : 0;
  a.dW = dW;
  a.part = (float*)(base + L.part);
  a.bits = bits;
  a.zero_words = accumulate ? 0 : cdiv(V, kZeroRows);
  return dt == DT_BF16 ? launch_runs<__bf16>(a, ids, dY, s) : launch_runs<float>(a, ids, dY, s);
}

}  // namespace ckl
