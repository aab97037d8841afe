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
// workgroups of the same launch (by a bit per token), so every byte of dW is
// written once; those zeros bound the call for large vocabularies.
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

// Bit v of `bits` is set where token v occurs.
__global__ void __launch_bounds__(kThreads) clear_kernel(uint32_t* p, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i < n) p[i] = 0;
}
__device__ inline void mark(uint32_t* bits, uint32_t key, uint32_t V) {
  // the plain read spares a frequent token's word most of its atomics
  if (bits != nullptr && key < V && ((bits[key >> 5] >> (key & 31)) & 1u) == 0) atomicOr(&bits[key >> 5], 1u << (key & 31));
}

// Few positions: a position's place is the number of positions before it in
// (id, position) order, counted directly.  Four lanes share one position and
// the list passes through LDS; one launch in place of the radix sort's six.
constexpr int kRankMax = 8192;
constexpr int kRankTile = 2048;
__global__ void __launch_bounds__(kThreads) rank_kernel(const int32_t* __restrict__ ids, int N, uint32_t V,
                                                        uint32_t* __restrict__ skey, uint32_t* __restrict__ spos,
                                                        uint32_t* __restrict__ bits) {
  __shared__ __attribute__((aligned(16))) uint32_t tile[kRankTile];
  const int i = blockIdx.x * (kThreads / 4) + (threadIdx.x >> 2), part = threadIdx.x & 3;
  const uint32_t key = i < N ? key_of(ids, i, V) : 0;
  int place = 0;
  for (int t0 = 0; t0 < N; t0 += kRankTile) {
    const int n = min(kRankTile, N - t0);
    __syncthreads();
    for (int j = threadIdx.x; j < kRankTile; j += kThreads) tile[j] = j < n ? key_of(ids, t0 + j, V) : 0xFFFFFFFFu;
    __syncthreads();
    for (int j = 4 * part; j < n; j += 16) {
      const u32x4_t k = *(const u32x4_t*)&tile[j];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t kq = k[q];
        place += (kq < key || (kq == key && t0 + j + q < i)) ? 1 : 0;
      }
    }
  }
  place += __shfl_xor(place, 1);
  place += __shfl_xor(place, 2);
  if (i < N && part == 0) {
    skey[place] = key;
    spos[place] = (uint32_t)i;
    mark(bits, key, V);
  }
}

// Many positions: a stable radix sort of the keys, kDigit bits a pass (two
// passes up to 2^18 - 1 tokens).  Per pass: a histogram per tile, an exclusive
// scan of the counts in (digit, tile) order, and a scatter in which each wave
// ranks its own stretch of the tile in order.
constexpr int kDigit = 9;
constexpr int kDigits = 1 << kDigit;
constexpr int kSortTile = 2048;
constexpr int kSortWaves = kThreads / 64;
constexpr int kRounds = kSortTile / kThreads;  // 64-element rounds per wave

// Element i of the pass: from the ids on the first pass (keys == null).
__device__ inline uint32_t pass_key(const int32_t* ids, const uint32_t* keys, int64_t i, uint32_t V) {
  return keys != nullptr ? keys[i] : key_of(ids, i, V);
}

__global__ void __launch_bounds__(kThreads) sort_hist_kernel(const int32_t* __restrict__ ids,
                                                             const uint32_t* __restrict__ keys, int64_t N, uint32_t V,
                                                             int shift, int tiles, uint32_t* __restrict__ hist,
                                                             uint32_t* __restrict__ bits) {
  __shared__ uint32_t h[kDigits];
  for (int i = threadIdx.x; i < kDigits; i += kThreads) h[i] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * kSortTile;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = base + r * kThreads + threadIdx.x;
    if (i < N) {
      const uint32_t k = pass_key(ids, keys, i, V);
      atomicAdd(&h[(k >> shift) & (kDigits - 1)], 1u);
      if (keys == nullptr) mark(bits, k, V);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kDigits; i += kThreads) hist[(int64_t)i * tiles + blockIdx.x] = h[i];
}

// Exclusive scan of n counts in place, one workgroup.
constexpr int kScanThreads = 1024;
__global__ void __launch_bounds__(kScanThreads) sort_scan_kernel(uint32_t* __restrict__ hist, int64_t n) {
  __shared__ uint32_t wsum[kScanThreads / 64];
  const int64_t per = (n + kScanThreads - 1) / kScanThreads;
  const int64_t b = threadIdx.x * per, e = b + per < n ? b + per : n;
  uint32_t mine = 0;
  for (int64_t i = b; i < e; ++i) mine += hist[i];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  uint32_t x = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  if (lane == 63) wsum[w] = x;
  __syncthreads();
  uint32_t run = x - mine;
  for (int i = 0; i < w; ++i) run += wsum[i];
  for (int64_t i = b; i < e; ++i) {
    const uint32_t c = hist[i];
    hist[i] = run;
    run += c;
  }
}

__global__ void __launch_bounds__(kThreads) sort_scatter_kernel(const int32_t* __restrict__ ids,
                                                                const uint32_t* __restrict__ keys,
                                                                const uint32_t* __restrict__ pos, int64_t N,
                                                                uint32_t V, int shift, int tiles,
                                                                const uint32_t* __restrict__ offs,
                                                                uint32_t* __restrict__ keys_out,
                                                                uint32_t* __restrict__ pos_out) {
  __shared__ uint32_t cnt[kSortWaves][kDigits];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < kSortWaves * kDigits; i += kThreads) (&cnt[0][0])[i] = 0;
  __syncthreads();
  // wave w owns elements [64 kRounds w, 64 kRounds (w + 1)) of the tile, in order
  const int64_t base = (int64_t)blockIdx.x * kSortTile + (int64_t)w * 64 * kRounds;
  uint32_t key[kRounds], rank[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t i = base + r * 64 + lane;
    key[r] = i < N ? pass_key(ids, keys, i, V) : 0xFFFFFFFFu;
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
    const uint32_t before = __builtin_amdgcn_mbcnt_hi((uint32_t)(same >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)same, 0));
    const uint32_t old = in ? cnt[w][dg] : 0;
    rank[r] = old + before;
    // one lane per digit moves the wave's counter on (LDS operations of one
    // wave are in order; the barrier keeps the compiler from moving them)
    __builtin_amdgcn_wave_barrier();
    if (in && before == 0) cnt[w][dg] = old + (uint32_t)__popcll(same);
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  // counts of the earlier waves, and the tile's place in the whole list
  for (int d = threadIdx.x; d < kDigits; d += kThreads) {
    uint32_t run = offs[(int64_t)d * tiles + blockIdx.x];
#pragma unroll
    for (int i = 0; i < kSortWaves; ++i) {
      const uint32_t c = cnt[i][d];
      cnt[i][d] = run;
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
      pos_out[at] = pos != nullptr ? pos[i] : (uint32_t)i;
    }
  }
}

// ---------------------------------------------------------------- sums of runs
// A wave takes one tile of `tlen` sorted positions and one slice of 64 chunks
// of the row (512 bf16 or 256 fp32 columns).  part[2 t] holds tile t's piece
// of the run that came in from tile t - 1, part[2 t + 1] its piece of the run
// that goes on into tile t + 1 (a tile inside one run has the first only).
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
  const uint32_t* bits;
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

template <typename T>
__global__ void __launch_bounds__(kThreads) run_sum_kernel(RunArgs a, const T* __restrict__ dY, int64_t reduce_blocks,
                                                           int groups) {
  constexpr int kN = Chunk<T>::kN;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if ((int64_t)blockIdx.x >= reduce_blocks) {
    // rows of absent tokens
    const int64_t word = (int64_t)blockIdx.x - reduce_blocks;
    const uint32_t present = a.bits[word];
    const int64_t v0 = word * kZeroRows;
    const int64_t cols4 = a.d / 4;
    for (int r = wave; r < kZeroRows; r += kThreads / 64) {
      if (v0 + r >= a.V || ((present >> r) & 1u)) continue;
      f32x4_t* dst = (f32x4_t*)(a.dW + (v0 + r) * a.d);
      for (int64_t c = lane; c < cols4; c += 64) dst[c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    return;
  }
  const int64_t t = (int64_t)blockIdx.x / groups;
  const int slice = (int)((int64_t)blockIdx.x - t * groups) * (kThreads / 64) + wave;
  if (slice >= a.slices) return;
  const int c = slice * 64 + lane;
  const bool on = c < a.cpr;
  const int64_t b = t * a.tlen, e = b + a.tlen < a.N ? b + a.tlen : a.N;
  const uint32_t before = b > 0 ? a.skey[b - 1] : 0xFFFFFFFFu;
  const uint32_t after = e < a.N ? a.skey[e] : 0xFFFFFFFFu;
  uint32_t cur = a.skey[b];
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
  constexpr int U = 8;  // rows in flight
  for (int64_t i0 = b; i0 < e; i0 += U) {
    u32x4_t v[U];
    uint32_t k[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int64_t i = i0 + j < e ? i0 + j : e - 1;
      k[j] = __builtin_amdgcn_readfirstlane(a.skey[i]);
      const uint32_t p = __builtin_amdgcn_readfirstlane(a.spos[i]);
      if (on && k[j] < a.V) v[j] = src[(int64_t)p * a.cpr + c];
    }
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

// Runs that cross tiles: the workgroup of the tile where such a run starts
// sums its pieces.  Its waves take equal stretches of the tiles and wave 0
// adds their sums in order.
constexpr int kJoinWaves = 8;
template <int kN>
__global__ void __launch_bounds__(kJoinWaves * 64) run_join_kernel(RunArgs a) {
  __shared__ float sums[kJoinWaves][64 * kN];
  const int64_t t = blockIdx.x;
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
  for (int slice = blockIdx.y; slice < a.slices; slice += gridDim.y) {
    const int c = slice * 64 + lane;
    const bool on = c < a.cpr;
    float acc[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) acc[i] = 0.f;
    if (on) {
#pragma unroll 4
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
    __syncthreads();
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
}

inline uint64_t align256(uint64_t x) { return (x + 255) & ~uint64_t(255); }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Sorted positions per tile: short tiles while there are few positions (more
// waves in flight), long ones later (fewer partial rows).
inline int tile_len(int64_t N) { return N <= 8192 ? 16 : N <= 65536 ? 32 : 64; }

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
hipError_t launch_runs(RunArgs a, const void* dY, int64_t zero_blocks, hipStream_t s) {
  constexpr int kN = Chunk<T>::kN;
  a.cpr = (int)(a.d / kN);
  a.slices = (int)cdiv(a.cpr, 64);
  const int groups = (int)cdiv(a.slices, kThreads / 64);
  const int64_t reduce_blocks = a.tiles * groups;
  hipLaunchKernelGGL(run_sum_kernel<T>, dim3((unsigned)(reduce_blocks + zero_blocks)), dim3(kThreads), 0, s, a,
                     (const T*)dY, reduce_blocks, groups);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.tiles < 2) return e;
  hipLaunchKernelGGL(run_join_kernel<kN>, dim3((unsigned)(a.tiles - 1), (unsigned)a.slices), dim3(kJoinWaves * 64), 0,
                     s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embed(Dtype dt, const int32_t* ids, const void* W, float scale, int64_t N, int64_t d, int64_t V,
                        void* out, hipStream_t s) {
  const int cpr = (int)(d / (dt == DT_BF16 ? 8 : 4));
  int lg = 0;
  while (lg < 6 && (1 << lg) < cpr) ++lg;
  const unsigned grid = (unsigned)cdiv(N, kThreads >> lg);
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
  return tiles * cdiv(slices, kThreads / 64) + cdiv(V, kZeroRows);
}

hipError_t launch_embed_bwd(Dtype dt, const int32_t* ids, const void* dY, float scale, int64_t N, int64_t d, int64_t V,
                            bool accumulate, float* dW, void* ws, hipStream_t s) {
  const BwdLayout L = bwd_layout(N, d, V);
  char* base = (char*)ws;
  uint32_t* skey = (uint32_t*)(base + L.key0);
  uint32_t* spos = (uint32_t*)(base + L.pos0);
  // an accumulating call leaves the other rows alone and needs no bits
  uint32_t* bits = accumulate ? nullptr : (uint32_t*)(base + L.bits);
  hipError_t e = hipSuccess;
#define EMBED_TRY()                            \
  if ((e = hipGetLastError()) != hipSuccess) return e
  if (bits != nullptr) {
    const int64_t words = cdiv(V, 32);
    hipLaunchKernelGGL(clear_kernel, dim3((unsigned)cdiv(words, kThreads)), dim3(kThreads), 0, s, bits, words);
    EMBED_TRY();
  }
  if (L.passes == 0) {
    hipLaunchKernelGGL(rank_kernel, dim3((unsigned)cdiv(N, kThreads / 4)), dim3(kThreads), 0, s, ids, (int)N,
                       (uint32_t)V, skey, spos, bits);
    EMBED_TRY();
  } else {
    uint32_t* key1 = (uint32_t*)(base + L.key1);
    uint32_t* pos1 = (uint32_t*)(base + L.pos1);
    uint32_t* hist = (uint32_t*)(base + L.hist);
    const uint32_t *kin = nullptr, *pin = nullptr;  // the first pass reads the ids
    const dim3 grid((unsigned)L.sort_tiles);
    const int st = (int)L.sort_tiles;
    for (int p = 0; p < L.passes; ++p) {
      // the last pass writes skey / spos
      uint32_t* kout = (L.passes - p) % 2 ? skey : key1;
      uint32_t* pout = (L.passes - p) % 2 ? spos : pos1;
      hipLaunchKernelGGL(sort_hist_kernel, grid, dim3(kThreads), 0, s, ids, kin, N, (uint32_t)V, p * kDigit, st, hist,
                         bits);
      EMBED_TRY();
      hipLaunchKernelGGL(sort_scan_kernel, dim3(1), dim3(kScanThreads), 0, s, hist, (int64_t)st * kDigits);
      EMBED_TRY();
      hipLaunchKernelGGL(sort_scatter_kernel, grid, dim3(kThreads), 0, s, ids, kin, pin, N, (uint32_t)V, p * kDigit, st,
                         hist, kout, pout);
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
  const int64_t zero_blocks = bits != nullptr ? cdiv(V, kZeroRows) : 0;
  return dt == DT_BF16 ? launch_runs<__bf16>(a, dY, zero_blocks, s) : launch_runs<float>(a, dY, zero_blocks, s);
}

}  // namespace ckl
