// Log-probabilities of given tokens and entropy from hidden states and the head's
// weight, without N x V logits, and their gradients.
//
// Forward: the logits contraction of a chunk of rows keeps, of every slice of a
// row (the ids of one wave), its largest logit m_s, sum exp(z - m_s) and
// sum exp(z - m_s) (z - m_s), and nothing else; a merge of the slices gives the
// row's statistics.  The given tokens' logits are T dot products a row
// (T d products beside the contraction's V d).
//
// Backward: the contraction runs again and its epilogue turns logits into the
// gradient's dense part G_j = -p_j (w + u (log p_j + entropy)), w the sum of the
// row's given weights, and dH = G W, dW = G^T H follow as in the loss.  One given
// token a row is added by the epilogue; of several, a kernel of its own writes
// their elements from their log-probabilities.
//
// Roundings: G is held in the path's type, as in the loss, because the matrix cores
// take bf16 operands at 16 times fp32's rate; it adds a half step of its own to that of
// a bf16 result (4,096 rows: errors of dH and dW 2.4e-3 of their norm, 1.7e-3 with G in
// fp32).  A bf16 logit is one fp32 sum over d (entropies 2.4e-7; a slab at a time, as
// fp32 products are summed, 0.9e-7 for up to 5 % of the time).
//
// Many rows are bound by the matrix cores, few by reading W.  Measured (MI355X):
//  4,096 rows (3,686 count) x 201,088 x 2,880 bf16: forward 3.37 ms (1,267 TFLOP/s),
//    gradient's logits 3.49, dH 3.75, dW 3.74 ms; both passes 14.4 to 14.9 ms, by card.
//  256 rows of the same: forward 310 us, backward 1,250 (dW 616 of it, 1.16 GB written).
//  1 row: 191 us for W's 1.16 GB (6.1 TB/s), 7 for the merge; backward 770 us.  fp32: 577
//    us, bound by the matrix cores, since a tile of 64 rows multiplies 63 of padding.
//  256 x 4,096 x 256 fp32, both passes: 46 us, six launches of 3 to 13 us.
#include <math.h>

#include "gemm_core.hpp"
#include "row_io.hpp"

namespace ckl {

namespace {

constexpr float kFar = -1000.f;  // exp(kFar) is 0 in fp32

// z = H_n . W_id in fp32, by one wave.
template <typename T>
__device__ inline float given_logit(const HeadArgs& p, int64_t n, int32_t id) {
  const T* h = (const T*)p.H + n * p.d;
  const T* w = (const T*)p.W + (int64_t)id * p.d;
  float s = 0.f;
  int64_t k = 8 * (threadIdx.x & 63);
  for (; k + 512 < p.d; k += 1024) {  // two vectors of each in flight
    Eight<T> a, b, c, e;
    a.load(h + k);
    b.load(w + k);
    c.load(h + k + 512);
    e.load(w + k + 512);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = __builtin_fmaf(a.get(i), b.get(i), s);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = __builtin_fmaf(c.get(i), e.get(i), s);
  }
  if (k < p.d) {
    Eight<T> a, b;
    a.load(h + k);
    b.load(w + k);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = __builtin_fmaf(a.get(i), b.get(i), s);
  }
  return lanes_sum(s, 64);
}

// Rows [r0, r0 + rows) of the call: the slices' statistics to the rows', and the
// given tokens' log-probabilities.  With a compacted chunk, pos gives each row's
// place in it, -1 for a masked one.
template <typename T, int NT>
__global__ void __launch_bounds__(NT) head_rows_kernel(HeadArgs p, int64_t r0, const float2* __restrict__ part,
                                                      const float* __restrict__ part_a, int n_slices,
                                                      const int* __restrict__ pos) {
  constexpr int NW = NT / 64, U = 8;  // slices in flight per thread
  __shared__ float red[3 * NW];
  const int64_t row = r0 + blockIdx.x;
  const int t = threadIdx.x, w = t >> 6;
  const int64_t at = pos != nullptr ? pos[blockIdx.x] : (int64_t)blockIdx.x;
  if (at < 0) {
    for (int i = t; i < p.T; i += NT) p.logp[row * p.T + i] = 0.f;
    if (t == 0) p.entropy[row] = p.stats[row] = p.stats[p.N + row] = 0.f;
    return;
  }
  const float2* q = part + at * n_slices;
  const float* qa = part_a + at * n_slices;
  float M = -INFINITY, s = 0.f, a = 0.f;
  for (int i0 = t; i0 < n_slices; i0 += U * NT) {
    float2 v[U];
    float va[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * NT < n_slices ? i0 + u * NT : i0;
      v[u] = q[i];
      va[u] = qa[i];
    }
    float m = M;
#pragma unroll
    for (int u = 0; u < U; ++u) m = fmaxf(m, v[u].x);
    const float d0 = fmaxf(M - m, kFar), k0 = __expf(d0);
    a = __builtin_fmaf(s, d0, a) * k0;
    s *= k0;
    M = m;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * NT >= n_slices) continue;
      const float dm = fmaxf(v[u].x - m, kFar), k = __expf(dm);
      s = __builtin_fmaf(v[u].y, k, s);
      a = __builtin_fmaf(__builtin_fmaf(v[u].y, dm, va[u]), k, a);
    }
  }
  float top = wave_max(M);
  if ((t & 63) == 0) red[w] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NW; ++i) top = fmaxf(top, red[i]);
  const float d1 = fmaxf(M - top, kFar), k1 = __expf(d1);
  a = lanes_sum(__builtin_fmaf(s, d1, a) * k1, 64);
  s = lanes_sum(s * k1, 64);
  if ((t & 63) == 0) {
    red[NW + w] = s;
    red[2 * NW + w] = a;
  }
  __syncthreads();
  s = a = 0.f;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    s += red[NW + i];
    a += red[2 * NW + i];
  }
  const bool none = s == 0.f;  // every logit is -inf: log-probabilities -inf, entropy 0
  const float logs = none ? 0.f : logf(s), h = none ? 0.f : logs - a / s;
  for (int i = w; i < p.T; i += NW) {
    const int32_t id = p.ids[row * p.T + i];
    const bool in = id >= 0 && id < p.V;
    const float z = in ? given_logit<T>(p, row, id) : 0.f;
    // z and the contraction's logits add in different orders: their difference may round above 0
    const float l = none ? -INFINITY : __builtin_elementwise_minimum((z - top) - logs, 0.f);
    if ((t & 63) == 0) p.logp[row * p.T + i] = in ? l : 0.f;
  }
  if (t == 0) {
    p.entropy[row] = h < 0.f ? 0.f : h;
    p.stats[row] = none ? -INFINITY : top;
    p.stats[p.N + row] = logs;
  }
}

// Coefficients of the chunk's rows for the gradient's epilogue.
__global__ void __launch_bounds__(256) head_coef_kernel(HeadGradArgs p, int64_t r0, int64_t rows,
                                                       const int* __restrict__ vidx, const int* __restrict__ live,
                                                       float4* __restrict__ coef) {
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (i >= rows || (live != nullptr && i >= *live)) return;
  const int64_t n = r0 + (vidx != nullptr ? vidx[i] : i);
  float w = 0.f;
  for (int k = lane; k < p.T; k += 64) {
    const int32_t id = p.ids[n * p.T + k];
    if (id >= 0 && id < p.V) w += p.dlogp[n * p.T + k];
  }
  w = lanes_sum(w, 64);
  if (lane == 0) {
    const float u = p.dentropy != nullptr ? p.dentropy[n] : 0.f;
    coef[i] = make_float4(p.stats[n], p.stats[p.N + n], __builtin_fmaf(u, p.dentropy != nullptr ? p.entropy[n] : 0.f, w), u);
  }
}

// G at the given tokens, from their log-probabilities: one wave per row.  A token
// given more than once takes the sum of its weights, written by its first mention.
template <typename T>
__global__ void __launch_bounds__(256) head_given_kernel(HeadGradArgs p, int64_t r0, int64_t rows,
                                                        const int* __restrict__ vidx, const int* __restrict__ live,
                                                        const float4* __restrict__ coef, T* __restrict__ G, int64_t gblk) {
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (i >= rows || (live != nullptr && i >= *live)) return;
  const int64_t n = r0 + (vidx != nullptr ? vidx[i] : i);
  const int32_t* ids = p.ids + n * p.T;
  const float4 c = coef[i];
  if (c.x == -INFINITY) return;
  for (int k = lane; k < p.T; k += 64) {
    const int32_t id = ids[k];
    if (id < 0 || id >= p.V) continue;
    bool first = true;
    float w = 0.f;
    for (int j = 0; j < p.T; ++j)
      if (ids[j] == id) {
        first = first && j >= k;
        w += p.dlogp[n * p.T + j];
      }
    if (!first) continue;
    const float l = __builtin_elementwise_maximum(p.logp[n * p.T + k], kFar);
    const float g = w - __builtin_amdgcn_exp2f(l * kLog2e) * __builtin_fmaf(c.w, l, c.z);
    G[(i >> 6) * gblk + ((int64_t)id >> 6) * 4096 + (i & 63) * 64 + (id & 63)] = (T)g;
  }
}

// Tiles of an m x n product: 256 x 256 (eight waves, the loss's), 128 x 128 and
// 64 x 64 (four waves), the last two for products that would leave compute units
// without a tile.
int tile_edge(HeadTile t) { return t == TILE_256 ? 256 : t == TILE_128 ? 128 : 64; }
int64_t tiles_of(int64_t m, int64_t n, HeadTile t) {
  const int e = tile_edge(t);
  return ((m + e - 1) / e) * ((n + e - 1) / e);
}
// The time of n tiles on 256 compute units, in that of one turn of 256 x 256 tiles.  A
// compute unit holds one such tile, two of 128 or three of 64; by the rates with all
// of them busy (bf16: 1,305 TFLOP/s at 256 x 256, 1,021 at 128, 706 at 64; fp32: 126 at
// 128 and 121 at 64) and, of a last turn, with fewer (one bf16 tile of 128 a unit takes 2,805 us
// where one of 256 takes 6,195).  fp32 takes no 256 x 256 tile (130 TFLOP/s): its sums
// would not fit twice.
double tile_time(Dtype dt, HeadTile t, int64_t n) {
  static const double busy[2][3][3] = {{{1.0}, {0.45, 0.64}, {0.20, 0.27, 0.347}}, {{}, {0.36, 0.516}, {0.11, 0.155, 0.202}}};
  const auto& of = busy[dt == DT_BF16 ? 0 : 1][t];
  const int held = t == TILE_256 ? 1 : t == TILE_128 ? 2 : 3;
  const int64_t turns = n / (256 * held), rest = n - turns * 256 * held;
  return (double)turns * of[held - 1] + (rest > 0 ? of[(rest - 1) / 256] : 0.0);
}
struct TileCost {
  HeadTile tile;
  double cost;
};
TileCost best_tile(Dtype dt, int64_t m, int64_t n) {
  const int first = dt == DT_BF16 ? TILE_256 : TILE_128;
  TileCost best{TILE_64, 0};
  for (int t = first; t <= TILE_64; ++t) {
    const double cost = tile_time(dt, (HeadTile)t, tiles_of(m, n, (HeadTile)t));
    if (t == first || cost < best.cost) best = TileCost{(HeadTile)t, cost};
  }
  return best;
}
// WITH_256: whether a 256 x 256 tile may be asked for here.
template <typename T, bool AK, bool BKM, int EPI, int MS, bool WITH_256 = sizeof(T) == 2>
hipError_t launch_tile(HeadTile t, const GemmParams& p, hipStream_t s) {
  constexpr bool TWO = sizeof(T) == 4;
  if constexpr (WITH_256) {
    if (t == TILE_256) return launch_gemm<T, 256, 256, 2, 4, AK, BKM, EPI, 128, 2, MS>(p, s);
  }
  if (t == TILE_128) return launch_gemm<T, 128, 128, 2, 2, AK, BKM, EPI, 128, 2, MS, TWO>(p, s);
  return launch_gemm<T, 64, 64, 2, 2, AK, BKM, EPI, 128, 3, MS, TWO>(p, s);
}

// W is read as it lies: a copy in 64 x 64 tiles, as the loss makes for its three
// contractions of every chunk, did not pay here at any length (both passes of 201,088 x
// 2,880: 4,096 rows 14.93 ms without it and 15.27 with, 8,192 31.25 and 31.61, 32,768
// 128.1 and 133.0).
// Ids [lo, hi).
GemmParams logits_product(Dtype dt, const void* W, const void* Hc, int64_t lo, int64_t hi, int64_t d, int64_t rows,
                          HeadTile t, const int* live) {
  GemmParams p{};
  p.live = live;
  p.a = Operand{(const char*)W + lo * d * (dt == DT_BF16 ? 2 : 4), d, hi - lo, d, 0};
  p.b = Operand{Hc, d, rows, d, 0};
  p.tiles_m = cdiv64(hi - lo, tile_edge(t));
  p.tiles_n = cdiv64(rows, tile_edge(t));
  p.k_tiles = cdiv64(d, dt == DT_BF16 ? 64 : 32);
  p.splits = 1;
  p.k_tiles_per_split = p.k_tiles;
  p.group_m = 4;
  p.valid_m = hi - lo;
  p.valid_n = rows;
  return p;
}

// Ids of a slice of the statistics: what one wave of a tile covers.
int slice_of(HeadTile t) { return tile_edge(t) / 2; }

}  // namespace

// Whole turns of large tiles, and the ids that would make a last turn of a few in
// smaller ones, where that pays for the second launch, taken as 5 us, 195 / d turns
// (256 rows of 201,088 x 2,880: 348 us forward in one launch, 310 in two; 1,000 of
// 50,257 x 768 89 and 78).  fp32 tiles of 64 are as good as those of 128.
HeadTiling head_logits_tiling(Dtype dt, int64_t rows, int64_t V, int64_t d) {
  const TileCost plain = best_tile(dt, V, rows);
  HeadTiling best{plain.tile, plain.tile, V};
  if (dt != DT_BF16) return best;
  double least = 0.96 * plain.cost;
  for (int t = TILE_256; t < TILE_64; ++t) {
    const int e = tile_edge((HeadTile)t);
    const int64_t tn = (rows + e - 1) / e, main = tiles_of(V, rows, (HeadTile)t) / 256 * 256 / tn * e;
    if (main == 0 || main >= V) continue;
    const TileCost rest = best_tile(dt, V - main, rows);
    const double cost = tile_time(dt, (HeadTile)t, main / e * tn) + rest.cost + 195.0 / (double)d;
    if (cost < least) {
      least = cost;
      best = HeadTiling{(HeadTile)t, rest.tile, main};
    }
  }
  return best;
}

int head_slices(const HeadTiling& t, int64_t V) {
  const int64_t a = (t.main + slice_of(t.tile) - 1) / slice_of(t.tile);
  return (int)(a + (V - t.main + slice_of(t.rest) - 1) / slice_of(t.rest));
}

hipError_t launch_head_stats(Dtype dt, const HeadTiling& t, const HeadArgs& a, const void* Hc, int64_t rows, float2* part,
                             float* part_a, int n_slices, const int* live, hipStream_t s) {
  int at = 0;  // slices before this launch's
  for (int64_t lo = 0; lo < a.V;) {
    const HeadTile tile = lo == 0 ? t.tile : t.rest;
    const int64_t hi = lo == 0 ? t.main : a.V;
    GemmParams p = logits_product(dt, a.W, Hc, lo, hi, a.d, rows, tile, live);
    p.part = part + at;
    p.part_a = part_a + at;
    p.n_slices = n_slices;
    const hipError_t e = dt == DT_BF16 ? launch_tile<__bf16, true, true, EPI_STATS, 16>(tile, p, s)
                                       : launch_tile<float, true, true, EPI_STATS, 32>(tile, p, s);
    if (e != hipSuccess) return e;
    at += (int)((hi - lo + slice_of(tile) - 1) / slice_of(tile));
    lo = hi;
  }
  return hipSuccess;
}

hipError_t launch_head_rows(Dtype dt, const HeadArgs& p, int64_t r0, int64_t rows, const float2* part,
                            const float* part_a, int n_slices, const int* pos, hipStream_t s) {
  // few rows of many slices: a workgroup of 1,024 threads a row
  const bool wide = rows < 512 && n_slices > 2048;
  const dim3 grid((unsigned)rows), block(wide ? 1024 : 256);
  if (dt == DT_BF16 && wide)
    hipLaunchKernelGGL((head_rows_kernel<__bf16, 1024>), grid, block, 0, s, p, r0, part, part_a, n_slices, pos);
  else if (dt == DT_BF16)
    hipLaunchKernelGGL((head_rows_kernel<__bf16, 256>), grid, block, 0, s, p, r0, part, part_a, n_slices, pos);
  else if (wide)
    hipLaunchKernelGGL((head_rows_kernel<float, 1024>), grid, block, 0, s, p, r0, part, part_a, n_slices, pos);
  else
    hipLaunchKernelGGL((head_rows_kernel<float, 256>), grid, block, 0, s, p, r0, part, part_a, n_slices, pos);
  return hipGetLastError();
}

hipError_t launch_head_grad(Dtype dt, const HeadGradArgs& a, const void* W, const void* Hc, int64_t r0, int64_t rows,
                            const int* vidx, const int* live, float4* coef, void* G, int64_t gblk, hipStream_t s) {
  const dim3 grid((unsigned)((rows + 3) / 4));
  const HeadTiling t = head_logits_tiling(dt, rows, a.V, a.d);
  hipError_t e;
  if (a.T != 1) {
    hipLaunchKernelGGL(head_coef_kernel, grid, dim3(256), 0, s, a, r0, rows, vidx, live, coef);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  for (int64_t lo = 0; lo < a.V;) {
    const HeadTile tile = lo == 0 ? t.tile : t.rest;
    const int64_t hi = lo == 0 ? t.main : a.V;
    GemmParams p = logits_product(dt, W, Hc, lo, hi, a.d, rows, tile, live);
    p.out = (char*)G + (lo >> 6) * 4096 * (dt == DT_BF16 ? 2 : 4);
    p.ldo = gblk;
    if (a.T == 1) {  // the epilogue reads the rows' arrays and adds the given token's share itself
      p.one = GradRow{a.ids + r0,  a.dlogp + r0, a.dentropy != nullptr ? a.dentropy + r0 : nullptr,
                      a.entropy != nullptr ? a.entropy + r0 : nullptr, a.stats + r0, a.N, a.V, lo};
      p.g_rowmap = vidx;
    } else {
      p.coef = coef;
    }
    e = dt == DT_BF16 ? launch_tile<__bf16, true, true, EPI_GRAD, 16>(tile, p, s)
                      : launch_tile<float, true, true, EPI_GRAD, 32>(tile, p, s);
    if (e != hipSuccess) return e;
    lo = hi;
  }
  if (a.T <= 1) return hipSuccess;
  if (dt == DT_BF16)
    hipLaunchKernelGGL((head_given_kernel<__bf16>), grid, dim3(256), 0, s, a, r0, rows, vidx, live, coef, (__bf16*)G, gblk);
  else
    hipLaunchKernelGGL((head_given_kernel<float>), grid, dim3(256), 0, s, a, r0, rows, vidx, live, coef, (float*)G, gblk);
  return hipGetLastError();
}

// The split of dH's reduction over V and its tile: the least of the tiles' time and
// that of the partial slabs, written and read again at 5 TB/s; runs of at least 8
// k-steps.  No tile of more rows than the copies of G reach.
HeadSplit head_dh_split(Dtype dt, int64_t rows, int64_t d, int64_t V) {
  const int64_t steps = (V + (dt == DT_BF16 ? 63 : 31)) / (dt == DT_BF16 ? 64 : 32);
  // one turn of 256 x 256 tiles over all of V at the rates above, in seconds
  const double turn = 2.0 * 65536 * 256 * (double)V / (dt == DT_BF16 ? 1305e12 : 130e12);
  const int reach = dh_tile_rows(dt, rows, V);
  HeadSplit best{TILE_64, 1};
  double least = -1;
  for (int t = dt == DT_BF16 ? TILE_256 : TILE_128; t <= TILE_64; ++t)
    for (int n = 1; n <= 32 && (n == 1 || steps / n >= 8); ++n) {
      if (tile_edge((HeadTile)t) > reach) break;
      if (dh_fit_splits(dt, V, n) != n) continue;
      const double cost = tile_time(dt, (HeadTile)t, tiles_of(rows, d, (HeadTile)t) * n) / n +
                          (double)n * (double)rows * (double)d * 8 / 5e12 / turn;
      if (least < 0 || cost < least) {
        least = cost;
        best = HeadSplit{(HeadTile)t, n};
      }
    }
  return best;
}

hipError_t launch_head_dh(Dtype dt, const HeadSplit& h, const void* G, int64_t gblk, const void* W, int64_t V, int64_t d,
                          int64_t rows, float* slab, const int* live, hipStream_t s, bool tiled) {
  if (h.tile == TILE_256) return launch_dh(dt, G, gblk, W, V, d, rows, slab, h.splits, live, s, tiled);
  GemmParams p{};
  p.live = live;
  p.a = Operand{G, 0, rows, V, gblk};  // tiled: storage row = token, column = vocabulary id
  // storage row = vocabulary id (k), column = d (n)
  p.b = tiled ? Operand{W, 0, d, V, tile_row_stride(d)} : Operand{W, d, d, V, 0};
  p.tiles_m = cdiv64(rows, tile_edge(h.tile));
  p.tiles_n = cdiv64(d, tile_edge(h.tile));
  p.k_tiles = cdiv64(V, dt == DT_BF16 ? 64 : 32);
  p.k_tiles_per_split = cdiv64(p.k_tiles, h.splits);
  p.splits = cdiv64(p.k_tiles, p.k_tiles_per_split);
  p.group_m = 4;
  p.out = slab;
  p.ldo = d;
  p.split_stride = rows * d;
  p.valid_m = rows;
  p.valid_n = d;
  if (p.splits != h.splits) return hipErrorInvalidValue;
  if (dt == DT_BF16) return launch_tile<__bf16, true, false, EPI_SLAB, 32, false>(h.tile, p, s);
  return launch_tile<float, true, false, EPI_SLAB, 32, false>(h.tile, p, s);
}

hipError_t launch_head_dw(Dtype dt, const void* G, int64_t gblk, const void* Hc, int64_t V, int64_t d, int64_t rows,
                          const float* old, float* sums, int beta, void* rounded, const int* live, hipStream_t s) {
  const HeadTile t = best_tile(dt, V, d).tile;
  if (rounded == nullptr && t == TILE_256) return launch_dw(dt, G, gblk, Hc, V, d, rows, sums, beta, live, s);
  GemmParams p{};
  p.live = live;
  p.a = Operand{G, 0, V, rows, gblk};  // tiled: storage row = token (k), column = vocabulary id (m)
  p.b = Operand{Hc, d, d, rows, 0};
  p.tiles_m = cdiv64(V, tile_edge(t));
  p.tiles_n = cdiv64(d, tile_edge(t));
  p.k_tiles = cdiv64(rows, dt == DT_BF16 ? 64 : 32);
  p.splits = 1;
  p.k_tiles_per_split = p.k_tiles;
  p.group_m = 1;
  p.out = rounded != nullptr ? rounded : (void*)sums;
  p.ldo = d;
  p.old = old;
  p.beta = beta;
  p.valid_m = V;
  p.valid_n = d;
  if (rounded != nullptr) return launch_tile<__bf16, false, false, EPI_ROUND, 32>(t, p, s);
  if (dt == DT_BF16) return launch_tile<__bf16, false, false, EPI_ACCUM, 32, false>(t, p, s);
  return launch_tile<float, false, false, EPI_ACCUM, 32, false>(t, p, s);
}

}  // namespace ckl
