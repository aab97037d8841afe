// Log-probabilities of given tokens and entropy from hidden states and the head's
// weight, without N x V logits, and their gradients.
//
// Forward: the logits contraction of a chunk of rows keeps, of every 128-id
// slice of a row, its largest logit m_s, sum exp(z - m_s) and
// sum exp(z - m_s) (z - m_s), and nothing else; a merge of the slices gives the
// row's statistics.  The given tokens' logits are T dot products a row
// (T d products beside the contraction's V d).
//
// Backward: the contraction runs again and its epilogue turns logits into the
// gradient's dense part G_j = -p_j (w + u (log p_j + entropy)), w the sum of the
// row's given weights; the given tokens' own elements are then written from their
// log-probabilities, and dH = G W, dW = G^T H follow as in the loss.
#include <math.h>

#include "gemm_core.hpp"
#include "row_io.hpp"

namespace ckl {

namespace {

constexpr float kFar = -1000.f;  // exp(kFar) is 0 in fp32

// One wave per (row, given token): z = H_n . W_id in fp32, kept in logp until the
// row's statistics are known.
template <typename T>
__global__ void __launch_bounds__(256) given_logits_kernel(HeadArgs p) {
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (i >= p.N * p.T) return;
  const int lane = threadIdx.x & 63;
  const int64_t n = i / p.T;
  const int32_t id = p.ids[i];
  if (id < 0 || id >= p.V || (p.mask != nullptr && p.mask[n] == 0)) return;
  const T* h = (const T*)p.H + n * p.d;
  const T* w = (const T*)p.W + (int64_t)id * p.d;
  float s = 0.f;
  for (int64_t k = 8 * lane; k < p.d; k += 512) {
    Eight<T> a, b;
    a.load(h + k);
    b.load(w + k);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = __builtin_fmaf(a.get(e), b.get(e), s);
  }
  s = lanes_sum(s, 64);
  if (lane == 0) p.logp[i] = s;
}

// Rows [r0, r0 + rows) of the call: the slices' statistics to the rows'.  With a
// compacted chunk, pos gives each row's place in it, -1 for a masked one.
__global__ void __launch_bounds__(256) head_rows_kernel(HeadArgs p, int64_t r0, const float2* __restrict__ part,
                                                       const float* __restrict__ part_a, int n_slices,
                                                       const int* __restrict__ pos) {
  __shared__ float red[12];
  const int64_t row = r0 + blockIdx.x;
  const int t = threadIdx.x, w = t >> 6;
  const int64_t at = pos != nullptr ? pos[blockIdx.x] : (int64_t)blockIdx.x;
  if (at < 0) {
    for (int i = t; i < p.T; i += 256) p.logp[row * p.T + i] = 0.f;
    if (t == 0) p.entropy[row] = p.stats[row] = p.stats[p.N + row] = 0.f;
    return;
  }
  const float2* q = part + at * n_slices;
  const float* qa = part_a + at * n_slices;
  float M = -INFINITY;
  for (int i = t; i < n_slices; i += 256) M = fmaxf(M, q[i].x);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor(M, o));
  if ((t & 63) == 0) red[w] = M;
  __syncthreads();
  M = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  float s = 0.f, a = 0.f;
  for (int i = t; i < n_slices; i += 256) {
    const float2 v = q[i];
    const float dm = fmaxf(v.x - M, kFar), k = __expf(dm);
    s = __builtin_fmaf(v.y, k, s);
    a = __builtin_fmaf(__builtin_fmaf(v.y, dm, qa[i]), k, a);
  }
  s = lanes_sum(s, 64);
  a = lanes_sum(a, 64);
  if ((t & 63) == 0) {
    red[4 + w] = s;
    red[8 + w] = a;
  }
  __syncthreads();
  s = (red[4] + red[5]) + (red[6] + red[7]);
  a = (red[8] + red[9]) + (red[10] + red[11]);
  const float logs = logf(s), h = logs - a / s;
  for (int i = t; i < p.T; i += 256) {
    const int32_t id = p.ids[row * p.T + i];
    float* l = p.logp + row * p.T + i;
    *l = id >= 0 && id < p.V ? (*l - M) - logs : 0.f;
  }
  if (t == 0) {
    p.entropy[row] = h < 0.f ? 0.f : h;
    p.stats[row] = M;
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

GemmParams logits_product(Dtype dt, const void* W, bool tiled, const void* Hc, int64_t V, int64_t d, int64_t rows,
                          const int* live) {
  GemmParams p{};
  p.live = live;
  p.a = tiled ? Operand{W, 0, V, d, tile_row_stride(d)} : Operand{W, d, V, d, 0};
  p.b = Operand{Hc, d, rows, d, 0};
  p.tiles_m = cdiv64(V, 256);
  p.tiles_n = cdiv64(rows, 256);
  p.k_tiles = cdiv64(d, dt == DT_BF16 ? 64 : 32);
  p.splits = 1;
  p.k_tiles_per_split = p.k_tiles;
  p.group_m = 4;
  p.valid_m = V;
  p.valid_n = rows;
  return p;
}

}  // namespace

hipError_t launch_given_logits(Dtype dt, const HeadArgs& p, hipStream_t s) {
  const dim3 grid((unsigned)((p.N * p.T + 3) / 4));
  if (dt == DT_BF16)
    hipLaunchKernelGGL((given_logits_kernel<__bf16>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((given_logits_kernel<float>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

hipError_t launch_head_stats(Dtype dt, const HeadArgs& a, const void* Hc, int64_t rows, float2* part, float* part_a,
                             int n_slices, const int* live, hipStream_t s) {
  GemmParams p = logits_product(dt, a.W, false, Hc, a.V, a.d, rows, live);
  p.part = part;
  p.part_a = part_a;
  p.n_slices = n_slices;
  if (dt == DT_BF16) return launch_gemm<__bf16, 256, 256, 2, 4, true, true, EPI_STATS, 128, 2, 16>(p, s);
  return launch_gemm<float, 256, 256, 2, 4, true, true, EPI_STATS, 128, 2>(p, s);
}

hipError_t launch_head_rows(const HeadArgs& p, int64_t r0, int64_t rows, const float2* part, const float* part_a,
                            int n_slices, const int* pos, hipStream_t s) {
  hipLaunchKernelGGL(head_rows_kernel, dim3((unsigned)rows), dim3(256), 0, s, p, r0, part, part_a, n_slices, pos);
  return hipGetLastError();
}

hipError_t launch_head_grad(Dtype dt, const HeadGradArgs& a, const void* W, bool tiled, const void* Hc, int64_t r0,
                            int64_t rows, const int* vidx, const int* live, float4* coef, void* G, int64_t gblk,
                            hipStream_t s) {
  const dim3 grid((unsigned)((rows + 3) / 4));
  hipLaunchKernelGGL(head_coef_kernel, grid, dim3(256), 0, s, a, r0, rows, vidx, live, coef);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  GemmParams p = logits_product(dt, W, tiled, Hc, a.V, a.d, rows, live);
  p.coef = coef;
  p.out = G;
  p.ldo = gblk;
  e = dt == DT_BF16 ? launch_gemm<__bf16, 256, 256, 2, 4, true, true, EPI_GRAD, 128, 2, 16>(p, s)
                    : launch_gemm<float, 256, 256, 2, 4, true, true, EPI_GRAD, 128, 2>(p, s);
  if (e != hipSuccess || a.T == 0) return e;
  if (dt == DT_BF16)
    hipLaunchKernelGGL((head_given_kernel<__bf16>), grid, dim3(256), 0, s, a, r0, rows, vidx, live, coef, (__bf16*)G, gblk);
  else
    hipLaunchKernelGGL((head_given_kernel<float>), grid, dim3(256), 0, s, a, r0, rows, vidx, live, coef, (float*)G, gblk);
  return hipGetLastError();
}

hipError_t launch_dw_round(const void* G, int64_t gblk, const void* Hc, int64_t V, int64_t d, int64_t rows,
                           const float* old, void* dW, const int* live, hipStream_t s) {
  GemmParams p{};
  p.live = live;
  p.a = Operand{G, 0, V, rows, gblk};  // tiled: storage row = token (k), column = vocabulary id (m)
  p.b = Operand{Hc, d, d, rows, 0};
  p.tiles_m = cdiv64(V, 256);
  p.tiles_n = cdiv64(d, 256);
  p.k_tiles = cdiv64(rows, 64);
  p.splits = 1;
  p.k_tiles_per_split = p.k_tiles;
  p.group_m = 1;
  p.out = dW;
  p.ldo = d;
  p.old = old;
  p.valid_m = V;
  p.valid_n = d;
  return launch_gemm<__bf16, 256, 256, 2, 4, false, false, EPI_ROUND, 128, 2>(p, s);
}

}  // namespace ckl
