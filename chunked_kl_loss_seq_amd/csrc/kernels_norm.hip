// The residual's norms around a block, and dropout.
//
//   u  = w_post y / rms(y)             rms(v) = sqrt(mean v^2 + eps); u = y without w_post
//   r' = r + s m gate u                m = 0 or 1 / (1 - p) per element (Philox, never stored)
//   x  = w_pre r' / rms(r')            from the fp32 r', not from its rounded copy
//
// With n1 = y / rms(y), n2 = r' / rms(r'), f = s m, a = dx w_pre:
//   D      = dr' + (a - n2 mean(a n2)) / rms(r')           = dr
//   dw_pre = sum_rows dx n2       dgate = f D u  (summed over rows for a gate [d])
//   dw_post = sum_rows f gate D n1
//   dy     = (e - n1 mean(e n1)) / rms(y),  e = f gate w_post D
// The second mean needs D, which needs the first; but with q = f gate w_post n1
//   sum e n1 = sum q (dr' + a / rms(r')) - (mean(a n2) / rms(r')) sum q n2,
// so one round of three sums serves a row.
#include <hip/hip_runtime.h>

#include "row_io.hpp"

namespace ckl {

namespace {

// ------------------------------------------------------------------ dropout
constexpr int kDropThreads = 256;
constexpr int kDropGroups = 4;  // groups of eight elements per thread

template <typename T>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const T* __restrict__ x, int64_t n, Drop r,
                                                              T* __restrict__ out) {
  const uint64_t offset = drop_offset(r);
  const int64_t g0 = (int64_t)blockIdx.x * (kDropThreads * kDropGroups) + threadIdx.x;
  Eight<T> v[kDropGroups];
#pragma unroll
  for (int u = 0; u < kDropGroups; ++u) {
    const int64_t i = (g0 + u * kDropThreads) * 8;
    if (i + 8 <= n) v[u].load(x + i);
  }
#pragma unroll
  for (int u = 0; u < kDropGroups; ++u) {
    const int64_t g = g0 + u * kDropThreads, i = g * 8;
    if (i >= n) return;
    const row_u32x4 w = philox((uint64_t)g, offset, r.seed);
    if (i + 8 <= n) {
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = bits16(w, e) >= r.border ? v[u].get(e) * r.keep : 0.f;
      v[u].set(f);
      v[u].store(out + i);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i + e < n) out[i + e] = bits16(w, e) >= r.border ? (T)((float)x[i + e] * r.keep) : (T)0.f;
    }
  }
}

// ------------------------------------------------------------------ norms
// A row goes to a team of `lanes` lanes of one wave (a power of two that covers
// d / 8, several rows a wave for short rows), or to all waves of a workgroup;
// lane t holds elements 8 (t + i team) .. + 7, i < NV, in registers, so a row is
// read once.  Workgroups walk over rows, and in the backward pass each keeps its
// columns' sums in registers until its last row.
struct Team {
  int lanes;   // lanes of one row within a wave
  int teams;   // rows side by side in a wave (64 / lanes; 1 for several waves)
  int waves;   // waves of a workgroup
};

__device__ inline float team_sum(float v, const Team& t, float* red, int slot) {
  v = lanes_sum(v, t.lanes);
  if (t.waves == 1) return v;
  if ((threadIdx.x & 63) == 0) red[slot * 16 + (threadIdx.x >> 6)] = v;
  return v;
}

// Sums of K values over the team, in every lane.  `red` alternates between two
// halves from one call to the next, so one barrier a call is enough.
template <int K>
__device__ inline void team_sums(float (&v)[K], const Team& t, float* red, int& half) {
  float* to = red + half * (K * 16);
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = team_sum(v[k], t, to, k);
  if (t.waves == 1) return;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float s = 0.f;
    for (int w = 0; w < t.waves; ++w) s += to[k * 16 + w];
    v[k] = s;
  }
  half ^= 1;
}

template <typename T, int NV, int MT>
__global__ void __launch_bounds__(MT) add_norm_kernel(NormArgs p, Team team) {
  __shared__ float red[2 * 16];
  int half = 0;
  const int lane = threadIdx.x & 63;
  const int t = team.waves > 1 ? threadIdx.x : lane & (team.lanes - 1);
  const int width = team.waves > 1 ? team.waves * 64 : team.lanes;
  const int sub = team.waves > 1 ? 0 : lane / team.lanes;
  const int d8 = (int)(p.d >> 3);
  const uint64_t offset = p.drop.border ? drop_offset(p.drop) : 0;
  const T* w1 = (const T*)p.w_post;
  const T* w2 = (const T*)p.w_pre;
  const T* gate = (const T*)p.gate;
  const float inv_d = 1.f / (float)p.d;
  const int64_t step = (int64_t)gridDim.x * team.teams;
  // every lane of a workgroup makes the same number of turns: the sums cross lanes
  for (int64_t row0 = (int64_t)blockIdx.x * team.teams; row0 < p.N; row0 += step) {
    const int64_t row = row0 + sub;
    const bool live = row < p.N;
    const int64_t base = row * p.d;
    Eight<T> y[NV], r[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t + i * width;
      if (live && c < d8) {
        y[i].load((const T*)p.y + base + 8 * c);
        r[i].load((const T*)p.r + base + 8 * c);
      }
    }
    float inv1 = 1.f;
    if (w1 != nullptr) {
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = t + i * width;
        if (live && c < d8) {
#pragma unroll
          for (int e = 0; e < 8; ++e) s[0] = __builtin_fmaf(y[i].get(e), y[i].get(e), s[0]);
        }
      }
      team_sums(s, team, red, half);
      inv1 = 1.f / sqrtf(s[0] * inv_d + p.eps);
    }
    float o[NV][8];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t + i * width;
      if (!live || c >= d8) continue;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = p.scale;
      if (p.drop.border) {
        const row_u32x4 w = philox((uint64_t)(base >> 3) + (uint64_t)c, offset, p.drop.seed);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = bits16(w, e) >= p.drop.border ? p.scale * p.drop.keep : 0.f;
      }
      if (gate != nullptr) {
        Eight<T> g;
        g.load(gate + (p.gate_rows ? base : 0) + 8 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= g.get(e);
      }
      if (w1 != nullptr) {
        Eight<T> w;
        w.load(w1 + 8 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= w.get(e) * inv1;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        o[i][e] = __builtin_fmaf(f[e], y[i].get(e), r[i].get(e));
        s[0] = __builtin_fmaf(o[i][e], o[i][e], s[0]);
      }
      Eight<T> v;
      v.set(o[i]);
      v.store((T*)p.r_out + base + 8 * c);
    }
    float inv2 = 1.f;
    if (w2 != nullptr) {
      team_sums(s, team, red, half);
      inv2 = 1.f / sqrtf(s[0] * inv_d + p.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = t + i * width;
        if (!live || c >= d8) continue;
        Eight<T> w;
        w.load(w2 + 8 * c);
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = o[i][e] * inv2 * w.get(e);
        w.set(f);
        w.store((T*)p.x + base + 8 * c);
      }
    }
    if (p.stats != nullptr && live && t == 0) {
      p.stats[row] = inv1;
      p.stats[p.N + row] = inv2;
    }
  }
}

// Columns' sums of a workgroup's rows: part[block][which][d], which = dw_post,
// dw_pre, dgate as far as they are asked for.
template <typename T, int NV, int MT>
__global__ void __launch_bounds__(MT) add_norm_bwd_kernel(NormArgs p, NormGrads q, Team team) {
  __shared__ float red[2 * 3 * 16];
  int half = 0;
  const int lane = threadIdx.x & 63;
  const int t = team.waves > 1 ? threadIdx.x : lane & (team.lanes - 1);
  const int width = team.waves > 1 ? team.waves * 64 : team.lanes;
  const int sub = team.waves > 1 ? 0 : lane / team.lanes;
  const int d8 = (int)(p.d >> 3);
  const uint64_t offset = p.drop.border ? drop_offset(p.drop) : 0;
  const T* w1 = (const T*)p.w_post;
  const T* w2 = (const T*)p.w_pre;
  const T* gate = (const T*)p.gate;
  const float factor = p.drop.border ? p.scale * p.drop.keep : p.scale;
  const float inv_d = 1.f / (float)p.d;
  float aw1[NV][8], aw2[NV][8], ag[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) aw1[i][e] = aw2[i][e] = ag[i][e] = 0.f;
  const int64_t step = (int64_t)gridDim.x * team.teams;
  for (int64_t row0 = (int64_t)blockIdx.x * team.teams; row0 < p.N; row0 += step) {
    const int64_t row = row0 + sub;
    const bool live = row < p.N;
    const int64_t base = row * p.d;
    const float inv1 = live && w1 != nullptr ? p.stats_in[row] : 1.f;
    const float inv2 = live && w2 != nullptr ? p.stats_in[p.N + row] : 1.f;
    // per element: h = f gate, n1, n2 and the gradients
    float n1[NV][8], n2[NV][8], a[NV][8], D[NV][8];
    uint32_t kept[NV];  // bit e: element e of the vector is kept
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t + i * width;
      if (!live || c >= d8) continue;
      Eight<T> v;
      v.load((const T*)p.y + base + 8 * c);
#pragma unroll
      for (int e = 0; e < 8; ++e) n1[i][e] = v.get(e) * inv1;
      float f[8];
      kept[i] = 0xFFu;
      if (p.drop.border) {
        const row_u32x4 w = philox((uint64_t)(base >> 3) + (uint64_t)c, offset, p.drop.seed);
        kept[i] = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) kept[i] |= (bits16(w, e) >= p.drop.border ? 1u : 0u) << e;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = (kept[i] >> e) & 1u ? factor : 0.f;
      if (gate != nullptr) {
        v.load(gate + (p.gate_rows ? base : 0) + 8 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= v.get(e);
      }
      if (w1 != nullptr) {
        v.load(w1 + 8 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= v.get(e);
      }
      // f n1 = f gate u: the branch's share of r'
      v.load((const T*)p.r + base + 8 * c);
#pragma unroll
      for (int e = 0; e < 8; ++e) n2[i][e] = __builtin_fmaf(f[e], n1[i][e], v.get(e)) * inv2;
#pragma unroll
      for (int e = 0; e < 8; ++e) D[i][e] = 0.f;
      if (q.dr_in != nullptr) {
        v.load((const T*)q.dr_in + base + 8 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) D[i][e] = v.get(e);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) a[i][e] = 0.f;
      if (q.dx != nullptr) {
        v.load((const T*)q.dx + base + 8 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a[i][e] = v.get(e);
          aw2[i][e] = __builtin_fmaf(a[i][e], n2[i][e], aw2[i][e]);
        }
        v.load(w2 + 8 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[i][e] *= v.get(e);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float b = f[e] * n1[i][e];
        D[i][e] = __builtin_fmaf(a[i][e], inv2, D[i][e]);
        s[0] = __builtin_fmaf(a[i][e], n2[i][e], s[0]);
        s[1] = __builtin_fmaf(b, D[i][e], s[1]);
        s[2] = __builtin_fmaf(b, n2[i][e], s[2]);
      }
    }
    team_sums(s, team, red, half);
    const float c2 = s[0] * inv_d * inv2;              // mean(a n2) / rms(r')
    const float c1 = w1 != nullptr ? (s[1] - c2 * s[2]) * inv_d : 0.f;  // mean(e n1)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = t + i * width;
      if (!live || c >= d8) continue;
      Eight<T> v;
#pragma unroll
      for (int e = 0; e < 8; ++e) D[i][e] -= n2[i][e] * c2;
      v.set(D[i]);
      v.store((T*)q.dr + base + 8 * c);
      float f[8], o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = (kept[i] >> e) & 1u ? factor : 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= D[i][e];
      float wp[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) wp[e] = 1.f;
      if (w1 != nullptr) {
        v.load(w1 + 8 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) wp[e] = v.get(e);
      }
      if (gate != nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = f[e] * n1[i][e] * wp[e];
        if (p.gate_rows) {
          v.set(o);
          v.store((T*)q.dgate + base + 8 * c);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) ag[i][e] += o[e];
        }
        v.load(gate + (p.gate_rows ? base : 0) + 8 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= v.get(e);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        aw1[i][e] = __builtin_fmaf(f[e], n1[i][e], aw1[i][e]);
        o[e] = (f[e] * wp[e] - n1[i][e] * c1) * inv1;
      }
      v.set(o);
      v.store((T*)q.dy + base + 8 * c);
    }
  }
  // rows side by side in the wave hold the same columns
  if (team.teams > 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        for (int o = 32; o >= team.lanes; o >>= 1) {
          aw1[i][e] += __shfl_xor(aw1[i][e], o);
          aw2[i][e] += __shfl_xor(aw2[i][e], o);
          ag[i][e] += __shfl_xor(ag[i][e], o);
        }
    if (sub != 0) return;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = t + i * width;
    if (c >= d8) continue;
    float* to = q.part + (int64_t)blockIdx.x * q.sums * p.d + 8 * c;
    if (w1 != nullptr) {
#pragma unroll
      for (int e = 0; e < 8; ++e) to[e] = aw1[i][e];
      to += p.d;
    }
    if (w2 != nullptr) {
#pragma unroll
      for (int e = 0; e < 8; ++e) to[e] = aw2[i][e];
      to += p.d;
    }
    if (gate != nullptr && !p.gate_rows) {
#pragma unroll
      for (int e = 0; e < 8; ++e) to[e] = ag[i][e];
    }
  }
}

// out[c] = the sum of part[b][c] over the workgroups b, in a fixed order: 64
// columns a workgroup, 16 threads a column.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* __restrict__ part, int rows, int64_t cols,
                                                         int64_t d, float* o0, float* o1, float* o2) {
  __shared__ float red[16][64];
  const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + x;
  float s = 0.f;
  if (c < cols)
    for (int b = y; b < rows; b += 16) s += part[(int64_t)b * cols + c];
  red[y][x] = s;
  __syncthreads();
  if (y != 0 || c >= cols) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) s += red[i][x];
  float* o = c < d ? o0 : c < 2 * d ? o1 : o2;
  o[c % d] = s;
}

// Lanes, rows a wave and waves for rows of d elements with up to `most` vectors
// a lane, and how many are used.  Workgroups are held to 512 threads, so that a
// lane can have 256 registers; rows of more than 8 x 64 x 8 x 3 elements take
// up to 1024 threads with two vectors each.
constexpr int kNormVec = 3;
struct Shape {
  Team team;
  int nv;
};
Shape shape_of(int64_t d) {
  const int64_t d8 = d / 8;
  Shape r{{64, 1, 1}, 1};
  if (d8 <= 64) {
    while (r.team.lanes > 1 && r.team.lanes / 2 >= d8) r.team.lanes /= 2;
    r.team.teams = 64 / r.team.lanes;
    return r;
  }
  int most = kNormVec;
  if (d8 > 8 * 64 * most) most = 2;
  r.team.waves = (int)((d8 + 64 * most - 1) / (64 * most));
  r.nv = (int)((d8 + 64 * r.team.waves - 1) / (64 * r.team.waves));
  return r;
}

// Workgroups of the backward pass, each with its partial sums.
int bwd_blocks(int64_t N, const Team& t) {
  const int64_t need = (N + t.teams - 1) / t.teams;
  const int64_t most = t.waves == 1 ? 2048 : t.waves == 2 ? 1024 : 512;
  return (int)(need < most ? need : most);
}

template <typename T>
hipError_t add_norm_of(const NormArgs& p, hipStream_t s) {
  const Shape h = shape_of(p.d);
  const int64_t need = (p.N + h.team.teams - 1) / h.team.teams;
  const int64_t most = 256 * 32 / h.team.waves;
  const dim3 grid((unsigned)(need < most ? need : most)), block(64 * h.team.waves);
  if (block.x > 512)
    hipLaunchKernelGGL((add_norm_kernel<T, 2, 1024>), grid, block, 0, s, p, h.team);
  else if (h.nv == 1)
    hipLaunchKernelGGL((add_norm_kernel<T, 1, 512>), grid, block, 0, s, p, h.team);
  else if (h.nv == 2)
    hipLaunchKernelGGL((add_norm_kernel<T, 2, 512>), grid, block, 0, s, p, h.team);
  else
    hipLaunchKernelGGL((add_norm_kernel<T, 3, 512>), grid, block, 0, s, p, h.team);
  return hipGetLastError();
}

template <typename T>
hipError_t add_norm_bwd_of(const NormArgs& p, const NormGrads& q, hipStream_t s) {
  const Shape h = shape_of(p.d);
  const int blocks = bwd_blocks(p.N, h.team);
  const dim3 grid(blocks), block(64 * h.team.waves);
  if (block.x > 512)
    hipLaunchKernelGGL((add_norm_bwd_kernel<T, 2, 1024>), grid, block, 0, s, p, q, h.team);
  else if (h.nv == 1)
    hipLaunchKernelGGL((add_norm_bwd_kernel<T, 1, 512>), grid, block, 0, s, p, q, h.team);
  else if (h.nv == 2)
    hipLaunchKernelGGL((add_norm_bwd_kernel<T, 2, 512>), grid, block, 0, s, p, q, h.team);
  else
    hipLaunchKernelGGL((add_norm_bwd_kernel<T, 3, 512>), grid, block, 0, s, p, q, h.team);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || q.sums == 0) return e;
  float* outs[3] = {nullptr, nullptr, nullptr};
  int n = 0;
  if (p.w_post != nullptr) outs[n++] = q.dw_post;
  if (p.w_pre != nullptr) outs[n++] = q.dw_pre;
  if (p.gate != nullptr && !p.gate_rows) outs[n++] = (float*)q.dgate;
  const int64_t cols = q.sums * p.d;
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((cols + 63) / 64)), dim3(1024), 0, s, q.part, blocks, cols, p.d,
                     outs[0], outs[1], outs[2]);
  return hipGetLastError();
}

}  // namespace

int64_t dropout_blocks(int64_t n) {
  const int64_t per = (int64_t)kDropThreads * kDropGroups * 8;
  return (n + per - 1) / per;
}

hipError_t launch_dropout(Dtype dt, const void* x, int64_t n, const Drop& r, void* out, hipStream_t s) {
  const dim3 grid((unsigned)dropout_blocks(n)), block(kDropThreads);
  if (dt == DT_BF16)
    hipLaunchKernelGGL((dropout_kernel<__bf16>), grid, block, 0, s, (const __bf16*)x, n, r, (__bf16*)out);
  else
    hipLaunchKernelGGL((dropout_kernel<float>), grid, block, 0, s, (const float*)x, n, r, (float*)out);
  return hipGetLastError();
}

hipError_t launch_add_norm(Dtype dt, const NormArgs& p, hipStream_t s) {
  return dt == DT_BF16 ? add_norm_of<__bf16>(p, s) : add_norm_of<float>(p, s);
}

uint64_t add_norm_bwd_workspace(int64_t N, int64_t d, int sums) {
  return N > 0 ? (uint64_t)bwd_blocks(N, shape_of(d).team) * (uint64_t)sums * (uint64_t)d * 4 : 0;
}

hipError_t launch_add_norm_bwd(Dtype dt, const NormArgs& p, const NormGrads& q, hipStream_t s) {
  return dt == DT_BF16 ? add_norm_bwd_of<__bf16>(p, q, s) : add_norm_bwd_of<float>(p, q, s);
}

}  // namespace ckl
