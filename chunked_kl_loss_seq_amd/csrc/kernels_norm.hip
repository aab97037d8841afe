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
//
// Bound by HBM: forward two arrays read and two written, backward four and two.  The
// numbers' generator (about 30 us of vector instructions for 94 M elements) hides
// behind them.
// Measured (MI355X, bf16): 32,768 x 2,880 with both weights, a gate [d] and p = 0.1:
// forward 141 us (5.3 TB/s), backward 237 us (4.8 TB/s), of which the sums of columns
// take 5.  8,192 x 8,192 backward 162 us (5.0 TB/s).  One row of 2,880: 3.7 us.
// dropout of 94 M bf16 elements 67 us (5.6 TB/s).
// Rows wider than 8,192 are far from that backward (4,096 x 12,288: 260 us, 117 at the
// copy's rate): 1,024 threads hold two vectors each, which do not fit 128 registers, and
// 144 to 208 bytes a lane go to scratch (fp32 170 to 300).  Besides those only fp32 with a
// gate of [N, d] spills: backward from 4,104 columns 20 to 36 bytes, forward above 8,192
// 68 to 96 (4,096 x 12,288 with dropout 244 us).
// What carried it: loads of the next row under way for a whole turn (a select right
// after each load had made every load wait for the one before), a barrier for LDS
// alone (the ordinary one waits for all loads), the columns' weights in LDS instead
// of registers, as many workgroups as fit at once, sums over lanes in registers.
#include <hip/hip_runtime.h>

#include "row_io.hpp"

namespace ckl {

namespace {

// ------------------------------------------------------------------ dropout
constexpr int kDropThreads = 256;
constexpr int kDropGroups = 4;  // groups of eight elements per thread

template <typename T>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const T* x, int64_t n, Drop r, T* out) {  // out may be x
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
// A row goes to a team: `lanes` lanes of one wave (a power of two that covers
// d / 8; several rows a wave for short rows), or all waves of a workgroup.  Lane
// t of it holds elements 8 (t + i width) .. + 7, i < NV, in registers, so a row is
// read once; the weights of its columns are in LDS, for all rows of a workgroup.
// Workgroups walk over rows, and the next row's loads are issued before the current
// row's sums are joined (not in the backward pass of rows above 8,192, which has no
// registers for them).
struct Team {
  int lanes;   // lanes of one row within a wave
  int rows;    // rows side by side in a workgroup
  int span;    // waves of one row (1, or all of the workgroup's)
};

// Where a thread stands in its team.
struct Place {
  int t, width, sub;  // lane of the team, its lanes, the team's number in the workgroup
  __device__ inline Place(const Team& m) {
    if (m.span > 1) {
      t = threadIdx.x;
      width = blockDim.x;
      sub = 0;
    } else {
      t = threadIdx.x & (m.lanes - 1);
      width = m.lanes;
      sub = threadIdx.x / m.lanes;
    }
  }
};

// Sums of K values over the team, in every lane.  `red` alternates between two
// halves from one call to the next, so one barrier a call is enough.
template <int K>
__device__ inline void team_sums(float (&v)[K], const Team& m, float* red, int& half) {
  if (m.span == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = lanes_sum(v[k], m.lanes);
    return;
  }
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lanes_sum(v[k], 64);
  float* to = red + half * (K * 16);
  if ((threadIdx.x & 63) == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) to[k * 16 + (threadIdx.x >> 6)] = v[k];
  }
  lds_barrier();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float s = 0.f;
    for (int w = 0; w < m.span; ++w) s += to[k * 16 + w];
    v[k] = s;
  }
  half ^= 1;
}

// One vector of an array at byte `off` from the first of the workgroup's rows, if
// the array is there.  Nothing is done with it here, so that all of a row's loads
// are under way together: lanes without a column read the first ones, and are
// zeroed when the row's turn comes.  One 32-bit offset a vector serves all arrays.
template <typename T>
__device__ inline void load_at(Eight<T>& v, const void* rows, uint32_t off) {
  if (rows != nullptr) v.load((const T*)((const char*)rows + off));
}
template <typename T>
__device__ inline const void* rows_of(const void* x, int64_t row, int64_t d) {
  return x != nullptr ? (const T*)x + row * d : nullptr;
}
template <typename T>
__device__ inline T* row_at(void* x, int64_t row, int64_t d, uint32_t off) {
  return (T*)((char*)((T*)x + row * d) + off);
}
// The byte offset of vector c of this team's row, of rows row0 .. (a team past the
// last row takes the last one, and stores nothing).
template <typename T>
__device__ inline uint32_t offset_of(int64_t row0, int64_t N, int sub, uint32_t d, int c, bool in) {
  const uint32_t at = row0 + sub < N ? (uint32_t)sub : (uint32_t)(N - 1 - row0);
  return (at * d + (in ? 8u * (uint32_t)c : 0u)) * (uint32_t)sizeof(T);
}

// The columns' weights, in LDS for all rows of a workgroup (in registers they would
// halve the waves that a compute unit holds): `f`, the scale (and the kept ones'
// factor) x w_post x a gate [d], then `w2`, w_pre or zeros.  The two halves of a
// vector of 8 lie d / 2 apart, so that lanes read 16 adjacent bytes each.
__device__ inline float* half_at(float* w, int d, int c, int h) { return w + h * (d >> 1) + 4 * c; }
__device__ inline void read8(float* w, int d, int c, float (&v)[8]) {
  const row_f32x4 a = *(const row_f32x4*)half_at(w, d, c, 0), b = *(const row_f32x4*)half_at(w, d, c, 1);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = a[e];
    v[4 + e] = b[e];
  }
}
template <typename T, bool ROWS>
__device__ inline void column_weights(const NormArgs& p, float* f, float* w2) {
  const float k = p.drop.border ? p.scale * p.drop.keep : p.scale;
  const int d = (int)p.d, d8 = d >> 3;
  const bool gated = !ROWS && p.gate != nullptr;
  for (int c = threadIdx.x; c < d8; c += blockDim.x) {
    Eight<T> a, g, b;
    if (p.w_post != nullptr) a.load((const T*)p.w_post + 8 * c);
    if (gated) g.load((const T*)p.gate + 8 * c);
    b.clear();
    if (p.w_pre != nullptr) b.load((const T*)p.w_pre + 8 * c);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      row_f32x4 v, w;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = k;
        if (p.w_post != nullptr) v[j] *= a.get(4 * h + j);
        if (gated) v[j] *= g.get(4 * h + j);
        w[j] = b.get(4 * h + j);
      }
      *(row_f32x4*)half_at(f, d, c, h) = v;
      *(row_f32x4*)half_at(w2, d, c, h) = w;
    }
  }
  __syncthreads();
}

// Bit e: element e of the vector at element index 8 g is kept.
__device__ inline uint32_t kept_bits(const Drop& r, uint64_t offset, uint64_t g) {
  const row_u32x4 w = philox(g, offset, r.seed);
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m |= (bits16(w, e) >= r.border ? 1u : 0u) << e;
  return m;
}

// Waves a SIMD: what the registers are held to, and what the grids count on.
template <typename T, int NV, int MT, bool ROWS>
constexpr int fwd_waves() {
  if (MT > 512) return 4;
  return sizeof(T) == 2 ? (NV == 1 ? (ROWS ? 6 : 7) : 4) : (NV == 1 ? (ROWS ? 5 : 6) : (ROWS ? 3 : 4));
}
template <typename T, int MT>
constexpr int bwd_waves() {
  return MT > 512 || sizeof(T) == 2 ? 4 : 3;
}

template <typename T, int NV, int MT, bool ROWS, bool DROP>
__global__ void __launch_bounds__(MT) __attribute__((amdgpu_waves_per_eu(fwd_waves<T, NV, MT, ROWS>())))
add_norm_kernel(NormArgs p, Team team) {
  __shared__ float red[2 * 16];
  int half = 0;
  const Place at(team);
  const int d8 = (int)(p.d >> 3);
  const uint64_t offset = DROP ? drop_offset(p.drop) : 0;
  const float inv_d = 1.f / (float)p.d;
  extern __shared__ float columns[];
  float *f = columns, *w2 = columns + p.d;
  Eight<T> y[NV], r[NV], g[ROWS ? NV : 1];
  const auto fetch = [&](int64_t row0) {
    const void *ys = rows_of<T>(p.y, row0, p.d), *rs = rows_of<T>(p.r, row0, p.d);
    const void* gs = ROWS ? rows_of<T>(p.gate, row0, p.d) : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at.t + i * at.width;
      const uint32_t off = offset_of<T>(row0, p.N, at.sub, (uint32_t)p.d, c, c < d8);
      y[i].load((const T*)((const char*)ys + off));
      r[i].load((const T*)((const char*)rs + off));
      if constexpr (ROWS) g[i].load((const T*)((const char*)gs + off));
    }
  };
  const int64_t step = (int64_t)gridDim.x * team.rows;
  fetch((int64_t)blockIdx.x * team.rows);
  column_weights<T, ROWS>(p, f, w2);
  // every lane of a workgroup makes the same number of turns: the sums cross lanes
  for (int64_t row0 = (int64_t)blockIdx.x * team.rows; row0 < p.N; row0 += step) {
    const bool live = row0 + at.sub < p.N;
    const uint64_t group0 = (uint64_t)row0 * (uint64_t)d8 + (uint64_t)(uint32_t)(at.sub * d8);
    float b[NV][8], o[NV][8];  // the branch before its norm, then r'
    float s[1] = {0.f};
    uint32_t all = 0;  // the kept ones of all vectors, none past the row's end
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint32_t kept = 0xFFu;
      if constexpr (DROP) {
        kept = kept_bits(p.drop, offset, group0 + (uint32_t)(at.t + i * at.width));
        all |= (at.t + i * at.width < d8 ? kept : 0u) << (8 * i);
      }
      const int c = at.t + i * at.width;
      if (c >= d8) {
        y[i].clear();
        r[i].clear();
        if constexpr (ROWS) g[i].clear();
      }
      float k[8];
      read8(f, (int)p.d, c < d8 ? c : 0, k);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = y[i].get(e);
        s[0] = __builtin_fmaf(v, v, s[0]);
        b[i][e] = DROP && !((kept >> e) & 1u) ? 0.f : ROWS ? k[e] * g[i].get(e) * v : k[e] * v;
        o[i][e] = r[i].get(e);
      }
    }
    if (row0 + step < p.N) fetch(row0 + step);
    float inv1 = 1.f;
    if (p.w_post != nullptr) {
      team_sums(s, team, red, half);
      inv1 = 1.f / sqrtf(s[0] * inv_d + p.eps);
    }
    float by = inv1;
    if (DROP && __builtin_expect(!(inv1 < INFINITY), 0)) {  // 0 x NaN: what goes adds nothing to r, whatever y holds
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) b[i][e] = (all >> (8 * i + e)) & 1u ? b[i][e] * inv1 : 0.f;
      }
      by = 1.f;
    }
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at.t + i * at.width;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        o[i][e] = __builtin_fmaf(b[i][e], by, o[i][e]);
        s[0] = __builtin_fmaf(o[i][e], o[i][e], s[0]);
      }
      Eight<T> v;
      v.set(o[i]);
      if (live && c < d8) v.store(row_at<T>(p.r_out, row0, p.d, offset_of<T>(row0, p.N, at.sub, (uint32_t)p.d, c, true)));
    }
    float inv2 = 1.f;
    if (p.w_pre != nullptr) {
      team_sums(s, team, red, half);
      inv2 = 1.f / sqrtf(s[0] * inv_d + p.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = at.t + i * at.width;
        float k[8];
        read8(w2, (int)p.d, c < d8 ? c : 0, k);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[i][e] *= inv2 * k[e];
        Eight<T> v;
        v.set(o[i]);
        if (live && c < d8) v.store(row_at<T>(p.x, row0, p.d, offset_of<T>(row0, p.N, at.sub, (uint32_t)p.d, c, true)));
      }
    }
    if (p.stats != nullptr && live && at.t == 0) {
      p.stats[row0 + at.sub] = inv1;
      p.stats[p.N + row0 + at.sub] = inv2;
    }
  }
}

// Per workgroup, part[block][which][d]: sum m D n1 (m the kept ones, times a row's
// gate) where `a`, from which dw_post and the gradient of a gate [d] follow by the
// columns' factors, and sum dx n2 with w_pre.
template <typename T, int NV, int MT, bool ROWS, bool DROP>
__global__ void __launch_bounds__(MT) __attribute__((amdgpu_waves_per_eu(bwd_waves<T, MT>())))
add_norm_bwd_kernel(NormArgs p, NormGrads q, Team team) {
  __shared__ float red[2 * 3 * 16];
  extern __shared__ float columns[];
  float *f = columns, *w2 = columns + p.d;
  int half = 0;
  const Place at(team);
  const int d8 = (int)(p.d >> 3);
  const uint64_t offset = DROP ? drop_offset(p.drop) : 0;
  const float inv_d = 1.f / (float)p.d;
  const bool post = p.w_post != nullptr, pre = q.dx != nullptr;
  float aa[NV][8], a2[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) aa[i][e] = a2[i][e] = 0.f;
  Eight<T> y[NV], r[NV], dx[NV], dro[NV], g[ROWS ? NV : 1];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    dx[i].clear();
    dro[i].clear();
  }
  float inv1 = 1.f, inv2 = 1.f;
  const auto fetch = [&](int64_t row0) {
    const void *ys = rows_of<T>(p.y, row0, p.d), *rs = rows_of<T>(p.r, row0, p.d);
    const void *xs = rows_of<T>(q.dx, row0, p.d), *os = rows_of<T>(q.dr_in, row0, p.d);
    const void* gs = ROWS ? rows_of<T>(p.gate, row0, p.d) : nullptr;
    const bool live = row0 + at.sub < p.N;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at.t + i * at.width;
      const uint32_t off = offset_of<T>(row0, p.N, at.sub, (uint32_t)p.d, c, c < d8);
      y[i].load((const T*)((const char*)ys + off));
      r[i].load((const T*)((const char*)rs + off));
      if constexpr (ROWS) g[i].load((const T*)((const char*)gs + off));
      load_at<T>(dx[i], xs, off);
      load_at<T>(dro[i], os, off);
    }
    const int64_t rc = live ? row0 + at.sub : p.N - 1;
    if (post) inv1 = p.stats_in[rc];
    if (pre) inv2 = p.stats_in[p.N + rc];
  };
  // rows so wide that 1,024 threads hold two vectors each have no registers for the next one's values
  constexpr bool AHEAD = MT <= 512 || NV == 1;
  const int64_t step = (int64_t)gridDim.x * team.rows;
  if (AHEAD) fetch((int64_t)blockIdx.x * team.rows);
  column_weights<T, ROWS>(p, f, w2);
  for (int64_t row0 = (int64_t)blockIdx.x * team.rows; row0 < p.N; row0 += step) {
    const bool live = row0 + at.sub < p.N;
    const uint64_t group0 = (uint64_t)row0 * (uint64_t)d8 + (uint64_t)(uint32_t)(at.sub * d8);
    if (!AHEAD) fetch(row0);
    // the row's values move aside, so that the next row's are under way for all of this one's turn
    const float i1 = inv1, i2 = inv2;
    Eight<T> cy[NV], cr[NV], cx[NV], co[NV], cg[ROWS ? NV : 1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      cy[i] = y[i];
      cr[i] = r[i];
      cx[i] = dx[i];
      co[i] = dro[i];
      if constexpr (ROWS) cg[i] = g[i];
    }
    if (AHEAD && row0 + step < p.N) fetch(row0 + step);
    float n1[NV][8], n2[NV][8], D[NV][8], gr[ROWS ? NV : 1][8];
    uint32_t kept[NV];
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      __builtin_amdgcn_sched_barrier(0);  // one vector after the other: their weights together would not fit
      kept[i] = 0xFFu;
      if constexpr (DROP) kept[i] = kept_bits(p.drop, offset, group0 + (uint32_t)(at.t + i * at.width));
      const int c = at.t + i * at.width;
      if (!live || c >= d8) {  // nothing of it enters a sum
        cy[i].clear();
        cr[i].clear();
        cx[i].clear();
        co[i].clear();
        if constexpr (ROWS) cg[i].clear();
      }
      const float j1 = !DROP || (live && c < d8) ? i1 : 0.f;  // nor 0 x NaN
      float k[8], k2[8], b[8];
      read8(f, (int)p.d, c < d8 ? c : 0, k);
      read8(w2, (int)p.d, c < d8 ? c : 0, k2);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n1[i][e] = cy[i].get(e) * j1;
        b[e] = k[e] * n1[i][e];
        if constexpr (ROWS) b[e] *= gr[i][e] = cg[i].get(e);
        if (DROP && !((kept[i] >> e) & 1u)) b[e] = 0.f;
        D[i][e] = co[i].get(e);
      }
      if (pre) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          n2[i][e] = (cr[i].get(e) + b[e]) * i2;
          const float x = cx[i].get(e), a = x * k2[e];
          a2[i][e] = __builtin_fmaf(x, n2[i][e], a2[i][e]);
          D[i][e] = __builtin_fmaf(a, i2, D[i][e]);
          s[0] = __builtin_fmaf(a, n2[i][e], s[0]);
          s[2] = __builtin_fmaf(b[e], n2[i][e], s[2]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) n2[i][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) s[1] = __builtin_fmaf(b[e], D[i][e], s[1]);
    }
    team_sums(s, team, red, half);
    const float c2 = s[0] * inv_d * i2;                        // mean(a n2) / rms(r')
    const float c1 = post ? (s[1] - c2 * s[2]) * inv_d : 0.f;  // mean(e n1)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at.t + i * at.width;
      __builtin_amdgcn_sched_barrier(0);
      const bool out = live && c < d8;
      const uint32_t off = offset_of<T>(row0, p.N, at.sub, (uint32_t)p.d, c, true);
      float o[8], og[8], k[8];
      read8(f, (int)p.d, c < d8 ? c : 0, k);
#pragma unroll
      for (int e = 0; e < 8; ++e) D[i][e] = __builtin_fmaf(-c2, n2[i][e], D[i][e]);
      Eight<T> v;
      v.set(D[i]);
      if (out) v.store(row_at<T>(q.dr, row0, p.d, off));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float m = DROP && !((kept[i] >> e) & 1u) ? 0.f : D[i][e];
        if constexpr (ROWS) {
          og[e] = k[e] * m * n1[i][e];
          m *= gr[i][e];
        }
        aa[i][e] = __builtin_fmaf(m, n1[i][e], aa[i][e]);
        o[e] = __builtin_fmaf(k[e], m, -n1[i][e] * c1) * i1;
      }
      v.set(o);
      if (out) v.store(row_at<T>(q.dy, row0, p.d, off));
      if constexpr (ROWS) {
        v.set(og);
        if (out) v.store(row_at<T>(q.dgate, row0, p.d, off));
      }
    }
  }
  float* to = q.part + (int64_t)blockIdx.x * q.sums * p.d;
  float* to2 = q.a ? to + p.d : to;
  if (team.rows == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at.t + i * at.width;
      if (c >= d8) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (q.a) to[8 * c + e] = aa[i][e];
        if (p.w_pre != nullptr) to2[8 * c + e] = a2[i][e];
      }
    }
    return;
  }
  // rows side by side hold the same columns: within the wave first, then wave by wave
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      for (int o = 32; o >= team.lanes; o >>= 1) {
        aa[i][e] += __shfl_xor(aa[i][e], o);
        a2[i][e] += __shfl_xor(a2[i][e], o);
      }
  const int wave = threadIdx.x >> 6;
  float* sums = columns;
  __syncthreads();  // the weights are read no more
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) {
    if (w == wave && (int)(threadIdx.x & 63) < team.lanes) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = at.t + i * at.width;
        if (c >= d8) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float* u = sums + 8 * c + e;
          u[0] = w == 0 ? aa[i][e] : u[0] + aa[i][e];
          u[p.d] = w == 0 ? a2[i][e] : u[p.d] + a2[i][e];
        }
      }
    }
    __syncthreads();
  }
  for (int64_t c = threadIdx.x; c < p.d; c += blockDim.x) {
    if (q.a) to[c] = sums[c];
    if (p.w_pre != nullptr) to2[c] = sums[p.d + c];
  }
}

// The workgroups' sums of a column, in a fixed order: 32 columns a workgroup, 32
// threads a column, 8 loads of each in flight (64 columns: 1.7 us more for 4,099 x 1,000
// fp32, 16: 1 us more for a pass of 32,768 x 2,880).
constexpr int kSumCols = 32, kSumRows = 1024 / kSumCols;
template <typename T>
__global__ void __launch_bounds__(1024) column_sum_kernel(NormArgs p, NormGrads q, int rows) {
  __shared__ float red[kSumRows][kSumCols];
  const int x = threadIdx.x % kSumCols, y = threadIdx.x / kSumCols;
  const int64_t cols = q.sums * p.d;
  const int64_t c = (int64_t)blockIdx.x * kSumCols + x;
  float s = 0.f;
  if (c < cols) {
    const float* from = q.part + c;
    int b = y;
    for (; b + 7 * kSumRows < rows; b += 8 * kSumRows) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = from[(int64_t)(b + kSumRows * i) * cols];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; b < rows; b += kSumRows) s += from[(int64_t)b * cols];
  }
  red[y][x] = s;
  __syncthreads();
  if (y != 0 || c >= cols) return;
#pragma unroll
  for (int i = 1; i < kSumRows; ++i) s += red[i][x];
  if (!q.a || c >= p.d) {
    q.dw_pre[q.a ? c - p.d : c] = s;
    return;
  }
  s *= p.drop.border ? p.scale * p.drop.keep : p.scale;
  const bool vec = p.gate != nullptr && !p.gate_rows;
  if (p.w_post != nullptr) q.dw_post[c] = vec ? s * (float)((const T*)p.gate)[c] : s;
  if (vec) ((float*)q.dgate)[c] = p.w_post != nullptr ? s * (float)((const T*)p.w_post)[c] : s;
}

// A row's lanes, and how many vectors of 8 each holds: up to `most`, or two where 16
// waves would not do.  Forward two (32,768 x 2,880 bf16 146 us, with one 190), backward
// one (272 us, with two 330; both before sums over lanes stayed in registers): fewer registers, more rows under way.
constexpr int kFwdVec = 2, kBwdVec = 1;
struct Shape {
  Team team;
  int nv, threads;
};
Shape shape_of(int64_t d, int most) {
  const int64_t d8 = d / 8;
  Shape r{{64, 4, 1}, 1, 256};
  if (d8 <= 64 * most) {  // four waves, a row each, or several where it is short
    if (d8 <= 64) {
      while (r.team.lanes > 1 && r.team.lanes / 2 >= d8) r.team.lanes /= 2;
      r.team.rows = 256 / r.team.lanes;
    } else {
      r.nv = (int)((d8 + 63) / 64);
    }
    return r;
  }
  if (d8 > 16 * 64 * most) most = 2;
  r.team.span = (int)((d8 + 64 * most - 1) / (64 * most));
  r.team.rows = 1;
  r.nv = (int)((d8 + 64 * r.team.span - 1) / (64 * r.team.span));
  r.threads = 64 * r.team.span;
  return r;
}

// Workgroups: as many as the 256 compute units hold at once with `waves` waves a
// SIMD, since one more would run after all others.
int blocks_of(int64_t N, const Shape& h, int waves) {
  const int64_t need = (N + h.team.rows - 1) / h.team.rows;
  const int64_t unit = 4 * waves / (h.threads / 64);
  const int64_t most = 256 * (unit > 0 ? unit : 1);
  return (int)(need < most ? need : most);
}
template <typename T, bool ROWS>
int fwd_blocks(int64_t N, const Shape& h) {
  return blocks_of(N, h, h.threads > 512 ? fwd_waves<T, 2, 1024, ROWS>()
                         : h.nv == 1    ? fwd_waves<T, 1, 512, ROWS>()
                                        : fwd_waves<T, 2, 512, ROWS>());
}
// The backward pass's, each with its sums.
template <typename T>
int bwd_blocks(int64_t N, const Shape& h) {
  return blocks_of(N, h, h.threads > 512 ? bwd_waves<T, 1024>() : bwd_waves<T, 512>());
}

template <typename T, int NV, int MT>
void add_norm_as(const NormArgs& p, const Shape& h, dim3 grid, hipStream_t s) {
  const dim3 block(h.threads);
  const bool drop = p.drop.border != 0;
  const size_t lds = (size_t)p.d * 8;
  if (p.gate_rows && drop)
    hipLaunchKernelGGL((add_norm_kernel<T, NV, MT, true, true>), grid, block, lds, s, p, h.team);
  else if (p.gate_rows)
    hipLaunchKernelGGL((add_norm_kernel<T, NV, MT, true, false>), grid, block, lds, s, p, h.team);
  else if (drop)
    hipLaunchKernelGGL((add_norm_kernel<T, NV, MT, false, true>), grid, block, lds, s, p, h.team);
  else
    hipLaunchKernelGGL((add_norm_kernel<T, NV, MT, false, false>), grid, block, lds, s, p, h.team);
}

template <typename T>
hipError_t add_norm_of(const NormArgs& p, hipStream_t s) {
  const Shape h = shape_of(p.d, kFwdVec);
  const dim3 grid(p.gate_rows ? fwd_blocks<T, true>(p.N, h) : fwd_blocks<T, false>(p.N, h));
  if (h.threads > 512)
    add_norm_as<T, 2, 1024>(p, h, grid, s);
  else if (h.nv == 1)
    add_norm_as<T, 1, 512>(p, h, grid, s);
  else
    add_norm_as<T, 2, 512>(p, h, grid, s);
  return hipGetLastError();
}

template <typename T, int NV, int MT>
void add_norm_bwd_as(const NormArgs& p, const NormGrads& q, const Shape& h, dim3 grid, hipStream_t s) {
  const dim3 block(h.threads);
  const bool drop = p.drop.border != 0;
  const size_t lds = (size_t)p.d * 8;
  if (p.gate_rows && drop)
    hipLaunchKernelGGL((add_norm_bwd_kernel<T, NV, MT, true, true>), grid, block, lds, s, p, q, h.team);
  else if (p.gate_rows)
    hipLaunchKernelGGL((add_norm_bwd_kernel<T, NV, MT, true, false>), grid, block, lds, s, p, q, h.team);
  else if (drop)
    hipLaunchKernelGGL((add_norm_bwd_kernel<T, NV, MT, false, true>), grid, block, lds, s, p, q, h.team);
  else
    hipLaunchKernelGGL((add_norm_bwd_kernel<T, NV, MT, false, false>), grid, block, lds, s, p, q, h.team);
}

template <typename T>
hipError_t add_norm_bwd_of(const NormArgs& p, NormGrads q, hipStream_t s) {
  q.a = p.w_post != nullptr || (p.gate != nullptr && !p.gate_rows);
  q.sums = (q.a ? 1 : 0) + (p.w_pre != nullptr ? 1 : 0);
  const Shape h = shape_of(p.d, kBwdVec);
  const int blocks = bwd_blocks<T>(p.N, h);
  const dim3 grid(blocks);
  if (h.threads > 512 && h.nv == 1)
    add_norm_bwd_as<T, 1, 1024>(p, q, h, grid, s);
  else if (h.threads > 512)
    add_norm_bwd_as<T, 2, 1024>(p, q, h, grid, s);
  else
    add_norm_bwd_as<T, 1, 512>(p, q, h, grid, s);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || q.sums == 0) return e;
  hipLaunchKernelGGL((column_sum_kernel<T>), dim3((unsigned)((q.sums * p.d + kSumCols - 1) / kSumCols)), dim3(1024), 0, s, p, q, blocks);
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
  const Shape h = shape_of(d, kBwdVec);  // the most workgroups of all types
  return N > 0 ? (uint64_t)bwd_blocks<__bf16>(N, h) * (uint64_t)sums * (uint64_t)d * 4 : 0;
}

hipError_t launch_add_norm_bwd(Dtype dt, const NormArgs& p, const NormGrads& q, hipStream_t s) {
  return dt == DT_BF16 ? add_norm_bwd_of<__bf16>(p, q, s) : add_norm_bwd_of<float>(p, q, s);
}

}  // namespace ckl
