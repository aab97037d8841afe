// Loads and stores of eight consecutive elements, wave reductions, and the
// counter-based generator, shared by the row-wise operators (log-probabilities,
// the residual's norms, dropout).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"

namespace ckl {

typedef uint32_t row_u32x4 __attribute__((ext_vector_type(4)));
typedef float row_f32x4 __attribute__((ext_vector_type(4)));
// 16 bytes at the alignment of an element: gfx950 loads and stores them at any
// address, so rows of odd lengths and strides need no path of their own.
struct __attribute__((packed, aligned(2))) Raw16 {
  row_u32x4 v;
};

template <typename T>
struct Eight;
template <>
struct Eight<__bf16> {
  row_u32x4 a;
  __device__ inline void clear() { a = row_u32x4{0, 0, 0, 0}; }
  __device__ inline void load(const __bf16* p) { a = ((const Raw16*)p)->v; }
  __device__ inline void store(__bf16* p) const { ((Raw16*)p)->v = a; }
  __device__ inline float get(int i) const {
    const uint32_t w = a[i >> 1];
    return __builtin_bit_cast(float, (i & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
  __device__ inline void set(const float (&f)[8]) {
    typedef __attribute__((__vector_size__(8 * sizeof(__bf16)))) __bf16 bf16x8_t;
    const bf16x8_t v = {(__bf16)f[0], (__bf16)f[1], (__bf16)f[2], (__bf16)f[3],
                        (__bf16)f[4], (__bf16)f[5], (__bf16)f[6], (__bf16)f[7]};
    a = __builtin_bit_cast(row_u32x4, v);
  }
};
template <>
struct Eight<float> {
  row_u32x4 a, b;
  __device__ inline void clear() { a = b = row_u32x4{0, 0, 0, 0}; }
  __device__ inline void load(const float* p) {
    a = ((const Raw16*)p)->v;
    b = ((const Raw16*)(p + 4))->v;
  }
  __device__ inline void store(float* p) const {
    ((Raw16*)p)->v = a;
    ((Raw16*)(p + 4))->v = b;
  }
  __device__ inline float get(int i) const { return __builtin_bit_cast(float, i < 4 ? a[i] : b[i - 4]); }
  __device__ inline void set(const float (&f)[8]) {
    a = row_u32x4{__builtin_bit_cast(uint32_t, f[0]), __builtin_bit_cast(uint32_t, f[1]),
                  __builtin_bit_cast(uint32_t, f[2]), __builtin_bit_cast(uint32_t, f[3])};
    b = row_u32x4{__builtin_bit_cast(uint32_t, f[4]), __builtin_bit_cast(uint32_t, f[5]),
                  __builtin_bit_cast(uint32_t, f[6]), __builtin_bit_cast(uint32_t, f[7])};
  }
};

// A lane's value from a neighbour of its row of 16 by data-parallel move.
template <int CTRL>
__device__ inline float dpp(float v) {
  const int b = __builtin_bit_cast(int, v);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(b, b, CTRL, 0xF, 0xF, true));
}
// The two rows of 16 (two halves of 32) of each lane's pair, the lower one first.
__device__ inline float2 rows16(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  return make_float2(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ inline float2 rows32(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  return make_float2(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E;       // quad_perm: lane i takes i ^ 1, i ^ 2
constexpr int kMirror8 = 0x141, kMirror16 = 0x140;  // lane i takes 7 - i of its 8, 15 - i of its 16

// Sum over `lanes` consecutive lanes (a power of two up to 64), in every lane.  In
// registers: with shuffles through LDS, six for each of a row's sums one after the
// other, the norms' backward pass of 23,301 x 2,880 bf16 with dropout took 205 us for 174.
__device__ inline float lanes_sum(float v, int lanes) {
  if (lanes > 1) v += dpp<kSwap1>(v);
  if (lanes > 2) v += dpp<kSwap2>(v);
  if (lanes > 4) v += dpp<kMirror8>(v);
  if (lanes > 8) v += dpp<kMirror16>(v);
  if (lanes > 16) {
    const float2 r = rows16(v);
    v = r.x + r.y;
  }
  if (lanes > 32) {
    const float2 r = rows32(v);
    v = r.x + r.y;
  }
  return v;
}
// Largest value of the wave (NaN left out), in every lane.
__device__ inline float wave_max(float v) {
  v = fmaxf(v, dpp<kSwap1>(v));
  v = fmaxf(v, dpp<kSwap2>(v));
  v = fmaxf(v, dpp<kMirror8>(v));
  v = fmaxf(v, dpp<kMirror16>(v));
  float2 r = rows16(v);
  r = rows32(fmaxf(r.x, r.y));
  return fmaxf(r.x, r.y);
}

// A barrier that orders LDS only: __syncthreads also waits for every global load
// and store of the wave, and with it for the next row's loads.
__device__ inline void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// ------------------------------------------------------------------ random bits
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC11): ten rounds of two 32 x 32 -> 64 bit products on a
// 128-bit counter under a 64-bit key.  Counter: the group of eight elements in
// the low 64 bits, the caller's offset in the high ones; key: the seed.  Element
// 8 g + i of a tensor takes bits 16 (i % 2) .. + 15 of word i / 2 of group g, so
// an element's number depends on (seed, offset, its index) alone, whatever the
// launch, and the mask need not be kept for the gradient.
__device__ inline row_u32x4 philox(uint64_t group, uint64_t offset, uint64_t seed) {
  uint32_t c0 = (uint32_t)group, c1 = (uint32_t)(group >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p = (uint64_t)c0 * 0xD2511F53u, q = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(q >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)q;
    c2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return row_u32x4{c0, c1, c2, c3};
}
__device__ inline uint32_t bits16(const row_u32x4& w, int i) { return (i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu; }

__device__ inline uint64_t drop_offset(const Drop& r) { return r.offset + (r.at != nullptr ? (uint64_t)*r.at : 0u); }

}  // namespace ckl
