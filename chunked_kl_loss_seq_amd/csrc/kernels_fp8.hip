// Matrix product in 8-bit floating point (OCP e4m3) with a scale per block of
// 128, and the quantisers of its operands: the head of a teacher or a served
// student whose weight is held in 8 bits.
//
//   rows    x [M, d]:  s[kb][m] = amax of x[m][128 kb ..] / 448
//   weight  w [V, d]:  s[vb][kb] = amax of the 128 x 128 block / 448
//   q = e4m3(x / s), to nearest even, so |q| <= 448, the type's largest
//   out[m][v] = sum_kb xs[kb][m] ws[v / 128][kb] sum_{k in block kb} xq[m][k] wq[v][k]
//
// Two ways to multiply a block:
//   * bf16 results: v_mfma_f32_16x16x128_f8f6f4 reduces exactly one block of
//     128 k, so a block product is one instruction from a zero accumulator.
//     Within each group of 8 k the instruction aligns the products to the
//     group's largest exponent and drops what lies more than 13 bits below it
//     (measured: beside 1, 2^-13 is kept and 2^-14 is not; between groups and
//     into the accumulator 2^-23 is kept).  That is below 7 x 2^-13 of a
//     group's largest product, about 3e-5 of a result in the mean, a hundredth
//     of its rounding to bf16.
//   * fp32 results, which that would cost five bits, and the few-row kernel,
//     which waits for memory anyway: the values are widened to bf16 (exactly:
//     4-bit significands) and go through four v_mfma_f32_16x16x32_bf16, whose
//     sums hold fp32; half the rate.
// Either way the block product is multiplied by its scale into the running
// fp32 sum with four vector FMAs per lane (arbitrary fp32 scales; the
// instruction's own are powers of two per 32 k).  Tokens are the instruction's
// columns: a lane holds one token and four consecutive ids, so its scale is
// one register and its results are adjacent in memory.
//
//   * M <= 16 and a short weight (too few tiles to fill the chip), or M <= 2 and a
//     very long one.  Weight rows go straight from memory to registers, no LDS;
//     four waves share 32 rows, each taking a quarter of the k blocks, and add
//     their sums through LDS.  1 x 201,088 x 2,880: 105 us, 5.5 TB/s, the rate
//     of reading the weight.
//   * else tiles staged through a two-stage LDS ring by LDS DMA, one barrier
//     per block of k, of the size that is expected to end first.  Up to about
//     128 rows this is bound by reading the weight (16 x 201,088 x 2,880: 117-121
//     us, 4.8 TB/s).  2,048 x 201,088 x 2,880 takes 1,250 us (1,900 TFLOP/s; the
//     library's product with one scale 1,215): the matrix cores are busy 45 % of
//     the cycles at 2.0 GHz, vector instructions issue in 36 % of them, and a third
//     of the waves' time goes to the barrier and loads, a third to waiting for
//     issue.  Loading the next block's fragments across the barrier did not make
//     it faster (1,285 us for 1,277).  fp32 results of the same shape take 2,100 us.
#include "gemm_core.hpp"
#include "launch.hpp"

namespace ckl {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kBlk = 128;          // k per scale
constexpr float kE4m3Max = 448.f;

__device__ inline f32x4 block_product(const i32x8& a, const i32x8& b) {
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  // format 0 = e4m3 for both operands; zero scale operands select the
  // instruction without scales
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}
__device__ inline i32x8 join(const u32x4& lo, const u32x4& hi) {
  i32x8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = (int)lo[i];
    v[4 + i] = (int)hi[i];
  }
  return v;
}

// 32 e4m3 values as four bf16 operands of 8 (the k order is the lane's own, the
// same for both operands).
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
struct Wide {
  bf16x8 v[4];
};
__device__ inline Wide widen(const i32x8& a) {
  Wide w;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a[2 * i + h], 1.f, false);
      const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a[2 * i + h], 1.f, true);
      w.v[i][4 * h] = lo[0];
      w.v[i][4 * h + 1] = lo[1];
      w.v[i][4 * h + 2] = hi[0];
      w.v[i][4 * h + 3] = hi[1];
    }
  return w;
}
__device__ inline f32x4 block_product(const Wide& a, const Wide& b) {
  f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], c, 0, 0, 0);
  return c;
}

// ---------------------------------------------------------------- quantisers
// Eight values of a row of x, fp32.
template <typename T>
__device__ inline void load8(const T* p, float* f) {
  if constexpr (sizeof(T) == 2) {
    const u32x4 v = *(const u32x4*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = v[i];
      f[2 * i] = __builtin_bit_cast(float, w << 16);
      f[2 * i + 1] = __builtin_bit_cast(float, w & 0xFFFF0000u);
    }
  } else {
    const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = a[i];
      f[4 + i] = b[i];
    }
  }
}
__device__ inline bool finite(float x) { return (__builtin_bit_cast(uint32_t, x) & 0x7F800000u) != 0x7F800000u; }
__device__ inline float amax8(const float* f) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, finite(f[i]) ? fabsf(f[i]) : 0.f);
  return m;
}
// The scale of a block: 1 where it is all zeros, and at least the smallest
// normal number, so that x / s stays finite.
__device__ inline float scale_of(float amax) { return amax > 0.f ? fmaxf(amax / kE4m3Max, 0x1p-126f) : 1.f; }
// x / s is the correctly rounded fp32 quotient, at most 448 (1 + 2^-23), which
// rounds to 448; a value that is not finite becomes NaN.
__device__ inline void store8(uint8_t* q, const float* f, float s) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = finite(f[i]) ? f[i] / s : __builtin_nanf("");
  u32x2 o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h], v[4 * h + 1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2], v[4 * h + 3], w, true);
    o[h] = (uint32_t)w;
  }
  *(u32x2*)q = o;
}

// Blocks of 1 x 128: 16 lanes per block, 8 values a lane.
constexpr int kQThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kQThreads) quantize_rows_kernel(const T* __restrict__ x, int64_t R, int64_t C,
                                                                 int kb_n, uint8_t* __restrict__ q,
                                                                 float* __restrict__ scales) {
  const int64_t g = (int64_t)blockIdx.x * (kQThreads / 16) + (threadIdx.x >> 4);  // block index
  const int l = threadIdx.x & 15;
  if (g >= R * kb_n) return;  // whole groups of 16 lanes: the shuffles below stay within one
  const int64_t r = g / kb_n;
  const int kb = (int)(g - r * kb_n);
  const int64_t c = (int64_t)kb * kBlk + 8 * l;
  float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const bool on = c < C;
  if (on) load8(x + r * C + c, f);
  float m = amax8(f);
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
  const float s = scale_of(m);
  if (l == 0) scales[(int64_t)kb * R + r] = s;
  if (on) store8(q + r * C + c, f, s);
}

// Blocks of 128 x 128: one workgroup each, held in registers between the two steps.
template <typename T>
__global__ void __launch_bounds__(kQThreads) quantize_blocks_kernel(const T* __restrict__ x, int64_t R, int64_t C,
                                                                   int kb_n, uint8_t* __restrict__ q,
                                                                   float* __restrict__ scales) {
  __shared__ float red[kQThreads / 64];
  const int64_t rb = blockIdx.x / kb_n;
  const int kb = (int)(blockIdx.x - rb * kb_n);
  const int64_t c = (int64_t)kb * kBlk + 8 * (threadIdx.x & 15);
  const int64_t r0 = rb * kBlk + (threadIdx.x >> 4);
  constexpr int kIt = kBlk / (kQThreads / 16);
  float f[kIt][8], m = 0.f;
#pragma unroll
  for (int i = 0; i < kIt; ++i) {
    const int64_t r = r0 + i * (kQThreads / 16);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[i][j] = 0.f;
    if (r < R && c < C) load8(x + r * C + c, f[i]);
    m = fmaxf(m, amax8(f[i]));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  m = red[0];
#pragma unroll
  for (int i = 1; i < kQThreads / 64; ++i) m = fmaxf(m, red[i]);
  const float s = scale_of(m);
  if (threadIdx.x == 0) scales[blockIdx.x] = s;
#pragma unroll
  for (int i = 0; i < kIt; ++i) {
    const int64_t r = r0 + i * (kQThreads / 16);
    if (r < R && c < C) store8(q + r * C + c, f[i], s);
  }
}

// ---------------------------------------------------------------- product
struct Fp8Args {
  const uint8_t* xq;  // [M, d]
  const float* xs;    // [kb, M]
  const uint8_t* wq;  // [V, d]
  const float* ws;    // [ceil(V / 128), kb]
  int64_t M, V, d;
  int kb;             // ceil(d / 128)
  void* out;          // [M, V]
  int vec;            // rows of out are 16-byte aligned
};

__device__ inline void put(float* p, float v) { *p = v; }
__device__ inline void put(__bf16* p, float v) { *p = (__bf16)v; }

// ------------------------------------------- few rows
constexpr int kFewRows = 16;   // tokens: one instruction's columns
constexpr int kFewIds = 32;    // weight rows per workgroup
constexpr int kFewWaves = 4;
template <typename TO>
__global__ void __launch_bounds__(kFewWaves * 64) fp8_few_kernel(Fp8Args p) {
  __shared__ f32x4 part[kFewWaves - 1][2][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int64_t v0 = (int64_t)blockIdx.x * kFewIds;
  const bool tok = c < p.M;
  const uint8_t* wrow[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int64_t v = v0 + 16 * i + c;
    if (v >= p.V) v = p.V - 1;  // read again, not stored
    wrow[i] = p.wq + v * p.d;
  }
  const uint8_t* xrow = p.xq + (tok ? c : 0) * p.d;
  const float* wscale = p.ws + (v0 / kBlk) * p.kb;  // 32 ids never cross a block of 128
  f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  const u32x4 zero = {0, 0, 0, 0};
  constexpr int U = 3;  // blocks in flight per wave
  for (int k0 = w; k0 < p.kb; k0 += U * kFewWaves) {
    u32x4 a[U][2][2], b[U][2];
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = k0 + u * kFewWaves;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // lane quarter g holds the 16-byte chunks g and 4 + g of the block
        const int64_t k = (int64_t)kb * kBlk + 64 * h + 16 * g;
        const bool in = kb < p.kb && k < p.d;
        a[u][0][h] = a[u][1][h] = b[u][h] = zero;
        if (in) {
          a[u][0][h] = *(const u32x4*)(wrow[0] + k);
          a[u][1][h] = *(const u32x4*)(wrow[1] + k);
        }
        if (in && tok) b[u][h] = *(const u32x4*)(xrow + k);
      }
      s[u] = kb < p.kb && tok ? p.xs[(int64_t)kb * p.M + c] * wscale[kb] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Wide bj = widen(join(b[u][0], b[u][1]));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const f32x4 t = block_product(widen(join(a[u][i][0], a[u][i][1])), bj);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][r] = __builtin_fmaf(t[r], s[u], acc[i][r]);
      }
    }
  }
  if (w > 0) {
    part[w - 1][0][lane] = acc[0];
    part[w - 1][1][lane] = acc[1];
  }
  __syncthreads();
  if (w > 0 || !tok) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int j = 0; j < kFewWaves - 1; ++j) acc[i] += part[j][i][lane];
    TO* dst = (TO*)p.out + c * p.V + v0 + 16 * i + 4 * g;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (v0 + 16 * i + 4 * g + r < p.V) put(dst + r, acc[i][r]);
  }
}

// ------------------------------------------- tiles
// BM ids x BN tokens, WM x (BN / 64) waves of (BM / WM) x 64.  The ring's stage
// holds the tile's 128-byte rows of both operands (16-byte chunks XOR-swizzled
// by the row) and the BN token scales of the block.
// Lane l's 4 bytes at byte voff of the resource go to LDS byte lds_addr + 4 l;
// see dma16 for why this is written out.
__device__ inline void dma4(const i32x4& rsrc, uint32_t voff, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds" ::"v"(voff), "s"(rsrc),
               "s"(lds_addr)
               : "memory", "m0");
}

// Copies R rows x 128 bytes (one block of k) of an operand into LDS, laid out
// as KTile.  One instruction of a wave fills 8 rows; a wave's next one lies
// NW x 8 rows on, a multiple of the swizzle's period, so one lane offset serves
// all and the resource moves on by the rows' distance (2,048 x 201,088 x 2,880
// 1,256 us; added to the lane offset 1,316; the instruction's scalar offset
// will not do, as the range check need not cover it).  Rows past the operand lie
// past the resource's end, k past d only on the last block: both read as zeros.
template <int R, int NW>
struct BlockDMA {
  static constexpr int kBytes = R * kBlk;
  static constexpr int kNI = kBytes / 1024 / NW;
  static_assert(kBytes % (1024 * NW) == 0, "whole loads per wave");
  static_assert((NW * 8) % 16 == 0 || kNI == 1, "the swizzle repeats every 16 rows");
  uint64_t org;      // row 0 of the tile, k = 0
  uint32_t voff, step, rows;
  __device__ inline void init(const uint8_t* ptr, int64_t row0, int64_t ext, int64_t d, int wave, int lane) {
    org = uniform64((uint64_t)ptr + (uint64_t)(row0 * d));
    rows = (uint32_t)(ext - row0 < R ? ext - row0 : R);
    const int row = wave * 8 + (lane >> 3);
    voff = (uint32_t)row * (uint32_t)d + (uint32_t)(chunk(wave, lane) * 16);
    step = (uint32_t)(NW * 8) * (uint32_t)d;
  }
  __device__ static inline int chunk(int wave, int lane) {
    const int row = wave * 8 + (lane >> 3);
    return (lane & 7) ^ ((row >> 1) & 7);
  }
  __device__ inline void issue(int64_t k0, int64_t d, uint32_t lds, int wave, int lane) const {
    uint64_t at = org + (uint64_t)k0;
    int32_t left = (int32_t)(rows * (uint32_t)d - (uint32_t)k0);
    uint32_t v = voff;
    if (d - k0 < kBlk && chunk(wave, lane) * 16 >= (int)(d - k0)) v = kOOB;
#pragma unroll
    for (int i = 0; i < kNI; ++i) {
      i32x4 rs = make_rsrc((const void*)at);
      rs.z = left > 0 ? left : 0;
      dma16(rs, v, lds + (uint32_t)((i * NW + wave) * 1024));
      at += step;
      left -= (int32_t)step;
    }
  }
};

// 16 rows x 128 k: lane l gets row row0 + l % 16, 16-byte chunks l / 16 and 4 + l / 16.
template <int R>
__device__ inline i32x8 load_frag8(const char* lds, int row0, int lane) {
  typedef KTile<R, kBlk> L;
  const int row = row0 + (lane & 15), g = lane >> 4;
  return join(*(const u32x4*)(lds + L::off(row, g)), *(const u32x4*)(lds + L::off(row, 4 + g)));
}

// Operand fragment of a path: 8-bit for bf16 results, widened for fp32 ones.
template <typename TO>
struct Frag8;
template <>
struct Frag8<__bf16> {
  typedef i32x8 type;
  __device__ static inline type of(const i32x8& v) { return v; }
};
template <>
struct Frag8<float> {
  typedef Wide type;
  __device__ static inline type of(const i32x8& v) { return widen(v); }
};

template <typename TO, int BM, int BN, int WM>
__global__ void __launch_bounds__(WM* BN) __attribute__((amdgpu_waves_per_eu(2)))
fp8_tile_kernel(Fp8Args p, GemmParams g) {
  constexpr int WN = BN / 64, NW = WM * WN, WTM = BM / WM, FM = WTM / 16, FN = 4;
  typedef BlockDMA<BM, NW> DA;
  typedef BlockDMA<BN, NW> DB;
  static_assert(WTM <= 128 && 128 % WTM == 0, "a wave's ids share one block of 128");
  constexpr int STAGE = DA::kBytes + DB::kBytes + BN * 4;
  constexpr int STORE = sizeof(TO) == 2 ? NW * 64 * WTM * 2 : 0;  // the epilogue's staging, in the ring's place
  __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE > STORE ? 2 * STAGE : STORE];
  const uint32_t lds0 = lds_addr(smem);
  const TileCoord tc = tile_coord(g);
  if (!tc.valid) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int64_t m0 = (int64_t)tc.tm * BM, n0 = (int64_t)tc.tn * BN;
  DA da;
  DB db;
  da.init(p.wq, m0, p.V, p.d, wave, lane);
  db.init(p.xq, n0, p.M, p.d, wave, lane);
  const uint64_t s_org = uniform64((uint64_t)p.xs + (uint64_t)n0 * 4);
  const uint32_t tokens = (uint32_t)(p.M - n0 < BN ? p.M - n0 : BN);
  auto issue = [&](int kb, int st) {
    const uint32_t at = lds0 + (uint32_t)(st * STAGE);
    const int64_t k0 = (int64_t)kb * kBlk;
    if (wave < WN) {  // wave w: the scales of tokens 64 w ..
      i32x4 rs = make_rsrc((const void*)(s_org + (uint64_t)kb * (uint64_t)p.M * 4));
      rs.z = (int32_t)(tokens * 4);
      dma4(rs, (uint32_t)tid * 4u, at + DA::kBytes + DB::kBytes + (uint32_t)wave * 256u);
    }
    da.issue(k0, p.d, at, wave, lane);
    db.issue(k0, p.d, at + DA::kBytes, wave, lane);
  };
  // The wave's weight scales, one per block of k: lane l holds block
  // 64 (kb / 64) + l, so that a block costs one v_readlane and no load's wait.
  // Ids past V are not stored and take the last scales.
  const int64_t vb_max = (p.V - 1) / kBlk;
  int64_t vb = (m0 + wm * WTM) / kBlk;
  if (vb > vb_max) vb = vb_max;
  const float* wscale = p.ws + vb * p.kb;
  float wsv = 0.f;

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int c = lane & 15, q = lane >> 4;
  issue(0, 0);
  for (int kb = 0; kb < p.kb; ++kb) {
    const int st = kb & 1;
    // block kb has landed, and every wave has left the other stage
    wait_vmcnt<0>();
    __syncthreads();
    if ((kb & 63) == 0) {
      wsv = wscale[kb + lane < p.kb ? kb + lane : p.kb - 1];
      asm volatile("" : "+v"(wsv));  // waited for here: behind the copies, the wait would cover them too
    }
    if (kb + 1 < p.kb) issue(kb + 1, st ^ 1);
    const float sw = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wsv), kb & 63));
    const char* sa = smem + st * STAGE;
    const char* sb = sa + DA::kBytes;
    const float* sc = (const float*)(sb + DB::kBytes) + wn * 64 + c;
    typename Frag8<TO>::type b[FN];
    float s[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      b[j] = Frag8<TO>::of(load_frag8<BN>(sb, wn * 64 + 16 * j, lane));
      s[j] = sc[16 * j] * sw;
    }
    // Row i's products run while row i - 1's are scaled and added, so that no
    // vector instruction waits for the matrix instruction before it, and row
    // i + 1's fragment loads.  The fences keep the scheduler from loading all
    // fragments at once, which spills.
    typename Frag8<TO>::type a = Frag8<TO>::of(load_frag8<BM>(sa, wm * WTM, lane));
    f32x4 t[2][FN];
#pragma unroll
    for (int i = 0; i <= FM; ++i) {
      i32x8 an;
      if (i + 1 < FM) an = load_frag8<BM>(sa, wm * WTM + 16 * (i + 1), lane);
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        if (i < FM) t[i & 1][j] = block_product(a, b[j]);
        if (i > 0)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[i - 1][j][r] = __builtin_fmaf(t[(i - 1) & 1][j][r], s[j], acc[i - 1][j][r]);
      }
      // the sums are wanted here, not moved to the end of the block of k
      if (i > 0)
#pragma unroll
        for (int j = 0; j < FN; ++j) asm volatile("" : "+v"(acc[i - 1][j]));
      if (i + 1 < FM) a = Frag8<TO>::of(an);
      if constexpr (sizeof(TO) == 2) {
        // one product, then the four additions of an earlier one
        if (i > 0 && i < FM) {
          if (i + 1 < FM) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // Lane (c, q), slot r of block (i, j) holds id mw + 16 i + 4 q + r of token nw + 16 j + c.
  const int64_t mw = m0 + wm * WTM, nw = n0 + wn * 64;
  if constexpr (sizeof(TO) == 2) {
    // bf16 rows leave through LDS in 16-byte pieces of a token's ids
    typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 bf16x4;
    constexpr int RC = WTM / 8;  // 16-byte chunks of a token's ids
    __syncthreads();
    char* wl = smem + wave * (64 * WTM * 2);
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int t = 16 * j + c;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const bf16x4 v = {(__bf16)acc[i][j][0], (__bf16)acc[i][j][1], (__bf16)acc[i][j][2], (__bf16)acc[i][j][3]};
        const int chunk = 2 * i + (q >> 1);
        *(bf16x4*)(wl + t * (WTM * 2) + ((chunk ^ (t & (RC - 1))) << 4) + 8 * (q & 1)) = v;
      }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < RC; ++x) {
      const int idx = x * 64 + lane;
      const int t = idx / RC, cc = idx % RC;
      const int64_t n = nw + t, m = mw + 8 * cc;
      if (n >= p.M || m >= p.V) continue;
      const u32x4 v = *(const u32x4*)(wl + t * (WTM * 2) + ((cc ^ (t & (RC - 1))) << 4));
      uint16_t* dst = (uint16_t*)p.out + n * p.V + m;
      if (p.vec) {  // V is a multiple of 8: the piece is inside the row
        *(u32x4*)dst = v;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t wd = v[e >> 1];
          if (m + e < p.V) dst[e] = (uint16_t)((e & 1) ? wd >> 16 : wd & 0xFFFFu);
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int64_t n = nw + 16 * j + c;
      if (n >= p.M) continue;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int64_t m = mw + 16 * i + 4 * q;
        if (m >= p.V) continue;
        float* dst = (float*)p.out + n * p.V + m;
        if (p.vec) {  // V is a multiple of 4
          *(f32x4*)dst = acc[i][j];
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (m + r < p.V) dst[r] = acc[i][j][r];
        }
      }
    }
  }
}

template <typename TO, int BM, int BN, int WM>
hipError_t launch_tiles(const Fp8Args& p, hipStream_t s) {
  GemmParams g{};
  g.tiles_m = cdiv64(p.V, BM);
  g.tiles_n = cdiv64(p.M, BN);
  g.splits = 1;
  g.group_m = 4;
  const int total = g.tiles_m * g.tiles_n;
  const int grid = ((total + 7) / 8) * 8;
  hipLaunchKernelGGL((fp8_tile_kernel<TO, BM, BN, WM>), dim3(grid), dim3(WM * BN), 0, s, p, g);
  return hipGetLastError();
}

// The product by the tile that is expected to end first: a tile takes `alone`
// microseconds per block of k where it has a compute unit to itself, and the
// 256 units together finish 256 tiles per `full` microseconds of each block
// where there are many (bf16 results; fp32 results take about 1.6 times as long
// for every tile).  Measured, in us (256 x 256, 128 x 128, 128 x 64, 64 x 64):
//   2,048 x 201,088 x 2,880: 1,256 1,499 - -    300 x 100,000 x 512: 44 35 35 44
//   128 x 201,088 x 2,880: 224 163 - -          1,000 x 5,000 x 1,024: 20 14 14 15
//   256 x 32,000 x 2,048: 33 23 29 34           40 x 5,000 x 4,096: 49 23 18 15
struct TileCost {
  int bm, bn;
  double alone, full;
};
constexpr TileCost kTileCosts[] = {
    {256, 256, 1.5, 2.26}, {128, 128, 0.90, 0.66}, {128, 64, 0.57, 0.44}, {64, 64, 0.48, 0.28}};

template <typename TO>
hipError_t launch_product(const Fp8Args& p, hipStream_t s) {
  // Few rows and fewer 64 x 64 tiles than compute units: the k blocks are split
  // over waves instead (8 x 10,000 x 4,096: 15 us, by tiles 19; with 500 tiles,
  // 4 x 32,000 x 2,048, 17 and 13).  Also one or two rows of a weight beyond the
  // 256 MB last-level cache, which come straight from memory: 1 x 201,088 x
  // 2,880 105 us (5.5 TB/s), by tiles 113.
  if (p.M <= kFewRows && (p.V < 64 * 256 || (p.M <= 2 && p.V * p.d > (int64_t)256 << 20))) {
    hipLaunchKernelGGL(fp8_few_kernel<TO>, dim3((unsigned)((p.V + kFewIds - 1) / kFewIds)), dim3(kFewWaves * 64), 0, s,
                       p);
    return hipGetLastError();
  }
  int best = 0;
  double least = 0.0;
  for (int i = 0; i < 4; ++i) {
    const TileCost& c = kTileCosts[i];
    const int64_t tiles = ((p.V + c.bm - 1) / c.bm) * ((p.M + c.bn - 1) / c.bn);
    const double us = (double)((tiles + 255) / 256) * c.full;
    const double cost = us > c.alone ? us : c.alone;
    if (i == 0 || cost < least) {
      best = i;
      least = cost;
    }
  }
  switch (best) {
    case 0: return launch_tiles<TO, 256, 256, 2>(p, s);
    case 1: return launch_tiles<TO, 128, 128, 2>(p, s);
    case 2: return launch_tiles<TO, 128, 64, 4>(p, s);
    default: return launch_tiles<TO, 64, 64, 4>(p, s);
  }
}

}  // namespace

hipError_t launch_quantize_fp8(Dtype dt, const void* x, int64_t R, int64_t C, bool rows, uint8_t* q, float* scales,
                               hipStream_t s) {
  const int kb = (int)((C + kBlk - 1) / kBlk);
  if (rows) {
    const int64_t groups = R * kb, per = kQThreads / 16;
    const dim3 grid((unsigned)((groups + per - 1) / per));
    if (dt == DT_BF16)
      hipLaunchKernelGGL(quantize_rows_kernel<__bf16>, grid, dim3(kQThreads), 0, s, (const __bf16*)x, R, C, kb, q,
                         scales);
    else
      hipLaunchKernelGGL(quantize_rows_kernel<float>, grid, dim3(kQThreads), 0, s, (const float*)x, R, C, kb, q,
                         scales);
  } else {
    const dim3 grid((unsigned)((R + kBlk - 1) / kBlk * kb));
    if (dt == DT_BF16)
      hipLaunchKernelGGL(quantize_blocks_kernel<__bf16>, grid, dim3(kQThreads), 0, s, (const __bf16*)x, R, C, kb, q,
                         scales);
    else
      hipLaunchKernelGGL(quantize_blocks_kernel<float>, grid, dim3(kQThreads), 0, s, (const float*)x, R, C, kb, q,
                         scales);
  }
  return hipGetLastError();
}

hipError_t launch_matmul_fp8(Dtype out_dt, const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                             int64_t M, int64_t V, int64_t d, void* out, hipStream_t s) {
  Fp8Args p{xq, xs, wq, ws, M, V, d, (int)((d + kBlk - 1) / kBlk), out, 0};
  const int64_t row = V * (out_dt == DT_BF16 ? 2 : 4);
  p.vec = row % 16 == 0 && (uintptr_t)out % 16 == 0;
  return out_dt == DT_BF16 ? launch_product<__bf16>(p, s) : launch_product<float>(p, s);
}

}  // namespace ckl
