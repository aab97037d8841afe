// Host-side launchers of the device kernels (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ckl {

enum Dtype : int { DT_BF16 = 0, DT_F32 = 1 };

// Elements between two 64-row tile rows of a 64 x 64-tiled matrix with V columns.
inline int64_t tile_row_stride(int64_t V) { return ((V + 63) / 64) * 4096; }

// Copy of a row-major [rows, cols] matrix (cols % 8 == 0) into the 64 x 64
// tiled layout, tile rows tile_row_stride(cols) elements apart.
hipError_t launch_tile_copy(Dtype dt, const void* src, int64_t rows, int64_t cols, void* dst, hipStream_t s);

// With a mask, a chunk is compacted first (launch_compact) and its kernels
// take `live`: a device int, the number of valid rows, which sit at the front
// of the chunk's buffers.  Rows at and after it are skipped: no logits, zero
// gradient rows.  Without a mask `live` is null and every row is computed.

// Tables of a chunk's cached ids, built by launch_id_tables and read by the
// logits contraction, which copies the fp32 logit at every cached id out of
// its accumulators before they become exp values.
// Layout by vocabulary tile: "pair" p = slices 2p, 2p + 1 = ids 256 p .. 256 p + 255.
struct IdTables {
  const void* bits;    // [pairs][cpad][2] 128-bit masks: bit b of (p, n, h) = id 256 p + 128 h + b is cached for row n
  const void* pre;     // [pairs][cpad] two uint16: distinct cached ids of row n below ids 256 p and 256 p + 128
  int64_t cpad;        // rows of the tables: the chunk's rows rounded up to a multiple of 256
  const int32_t* rank; // [rows][K]: rank of cached id k among its row's distinct ids, -1 if outside [0, V)
  float* zs;           // [rows][K]: logit of the cached id of rank q at zs[n][q]
  int K;
};
inline int64_t id_table_pairs(int64_t V) { return (V + 255) / 256; }

// Id tables of `rows` rows of cached ids [rows, K] (cpad >= rows, a multiple
// of 256); with live (compacted chunk), rows at and past *live get empty
// tables.  Ids outside [0, V) set bit 0 of *err, an id repeated within a row
// bit 1 (err may be null); both are left out of the tables, so no kernel
// reads or writes at them.
hipError_t launch_id_tables(const int32_t* ids, int K, int64_t rows, int64_t V, const int* live, void* bits,
                            void* pre, int64_t cpad, int32_t* rank, unsigned* err, hipStream_t s);

// The recomputing backward knows each row's log-normaliser before its logits:
// the logits epilogue then stores the gradient's dense part itself.
struct GradTerms {
  const float* lse;     // [rows] log-normalisers of the chunk's rows
  const int* rowmap;    // compacted chunk: chunk row of each compacted row (lse index), or null
  const float* scale;   // device scalar 1 / n_valid
  const float* gscale;  // device scalar multiplying the gradient, or null
};

// Logits of one chunk, kept as exp values: per (row n < rows, 128-id slice s)
// the slice max m and sum of exp(z - m) into part[n][s], and exp(z - m) for
// every z = H_c[n] . W[v] into P (element type of dt, tiled, tile rows pblk
// elements apart).  With tab, the fp32 logit at every cached id also goes to
// tab->zs.  P may be null (the forward alone): no exp values are stored.
// With grad, P receives w exp(m - lse) exp(z - m) instead, exactly
// as launch_dense would leave it (w = scale (x gscale) for the rows, 0 past
// them and past V).
// W is the tiled copy of the weight (tile_row_stride(d) elements between tile rows).
hipError_t launch_logits(Dtype dt, const void* Wt, const void* Hc, int64_t V, int64_t d, int64_t rows, void* P,
                         int64_t pblk, float2* part, int n_slices, const IdTables* tab, const GradTerms* grad,
                         const int* live, hipStream_t s);

// Rows of a dH tile: the most of 256, 128 and 64 whose span in the tiled G fits the
// copies' 2 GiB (see kernels_gemm.hip).
int dh_tile_rows(Dtype dt, int64_t rows, int64_t V);
// dH partial slabs of one chunk: slab[s][n][j] = sum over the s-th vocabulary
// split of G[n][v] W[v][j].  G is tiled like P, tile rows gblk elements apart;
// Wt is the tiled copy of the weight, or the row-major weight where `tiled` is false.
hipError_t launch_dh(Dtype dt, const void* G, int64_t gblk, const void* Wt, int64_t V, int64_t d, int64_t rows,
                     float* slab, int splits, const int* live, hipStream_t s, bool tiled = true);
// dH rows = sum of the slabs in split order, rounded once to the output type.
// With pos (compacted chunk), dH row j takes slab row pos[j], or zeros if -1.
hipError_t launch_dh_reduce(Dtype dt, const float* slab, int splits, int64_t rows, int64_t d, const int* pos,
                            void* dH, hipStream_t s);
// dW (+)= G^T H_c over the rows of one chunk; beta = 0 overwrites.
hipError_t launch_dw(Dtype dt, const void* G, int64_t gblk, const void* Hc, int64_t V, int64_t d, int64_t rows,
                     float* dW, int beta, const int* live, hipStream_t s);

// k-splits used for the dH contraction of a chunk of `rows` rows.
int dh_splits(Dtype dt, int64_t rows, int64_t d, int64_t V);
// The largest split count <= s that cuts the dH k-steps into exactly that many
// runs (what launch_dh requires).
int dh_fit_splits(Dtype dt, int64_t V, int s);
// tile width used along d by the dH and dW contractions.
int d_tile(Dtype dt, int64_t d);

// Per row of x [N, V] (bf16 or fp32), the K largest values and their ids, by
// value descending and equal values by id ascending (see kernels_topk.hip).
hipError_t launch_topk(Dtype dt, const void* x, int64_t N, int64_t V, int64_t K, int32_t* ids, float* vals,
                       hipStream_t s);

// out[n] = scale W[ids[n]] (zeros for an id outside [0, V)), see kernels_embed.hip.
hipError_t launch_embed(Dtype dt, const int32_t* ids, const void* W, float scale, int64_t N, int64_t d, int64_t V,
                        void* out, hipStream_t s);
// Its workgroups, of 256 threads.
int64_t embed_blocks(Dtype dt, int64_t N, int64_t d);
// dW[v] (+)= scale x the sum of dY's rows with id v; ws of embed_bwd_workspace bytes.
uint64_t embed_bwd_workspace(int64_t N, int64_t d, int64_t V);
hipError_t launch_embed_bwd(Dtype dt, const int32_t* ids, const void* dY, float scale, int64_t N, int64_t d, int64_t V,
                            bool accumulate, float* dW, void* ws, hipStream_t s);
// Workgroups of its largest launch, in units of 256 threads.
int64_t embed_bwd_blocks(Dtype dt, int64_t N, int64_t d, int64_t V);

// Settings of a sampling call: one value for all rows, or a device array [N].
struct SampleParams {
  double temperature;
  int64_t top_k;
  double top_p, min_p;
  const float* temperatures;
  const int32_t* top_ks;
  const float* top_ps;
  const float* min_ps;
};
// A token and its log-probability per row of x (rows ld elements apart), see
// kernels_sample.hip; ws of sample_workspace bytes, or null (long rows of a
// small batch are then not split).
uint64_t sample_workspace(Dtype dt, int64_t N, int64_t V);
hipError_t launch_sample(Dtype dt, const void* x, int64_t N, int64_t V, int64_t ld, const float* u,
                         const SampleParams& p, int32_t* ids, float* logp, void* ws, hipStream_t s);

// e4m3 values and their scales: per 1 x 128 block (rows; scales [ceil(C / 128), R])
// or per 128 x 128 block (scales [ceil(R / 128), ceil(C / 128)]), see kernels_fp8.hip.
hipError_t launch_quantize_fp8(Dtype dt, const void* x, int64_t R, int64_t C, bool rows, uint8_t* q, float* scales,
                               hipStream_t s);
// out [M, V] = the product of the rows xq (1 x 128 scales) with the weight wq (128 x 128 scales).
hipError_t launch_matmul_fp8(Dtype out_dt, const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                             int64_t M, int64_t V, int64_t d, void* out, hipStream_t s);

// A dropout's draw: elements whose 16 bits (see philox in row_io.hpp) are below
// `border` go, the others are multiplied by keep = 65536 / (65536 - border).
// `at`, if not null, is a device word added to the offset when the kernel runs,
// so that a captured step can move it on.
struct Drop {
  uint64_t seed, offset;
  const int64_t* at;
  uint32_t border;  // 0: nothing is dropped; 65536: everything
  float keep;
};
// out[i] = x[i] keep or 0, i < n (out may be x), see kernels_norm.hip; its workgroups, of 256 threads.
hipError_t launch_dropout(Dtype dt, const void* x, int64_t n, const Drop& r, void* out, hipStream_t s);
int64_t dropout_blocks(int64_t n);

// The residual's norms around a block, see kernels_norm.hip.
struct NormArgs {
  const void* y;       // [N, d] the block's output
  const void* r;       // [N, d] residual
  const void* w_post;  // [d] or null: y is not normalised
  const void* w_pre;   // [d] or null: no x
  const void* gate;    // [d], or [N, d] with gate_rows, or null
  bool gate_rows;
  float scale, eps;
  Drop drop;
  int64_t N, d;
  void* r_out;            // [N, d]
  void* x;                // [N, d]
  float* stats;           // [2, N] reciprocal rms of y and of r', or null
  const float* stats_in;  // the same, of the forward call (backward)
};
struct NormGrads {
  const void* dx;     // [N, d] or null
  const void* dr_in;  // [N, d] gradient of r_out, or null
  void* dy;           // [N, d]
  void* dr;           // [N, d]
  float* dw_post;     // [d]
  float* dw_pre;      // [d]
  void* dgate;        // fp32 [d], or [N, d] in the path's type
  float* part;        // add_norm_bwd_workspace bytes
  bool a;             // set by the launcher: whether dw_post or a gate [d]'s gradient is there
  int sums;           // set by the launcher: sums a column
};
constexpr int64_t kMaxNormWidth = 16384;  // d: a row is held in one workgroup's registers
hipError_t launch_add_norm(Dtype dt, const NormArgs& p, hipStream_t s);
uint64_t add_norm_bwd_workspace(int64_t N, int64_t d, int sums);
hipError_t launch_add_norm_bwd(Dtype dt, const NormArgs& p, const NormGrads& q, hipStream_t s);

// Log-probabilities of given tokens, entropy and alternatives of rows of logits,
// and their gradient, see kernels_logprob.hip.
struct LogprobArgs {
  const void* x;        // [N, V], rows ld elements apart
  int64_t N, V, ld;
  const int32_t* ids;   // [N, T]
  int T, top;
  const uint8_t* mask;  // [N] or null
  float* logp;          // [N, T]
  float* entropy;       // [N]
  float* stats;         // [2, N]: largest logit, log of the sum of exp(z - largest)
  int32_t* top_ids;     // [N, top]
  float* top_logp;      // [N, top]
  int slices;           // of a row, `per` logits each (set by the launcher, as what follows)
  int64_t per;
  float4* part;         // [N, slices] (largest, reference, sum, weighted sum)
  void* pairs;          // [N, slices, top] 64-bit (key, id) pairs
};
uint64_t logprob_workspace(int64_t N, int64_t V, int top);
// ws of logprob_workspace bytes, or null: rows are then not split.
hipError_t launch_logprob(Dtype dt, LogprobArgs p, void* ws, hipStream_t s);

struct LogprobGradArgs {
  const void* x;           // [N, V], rows ld elements apart
  int64_t N, V, ld, ldo;
  const int32_t* ids;      // [N, T]
  int T;
  const uint8_t* mask;     // [N] or null
  const float* stats;      // [2, N]
  const float* entropy;    // [N], or null without dentropy
  const float* dlogp;      // [N, T]
  const float* dentropy;   // [N] or null
  void* out;               // [N, V], rows ldo elements apart; may be x
  int64_t runs;            // workgroups of a row (set by the launcher)
};
hipError_t launch_logprob_grad(Dtype dt, LogprobGradArgs p, hipStream_t s);
int64_t logprob_grad_blocks(int64_t N, int64_t V);  // its workgroups, of 256 threads

// The same from hidden states H [N, d] and the head's weight W [V, d], see kernels_head.hip.
struct HeadArgs {
  const void *H, *W;
  int64_t N, d, V;
  const int32_t* ids;   // [N, T]
  int T;
  const uint8_t* mask;  // [N] or null
  float* logp;          // [N, T]
  float* entropy;       // [N]
  float* stats;         // [2, N]
};
// Edge of the square tiles of a product (see kernels_head.hip).
enum HeadTile : int { TILE_256 = 0, TILE_128 = 1, TILE_64 = 2 };
// The logits product's: ids [0, main) in `tile`, the others in `rest`, by a launch of their own.
struct HeadTiling {
  HeadTile tile, rest;
  int64_t main;
};
HeadTiling head_logits_tiling(Dtype dt, int64_t rows, int64_t V, int64_t d);
int head_slices(const HeadTiling& t, int64_t V);  // slices of a row's statistics
// The slices' statistics of a chunk of rows Hc (all of them, or the *live compacted ones).
hipError_t launch_head_stats(Dtype dt, const HeadTiling& t, const HeadArgs& a, const void* Hc, int64_t rows, float2* part,
                             float* part_a, int n_slices, const int* live, hipStream_t s);
// Entropy, stats and log-probabilities of rows [r0, r0 + rows); pos: of a compacted chunk, or null.
hipError_t launch_head_rows(Dtype dt, const HeadArgs& p, int64_t r0, int64_t rows, const float2* part,
                            const float* part_a, int n_slices, const int* pos, hipStream_t s);
struct HeadGradArgs {
  int64_t N, d, V;
  const int32_t* ids;      // [N, T]
  int T;
  const float* logp;       // [N, T]
  const float* stats;      // [2, N]
  const float* entropy;    // [N], or null without dentropy
  const float* dlogp;      // [N, T]
  const float* dentropy;   // [N] or null
};
// G of a chunk (tiled, tile rows gblk elements apart); coef: [rows].
hipError_t launch_head_grad(Dtype dt, const HeadGradArgs& a, const void* W, const void* Hc, int64_t r0, int64_t rows,
                            const int* vidx, const int* live, float4* coef, void* G, int64_t gblk, hipStream_t s);
// dH's partial slabs as launch_dh leaves them, in the given tile (of at most
// dh_tile_rows rows) and splits.
struct HeadSplit {
  HeadTile tile;
  int splits;
};
HeadSplit head_dh_split(Dtype dt, int64_t rows, int64_t d, int64_t V);
hipError_t launch_head_dh(Dtype dt, const HeadSplit& h, const void* G, int64_t gblk, const void* W, int64_t V, int64_t d,
                          int64_t rows, float* slab, const int* live, hipStream_t s, bool tiled = false);
// dW: fp32 `sums` (+)= G^T H_c; or, where `rounded` is not null, that bf16 array = G^T
// H_c, plus the fp32 `old` where given (bf16 operands).
hipError_t launch_head_dw(Dtype dt, const void* G, int64_t gblk, const void* Hc, int64_t V, int64_t d, int64_t rows,
                          const float* old, float* sums, int beta, void* rounded, const int* live, hipStream_t s);

constexpr int kMaxK = 2048;
constexpr int kMaxTop = 512;  // alternatives of a row

// Valid-token count n and scale 1/n (0 if n = 0) into scal (int64 n, float s).
hipError_t launch_mask_count(const uint8_t* mask, int64_t N, void* scal, hipStream_t s);
// Compaction of the chunk whose mask, H rows, ids and teacher logits start at
// the given pointers (`rows` positions): vidx[i] = the chunk row of the i-th
// valid one, pos[j] = the compact index of row j or -1, *live = the valid
// count; masked rows' kl_out (and lse_out, if not null) are set to 0; the
// valid rows of H, ids and logits are gathered to Hc, ids_c, tl_c (chunk
// buffers of rows_alloc rows), and Hc rows [*live, next multiple of 256) are
// zeroed.
hipError_t launch_compact(Dtype dt, const uint8_t* mask, int64_t rows, int64_t rows_alloc, const void* H,
                          int64_t d, const int32_t* ids, const float* tlogit, int K, int* vidx, int* pos,
                          int* live, float* kl_out, float* lse_out, void* Hc, int32_t* ids_c, float* tl_c,
                          hipStream_t s);

// Row pass of one chunk (see kernels_rows.hip).
struct RowArgs {
  void* P;              // tiled exp values in, gradient out (element type of the path)
  int64_t pblk;         // elements between tile rows of P
  float2* part;         // per row n_slices pairs: (max, sum exp) in, (max, gradient factor) out
  int n_slices;
  const int32_t* ids;   // [rows, K]
  const float* tlogit;  // [rows, K]
  const uint8_t* mask;  // [rows] or null
  const void* scal;     // device scalars (int64 n, float s); null -> scale_value
  float scale_value;
  int64_t V;
  int K;
  int64_t rows;
  float* scat;          // [rows, K] exact gradient values at the cached ids
  const float* lse_in;  // [rows] log-normalisers saved by a forward pass, or null: merge the slice pairs
  const float* gscale;  // device scalar multiplying the gradient, or null for 1
  const int* live;      // compacted chunk: rows at and after *live are skipped; null: none
  const int* vidx;      // compacted chunk: chunk row of each compacted row (row outputs, lse_in); or null
  float* kl_out;        // [rows] KL (0 for masked rows), or null
  float* lse_out;       // [rows] log-normalisers, or null
  const int32_t* rank;  // [rows, K] rank of each cached id among its row's distinct ids (-1: outside [0, V))
  const float* zs;      // [rows, K] exact logits of the cached ids, by rank
  float* zg_dbg;        // optional [rows, K]
  int32_t* sid_dbg;     // optional [rows, K]
};
hipError_t launch_row_stats(Dtype g_dt, const RowArgs& a, hipStream_t s);
// p[0 .. n) = v (a kernel, not a memset node, so that the call stays capturable)
hipError_t launch_fill_f32(float* p, int64_t n, float v, hipStream_t s);
hipError_t launch_dense(Dtype g_dt, const RowArgs& a, hipStream_t s);
hipError_t launch_scatter(Dtype g_dt, const RowArgs& a, hipStream_t s);

// Debug helpers: slice pairs and tiled exp values of caller-given fp32 logits
// (row stride ldz); and a tiled matrix copied out to row-major [rows, V].
hipError_t launch_partials_from_z(Dtype g_dt, const float* Z, int64_t ldz, int64_t rows, int64_t V, float2* part,
                                  int n_slices, void* P, int64_t pblk, hipStream_t s);
// Debug helper: zs[r][rank[r][k]] = Z[r][ids[r][k]] for the ids of the table.
hipError_t launch_zs_from_z(const float* Z, int64_t ldz, const int32_t* ids, const int32_t* rank, int64_t rows, int K,
                            float* zs, hipStream_t s);
hipError_t launch_untile(Dtype g_dt, const void* P, int64_t pblk, int64_t rows, int64_t V, void* out,
                         hipStream_t s);

// loss = s * sum of kl[0..N) in a fixed order, accumulated in double.
hipError_t launch_finalize(const float* kl, int64_t N, const void* scal, float* out_loss, hipStream_t s);

// byte offsets, in the device scalar block, of the gradient weight 1 / n_valid
// (fp32) and of the input-check flags (bit 0: a cached id outside [0, V);
// bit 1: an id repeated within a row)
constexpr int kScaleOffset = 8;
constexpr int kErrOffset = 16;

}  // namespace ckl
