// Internal launch interface of routed experts as operators of their own: the
// router, the products grouped by expert, and the products with 4-bit weights.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mok.h"

namespace mok {

// ---------------------------------------------------------------- router
struct RouteArgs {
  const void* logits;    // [T][E]
  const float* bias;     // [E] or NULL: added to the scores for the choice alone
  long long T;
  int E, k;
  int sigmoid, normalize;
  float scale;
  int64_t* experts;      // [T][k]
  float* weights;        // [T][k]
  float* lse;            // [T]
  // with the loads and mean scores (both or neither)
  int* counts;           // [E]
  float* mean_score;     // [E]
  float* part;           // [route_blocks][E] sums of scores, then [route_blocks][E] counts
};
struct RouteBwdArgs {
  const float* d_weights;  // [T][k]
  const void* logits;
  const int64_t* experts;
  const float* d_lse;         // [T] or NULL
  const float* d_mean_score;  // [E] or NULL
  void* d_logits;             // in the logits' type
  long long T;
  int E, k;
  int sigmoid, normalize;
  float scale;
};
int route_blocks(long long T, int E);
cudaError_t launch_route(const RouteArgs& a, int f32, cudaStream_t st);
cudaError_t launch_route_bwd(const RouteBwdArgs& a, int f32, cudaStream_t st);

// ---------------------------------------------------------------- 4-bit weights
// The layout of a matrix [N][K] (int4.cu): N in tiles of 16 rows, K in blocks of
// 128, both padded.
constexpr int kInt4Rows = 16, kInt4Block = 128;
constexpr int kInt4TileBytes = kInt4Rows * kInt4Block / 2;
struct Int4Shape {
  long long matrices;
  int N, K, group;
  __host__ __device__ long long row_tiles() const { return (static_cast<long long>(N) + kInt4Rows - 1) / kInt4Rows; }
  __host__ __device__ int blocks() const { return (K + kInt4Block - 1) / kInt4Block; }
  __host__ __device__ long long tiles() const { return matrices * row_tiles() * blocks(); }
  // scales (and zeros) of a tile: [16 rows][groups of a block]
  __host__ __device__ int tile_scales() const { return kInt4Rows * (kInt4Block / group); }
};
struct Int4LinearArgs {
  Int4Shape w;
  const uint8_t* codes;
  const uint16_t* scales;
  const uint8_t* zeros;      // or NULL: 8
  const uint16_t* x;
  const int64_t* experts;    // [rows] or NULL
  const void* bias;          // [matrices][N] or NULL
  void* y;                   // [rows][N]
  int rows;                  // of y
  int x_div;                 // row r of y reads row r / x_div of x
  int by_expert;             // (the launch's: a block to an expert, not to a row)
  int act;
  int out_f32, bias_f32;
  int* status;
};
cudaError_t launch_int4_quantize(const void* w, int f32, const Int4Shape& s, uint8_t* codes, uint16_t* scales, uint8_t* zeros,
                                 cudaStream_t st);
cudaError_t launch_int4_pack(const uint8_t* q, const uint16_t* qs, const uint8_t* qz, const Int4Shape& s, uint8_t* codes,
                             uint16_t* scales, uint8_t* zeros, cudaStream_t st);
cudaError_t launch_int4_dequantize(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, const Int4Shape& s,
                                   uint16_t* out, cudaStream_t st);
cudaError_t launch_int4_linear(const Int4LinearArgs& a, int num_sms, cudaStream_t st);
// The same for one matrix, by the tensor core of int4_tc.cu.
mok_status_t run_int4_tc(const Int4LinearArgs& a, cudaStream_t st);

// ---------------------------------------------------------------- products grouped by expert
constexpr int kMaxGroups = MOK_GROUPED_MAX_E;
// The products of grouped.cuh's rows kernel: the forward, and dx.
struct GroupedRowsParams {
  const int* counts;     // [E]
  int E;
  int L;                 // the output's contiguous length
  int M;                 // its rows
  int nk;                // K-blocks of 64
  int l_tiles;           // tiles of 256
  int act;
  const void* bias;      // [E][L] or NULL
  int bias_f32;
  void* out;             // [M][L]
  uint16_t* z;           // [M][L] bf16 or NULL
  // The kernel before it on the stream is grouped_weight_kernel, none of whose results this one reads: it starts as that
  // one's CTAs leave, without a wait, and waits for it at its end.  Right behind that kernel alone, each of whose CTAs waits
  // for all before it and only then lets the next kernel start: behind one that does so earlier, or that is not there, x
  // (dz) would be read before the pass that writes it has ended.
  int beside_last;
  int* status;
};
struct GroupedRowsCall {
  const uint16_t* w;     // [E][L][K], or [E][K][L] with w_mn
  const uint16_t* x;     // [M][K]
  int K;
  bool w_mn, out_f32;
};
mok_status_t run_grouped_rows(const GroupedRowsCall& c, const GroupedRowsParams& p, cudaStream_t st);

// The weight gradients: [E][N][K] from dz [M][N] and x [M][K].
struct GroupedWeightCall {
  const uint16_t* dz;
  const uint16_t* x;
  const int* counts;
  int E, M, N, K;
  uint16_t* out;
  int* status;
};
// The bias's gradient [E][N] from the sums of dz over each chunk of rows inside
// each group: part [grouped_dz_parts][N], out NULL for none.
struct GroupedBias {
  const float* part;
  float* out;
  int chunk;
};
// Part of the backward's workspace: the groups' first rows ([E + 1], 16-byte
// multiple) and two tensor maps for each.
size_t grouped_plan_bytes(int E);

// The backward's first pass: the plan, with the groups' maps of dz and x where
// `maps`; and where dz or part is wanted, dz = dy act'(z) in bf16 for the groups'
// rows, and the sums of its fp32 values over each chunk of rows inside each group.
struct GroupedDzCall {
  const void* dy;
  int dy_f32;
  const uint16_t* z;
  int act;
  uint16_t* dz;       // or NULL
  float* part;        // or NULL
};
int grouped_dz_chunk(int M, int N);   // rows of a chunk
inline long long grouped_dz_parts(int M, int N, int E) { return (static_cast<long long>(M) + grouped_dz_chunk(M, N) - 1) / grouped_dz_chunk(M, N) + E; }
mok_status_t run_grouped_dz(const GroupedWeightCall& c, const GroupedDzCall& d, bool maps, void* plan, cudaStream_t st);
mok_status_t run_grouped_weights(const GroupedWeightCall& c, const void* plan, const GroupedBias& bias, cudaStream_t st);
cudaError_t launch_grouped_bias(const GroupedBias& b, const void* plan, int E, int N, cudaStream_t st);

}  // namespace mok
