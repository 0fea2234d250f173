// Launches of the products grouped by expert (grouped.cuh): operand maps, the
// groups' plan, and the elementwise pass of the backward.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "api_util.h"
#include "clusters.h"
#include "grouped.cuh"
#include "internal.h"

namespace mok {
namespace {

// [planes][outer][inner] of bf16 with boxes of one plane, zeros outside; the
// box's inner bytes (64 or 128) are the swizzle.  planes 0: [outer][inner].
mok_status_t make_map(CUtensorMap* m, const void* base, long long inner, long long outer, long long planes, int box_inner, int box_outer) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(MOK_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer), static_cast<cuuint64_t>(planes)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(inner) * 2, static_cast<cuuint64_t>(inner) * outer * 2};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_outer), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, planes ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, box_inner == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(MOK_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d) for [%lld x %lld x %lld]", static_cast<int>(r), planes, outer, inner);
  return MOK_OK;
}

template <bool AMN, bool F32>
mok_status_t launch_rows(const GroupedRowsMaps& maps, const GroupedRowsParams& p, cudaStream_t st) {
  auto kern = grouped_rows_kernel<AMN, F32>;
  static KernelInfo info;
  int n = 0;
  MOK_CUDA(resident_clusters(kern, info, kGroupedThreads, GroupedRowsCfg::kSmemBytes, 2, &n));
  const long long items = (static_cast<long long>(p.M) / 256 + (p.E < p.M ? p.E : p.M)) * p.l_tiles;   // at most
  const int pairs = items < n ? static_cast<int>(items) : n;
  MOK_CUDA(launch_clusters(kern, dim3(2 * pairs), kGroupedThreads, GroupedRowsCfg::kSmemBytes, 2, st, maps, p));
  return MOK_OK;
}

// ---------------------------------------------------------------- plan
struct PlanMaps {
  CUtensorMap dz, x;
};
constexpr size_t plan_starts_bytes(int E) { return (static_cast<size_t>(E + 1) * sizeof(int) + 127) / 128 * 128; }

// One block: the groups' first rows; and each group's maps, which are the whole
// tensors' but for their length, which is the group's end.
__global__ void __launch_bounds__(1024) grouped_plan_kernel(const __grid_constant__ PlanMaps whole, const int* counts, int E, int M, int* starts,
                                                            CUtensorMap* dz, CUtensorMap* x, int* status) {
  __shared__ int start[kMaxGroups + 1];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    const bool bad = scan_groups(counts, E, M, start, nullptr, lane);
    if (bad && lane == 0) atomicCAS(status, 0, MOK_ERR_INDEX);
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += blockDim.x) starts[e] = start[e];
  if (!dz) return;
  for (int i = threadIdx.x; i < 2 * E; i += blockDim.x) {
    const int e = i >> 1;
    const uint4* from = reinterpret_cast<const uint4*>(i & 1 ? &whole.x : &whole.dz);
    CUtensorMap* to = (i & 1 ? x : dz) + e;
#pragma unroll
    for (int j = 0; j < 8; ++j) reinterpret_cast<uint4*>(to)[j] = from[j];
    const uint32_t rows = max(start[e + 1], 1);   // (a group that begins and ends at 0 is never read)
    asm volatile("tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 1, %1;" ::"l"(reinterpret_cast<uint64_t>(to)), "r"(rows) : "memory");
  }
  asm volatile("fence.proxy.tensormap::generic.release.gpu;" ::: "memory");
}

// ---------------------------------------------------------------- dz
constexpr int kDzRows = 8;   // rows in step in a block; 32 threads x 8 columns wide

// Chunks of rows are cut without regard to the groups; part[chunk + e] holds the
// sums over the rows of group e in a chunk: from one pair (chunk, e) to the next
// at least one of the two grows, so that no two share a place.
template <class DY, int ACT>
__global__ void __launch_bounds__(256) grouped_dz_kernel(const DY* __restrict__ dy, const uint16_t* __restrict__ z,
                                                         const int* __restrict__ starts, int E, int N, int chunk,
                                                         uint16_t* __restrict__ dz, float* __restrict__ part) {
  __shared__ float s[kDzRows][32][9];
  griddep_wait();
  griddep_launch_dependents();
  const int col = (blockIdx.x * 32 + threadIdx.x) * 8;
  int r0 = blockIdx.y * chunk;
  const int r1 = min(r0 + chunk, __ldg(starts + E));
  if (r0 >= r1) return;
  for (int e = find_group(starts, E, r0, threadIdx.x); r0 < r1; ++e) {
    const int end = min(__ldg(starts + e + 1), r1);
    if (end <= r0) continue;   // an empty group
    float sum[8] = {};
    if (col < N) {
      for (int r = r0 + threadIdx.y; r < end; r += kDzRows) {
        const long long at = static_cast<long long>(r) * N + col;
        float d[8];
        if constexpr (sizeof(DY) == 4) {
          const float4 a = __ldcs(reinterpret_cast<const float4*>(dy + at));
          const float4 b = __ldcs(reinterpret_cast<const float4*>(dy + at) + 1);
          d[0] = a.x, d[1] = a.y, d[2] = a.z, d[3] = a.w, d[4] = b.x, d[5] = b.y, d[6] = b.z, d[7] = b.w;
        } else {
          const uint4 a = __ldcs(reinterpret_cast<const uint4*>(dy + at));
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = bf16_at(&a, i);
        }
        if constexpr (ACT != LIN_NONE) {
          const uint4 a = __ldcs(reinterpret_cast<const uint4*>(z + at));
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] *= act_slope<ACT>(bf16_at(&a, i));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += d[i];
        if (dz)   // read again at once by the products: kept in L2
          *reinterpret_cast<uint4*>(dz + at) =
              make_uint4(pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]), pack_bf16(d[4], d[5]), pack_bf16(d[6], d[7]));
      }
    }
    r0 = end;
    if (!part) continue;
    __syncthreads();   // the last group's sums have been read
#pragma unroll
    for (int i = 0; i < 8; ++i) s[threadIdx.y][threadIdx.x][i] = sum[i];
    __syncthreads();
    const int t = threadIdx.y * 32 + threadIdx.x, c = t >> 3, i = t & 7;   // one column per thread
    float v = 0.f;
#pragma unroll
    for (int r = 0; r < kDzRows; ++r) v += s[r][c][i];
    const int out = (blockIdx.x * 32 + c) * 8 + i;
    if (out < N) part[(static_cast<long long>(blockIdx.y) + e) * N + out] = v;
  }
}

// A group's parts in order: 32 columns a block, 8 parts in step.
__global__ void __launch_bounds__(256) grouped_bias_kernel(const float* __restrict__ part, const int* __restrict__ starts, int N, int chunk,
                                                           float* __restrict__ d_bias) {
  __shared__ float s[8][33];
  griddep_wait();
  griddep_launch_dependents();
  const int e = blockIdx.y, col = blockIdx.x * 32 + threadIdx.x;
  const int r0 = __ldg(starts + e), r1 = __ldg(starts + e + 1);
  float v = 0.f;
  if (col < N && r0 < r1) {
    const int last = (r1 - 1) / chunk;
#pragma unroll 4
    for (int c = r0 / chunk + threadIdx.y; c <= last; c += 8) v += part[(static_cast<long long>(c) + e) * N + col];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && col < N) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += s[i][threadIdx.x];
    d_bias[static_cast<long long>(e) * N + col] = v;
  }
}

template <class DY>
cudaError_t dz_launch(const DY* dy, const uint16_t* z, int act, const int* starts, int E, int M, int N, uint16_t* dz, float* part,
                      cudaStream_t st) {
  const int chunk = grouped_dz_chunk(M, N);
  const dim3 grid((N + 255) / 256, (M + chunk - 1) / chunk), block(32, kDzRows);
  switch (act) {
    case LIN_RELU: return launch_dependent(grouped_dz_kernel<DY, LIN_RELU>, grid, block, 0, st, dy, z, starts, E, N, chunk, dz, part);
    case LIN_SILU: return launch_dependent(grouped_dz_kernel<DY, LIN_SILU>, grid, block, 0, st, dy, z, starts, E, N, chunk, dz, part);
    case LIN_GELU: return launch_dependent(grouped_dz_kernel<DY, LIN_GELU>, grid, block, 0, st, dy, z, starts, E, N, chunk, dz, part);
    case LIN_GELU_TANH:
      return launch_dependent(grouped_dz_kernel<DY, LIN_GELU_TANH>, grid, block, 0, st, dy, z, starts, E, N, chunk, dz, part);
    default: return launch_dependent(grouped_dz_kernel<DY, LIN_NONE>, grid, block, 0, st, dy, z, starts, E, N, chunk, dz, part);
  }
}

}  // namespace

mok_status_t run_grouped_rows(const GroupedRowsCall& c, const GroupedRowsParams& q, cudaStream_t st) {
  GroupedRowsParams p = q;
  p.nk = (c.K + kLinBK - 1) / kLinBK;
  p.l_tiles = (p.L + 255) / 256;
  if ((static_cast<long long>(p.M) / 256 + p.E) * p.l_tiles > 0x7fffffffll / 4) return fail(MOK_ERR_INVALID_ARG, "product too large");
  GroupedRowsMaps maps;
  mok_status_t s = c.w_mn ? make_map(&maps.w, c.w, p.L, c.K, p.E, 64, 64) : make_map(&maps.w, c.w, c.K, p.L, p.E, 64, 128);
  for (int b = 0; !s && b < 4; ++b) s = make_map(&maps.x[b], c.x, c.K, p.M, 0, 64, 16 << b);
  if (s) return s;
  if (c.w_mn) return launch_rows<true, false>(maps, p, st);
  return c.out_f32 ? launch_rows<false, true>(maps, p, st) : launch_rows<false, false>(maps, p, st);
}

size_t grouped_plan_bytes(int E) { return plan_starts_bytes(E) + 2 * static_cast<size_t>(E) * sizeof(CUtensorMap); }

mok_status_t launch_grouped_plan(const GroupedWeightCall& c, bool maps, void* plan, cudaStream_t st) {
  PlanMaps whole = {};
  CUtensorMap *dz = nullptr, *x = nullptr;
  if (maps) {
    mok_status_t s = make_map(&whole.dz, c.dz, c.N, c.M, 0, 64, 64);
    if (!s) s = make_map(&whole.x, c.x, c.K, c.M, 0, 64, 64);
    if (s) return s;
    dz = reinterpret_cast<CUtensorMap*>(static_cast<uint8_t*>(plan) + plan_starts_bytes(c.E));
    x = dz + c.E;
  }
  MOK_CUDA(launch_dependent(grouped_plan_kernel, dim3(1), dim3(1024), 0, st, whole, c.counts, c.E, c.M, static_cast<int*>(plan), dz, x,
                            c.status));
  return MOK_OK;
}

mok_status_t run_grouped_weights(const GroupedWeightCall& c, const void* plan, cudaStream_t st) {
  GroupedWeightParams p = {};
  p.starts = static_cast<const int*>(plan);
  p.dz = reinterpret_cast<const CUtensorMap*>(static_cast<const uint8_t*>(plan) + plan_starts_bytes(c.E));
  p.x = p.dz + c.E;
  p.E = c.E;
  p.N = c.N;
  p.K = c.K;
  p.n_tiles = (c.N + 255) / 256;
  p.k_tiles = (c.K + 255) / 256;
  p.status = c.status;
  const long long items = static_cast<long long>(p.E) * p.n_tiles * p.k_tiles;
  if (items > 0x7fffffffll / 4) return fail(MOK_ERR_INVALID_ARG, "product too large");
  GroupedWeightMaps maps;
  const mok_status_t s = make_map(&maps.out, c.out, c.K, c.N, c.E, 32, 32);
  if (s) return s;
  static KernelInfo info;
  int n = 0;
  MOK_CUDA(resident_clusters(grouped_weight_kernel, info, kGroupedThreads, GroupedWeightCfg::kSmemBytes, 2, &n));
  const int pairs = items < n ? static_cast<int>(items) : n;
  MOK_CUDA(launch_clusters(grouped_weight_kernel, dim3(2 * pairs), kGroupedThreads, GroupedWeightCfg::kSmemBytes, 2, st, maps, p));
  return MOK_OK;
}

int grouped_dz_chunk(int M, int N) {
  // about 8 blocks for each of 152 SMs, a chunk no shorter than 4 steps
  const int cols = (N + 255) / 256, want = (1216 + cols - 1) / cols;
  const int rows = ((M + want - 1) / want + kDzRows - 1) / kDzRows * kDzRows;
  return rows < 4 * kDzRows ? 4 * kDzRows : rows;
}

cudaError_t launch_grouped_dz(const void* dy, int dy_f32, const uint16_t* z, int act, const int* starts, int E, int M, int N,
                              uint16_t* dz, float* part, cudaStream_t st) {
  return dy_f32 ? dz_launch(static_cast<const float*>(dy), z, act, starts, E, M, N, dz, part, st)
                : dz_launch(static_cast<const uint16_t*>(dy), z, act, starts, E, M, N, dz, part, st);
}

cudaError_t launch_grouped_bias(const float* part, const int* starts, int E, int M, int N, float* d_bias, cudaStream_t st) {
  return launch_dependent(grouped_bias_kernel, dim3((N + 31) / 32, E), dim3(32, 8), 0, st, part, starts, N, grouped_dz_chunk(M, N),
                          d_bias);
}

}  // namespace mok
