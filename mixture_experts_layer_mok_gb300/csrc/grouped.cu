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
  using C = GroupedRowsCfg<F32>;
  auto kern = grouped_rows_kernel<AMN, F32>;
  static KernelInfo info;
  int n = 0;
  MOK_CUDA(resident_clusters(kern, info, C::kThreads, C::kSmemBytes, 2, &n));
  // at most, and with tiles in as many parts as they have 64 rows
  const long long items = (static_cast<long long>(p.M) / 256 + static_cast<long long>(p.M) / 64 + (p.E < p.M ? p.E : p.M)) * p.l_tiles;
  const int pairs = items < n ? static_cast<int>(items) : n;
  MOK_CUDA(launch_clusters(kern, dim3(2 * pairs), C::kThreads, C::kSmemBytes, 2, st, maps, p));
  return MOK_OK;
}

// ---------------------------------------------------------------- plan and dz
struct Plan {
  CUtensorMap dz, x;   // of the whole tensors
  const int* counts;
  int E, M;
  int* starts;
  CUtensorMap *to_dz, *to_x;   // or NULL
  int* status;
};
constexpr size_t plan_starts_bytes(int E) { return (static_cast<size_t>(E + 1) * sizeof(int) + 127) / 128 * 128; }

// By a block: the groups' first rows into start (shared memory), and by one that
// is to `write` them, the plan: each group's maps are the whole tensors' but for
// their length, which is the group's end.
__device__ __forceinline__ void make_plan(const Plan& p, int* start, bool write, int thread, int threads) {
  if (thread < 32) {
    const bool bad = scan_groups(p.counts, p.E, p.M, start, nullptr, thread);
    if (bad && write && thread == 0) atomicCAS(p.status, 0, MOK_ERR_INDEX);
  }
  __syncthreads();
  if (!write) return;
  for (int e = thread; e <= p.E; e += threads) p.starts[e] = start[e];
  if (!p.to_dz) return;
  for (int i = thread; i < 2 * p.E; i += threads) {
    const int e = i >> 1;
    const uint4* from = reinterpret_cast<const uint4*>(i & 1 ? &p.x : &p.dz);
    CUtensorMap* to = (i & 1 ? p.to_x : p.to_dz) + e;
#pragma unroll
    for (int j = 0; j < 8; ++j) reinterpret_cast<uint4*>(to)[j] = from[j];
    const uint32_t rows = max(start[e + 1], 1);   // (a group that begins and ends at 0 is never read)
    asm volatile("tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 1, %1;" ::"l"(reinterpret_cast<uint64_t>(to)), "r"(rows) : "memory");
  }
  asm volatile("fence.proxy.tensormap::generic.release.gpu;" ::: "memory");
}

// The plan alone, by one block.
__global__ void __launch_bounds__(1024) grouped_plan_kernel(const __grid_constant__ Plan plan) {
  __shared__ int start[kMaxGroups + 1];
  griddep_wait();
  griddep_launch_dependents();
  make_plan(plan, start, true, threadIdx.x, blockDim.x);
}

constexpr int kDzRows = 8;   // rows in step in a block; 32 threads x 8 columns wide

// One row's 8 columns at `at`: dy act'(z).
template <class DY, int ACT>
struct DzPiece {
  uint4 dy[sizeof(DY) == 4 ? 2 : 1], z;
  __device__ __forceinline__ void load(const DY* __restrict__ d, const uint16_t* __restrict__ zp, long long at) {
    dy[0] = __ldcs(reinterpret_cast<const uint4*>(d + at));
    if constexpr (sizeof(DY) == 4) dy[1] = __ldcs(reinterpret_cast<const uint4*>(d + at) + 1);
    if constexpr (ACT != LIN_NONE) z = __ldcs(reinterpret_cast<const uint4*>(zp + at));
  }
  __device__ __forceinline__ void value(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = sizeof(DY) == 4 ? __uint_as_float(reinterpret_cast<const uint32_t*>(dy)[i]) : bf16_at(dy, i);
      if constexpr (ACT != LIN_NONE) v[i] *= act_slope<ACT>(bf16_at(&z, i));
    }
  }
};

// Chunks of rows are cut without regard to the groups; part[chunk + e] holds the
// sums over the rows of group e in a chunk: from one pair (chunk, e) to the next
// at least one of the two grows, so that no two share a place.  The first block
// also writes the plan.
// dz goes to the tensor core's products, whose operands are bf16: one rounding more
// than the formula in 32 bits has (2.3e-3 of relative error in dx and d_weight for
// 1.7e-3), as in the dense projection.  The sums are of the unrounded values.
// Bound by memory: 201 MB of 32768 x 1024, two of three read, take 30 us.
template <class DY, int ACT>
__global__ void __launch_bounds__(256) grouped_dz_kernel(const __grid_constant__ Plan plan, const DY* __restrict__ dy,
                                                         const uint16_t* __restrict__ z, int N, int chunk, uint16_t* __restrict__ dz,
                                                         float* __restrict__ part) {
  __shared__ int start[kMaxGroups + 1];
  __shared__ float s[kDzRows][32][9];
  griddep_wait();
  griddep_launch_dependents();
  make_plan(plan, start, blockIdx.x == 0 && blockIdx.y == 0, threadIdx.y * 32 + threadIdx.x, 256);
  const int E = plan.E, col = (blockIdx.x * 32 + threadIdx.x) * 8;
  int r0 = blockIdx.y * chunk;
  const int r1 = r0 + min(chunk, start[E] - r0);   // (r0 + chunk may pass 2^31)
  if (r0 >= r1) return;
  for (int e = part ? find_group(start, E, r0, threadIdx.x) : 0; r0 < r1; ++e) {
    const int end = part ? min(start[e + 1], r1) : r1;   // without sums the groups do not matter
    if (end <= r0) continue;   // an empty group
    float sum[8] = {};
    if (col < N) {
      constexpr int kAtOnce = 4;   // rows whose loads are in flight together
      for (int r = r0 + threadIdx.y; r < end; r += kAtOnce * kDzRows) {
        DzPiece<DY, ACT> in[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) in[u].load(dy, z, static_cast<long long>(min(r + u * kDzRows, end - 1)) * N + col);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          if (r + u * kDzRows >= end) break;
          float d[8];
          in[u].value(d);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] += d[i];
          if (dz)   // read again at once by the products: kept in L2
            *reinterpret_cast<uint4*>(dz + static_cast<long long>(r + u * kDzRows) * N + col) =
                make_uint4(pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]), pack_bf16(d[4], d[5]), pack_bf16(d[6], d[7]));
        }
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

__global__ void __launch_bounds__(256) grouped_bias_kernel(const GroupedBias b, const int* starts, int E, int N) {
  griddep_wait();
  griddep_launch_dependents();
  grouped_bias_sums(b, starts, E, N, static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x,
                    static_cast<long long>(gridDim.x) * blockDim.x);
}

template <class DY>
cudaError_t dz_launch(const Plan& plan, const GroupedDzCall& d, int N, cudaStream_t st) {
  const DY* dy = static_cast<const DY*>(d.dy);
  const int chunk = grouped_dz_chunk(plan.M, N);
  const dim3 grid((N + 255) / 256, (plan.M - 1) / chunk + 1), block(32, kDzRows);
  const auto launch = [&](auto kern) { return launch_dependent(kern, grid, block, 0, st, plan, dy, d.z, N, chunk, d.dz, d.part); };
  switch (d.act) {
    case LIN_RELU: return launch(grouped_dz_kernel<DY, LIN_RELU>);
    case LIN_SILU: return launch(grouped_dz_kernel<DY, LIN_SILU>);
    case LIN_GELU: return launch(grouped_dz_kernel<DY, LIN_GELU>);
    case LIN_GELU_TANH: return launch(grouped_dz_kernel<DY, LIN_GELU_TANH>);
    default: return launch(grouped_dz_kernel<DY, LIN_NONE>);
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

mok_status_t run_grouped_dz(const GroupedWeightCall& c, const GroupedDzCall& d, bool maps, void* at, cudaStream_t st) {
  Plan plan = {};
  if (maps) {
    mok_status_t s = make_map(&plan.dz, c.dz, c.N, c.M, 0, 64, 64);
    if (!s) s = make_map(&plan.x, c.x, c.K, c.M, 0, 64, 64);
    if (s) return s;
    plan.to_dz = reinterpret_cast<CUtensorMap*>(static_cast<uint8_t*>(at) + plan_starts_bytes(c.E));
    plan.to_x = plan.to_dz + c.E;
  }
  plan.counts = c.counts;
  plan.E = c.E;
  plan.M = c.M;
  plan.starts = static_cast<int*>(at);
  plan.status = c.status;
  if (!d.dz && !d.part)
    MOK_CUDA(launch_dependent(grouped_plan_kernel, dim3(1), dim3(1024), 0, st, plan));
  else
    MOK_CUDA(d.dy_f32 ? dz_launch<float>(plan, d, c.N, st) : dz_launch<uint16_t>(plan, d, c.N, st));
  return MOK_OK;
}

mok_status_t run_grouped_weights(const GroupedWeightCall& c, const void* plan, const GroupedBias& bias, cudaStream_t st) {
  using C = GroupedWeightCfg;
  GroupedWeightParams p = {};
  p.starts = static_cast<const int*>(plan);
  p.dz = reinterpret_cast<const CUtensorMap*>(static_cast<const uint8_t*>(plan) + plan_starts_bytes(c.E));
  p.x = p.dz + c.E;
  p.E = c.E;
  p.N = c.N;
  p.K = c.K;
  p.n_tiles = (c.N + 255) / 256;
  p.k_tiles = (c.K + 255) / 256;
  p.bias = bias;
  p.status = c.status;
  const long long items = static_cast<long long>(p.E) * p.n_tiles * p.k_tiles;
  if (items > 0x7fffffffll / 4) return fail(MOK_ERR_INVALID_ARG, "product too large");
  GroupedWeightMaps maps;
  const mok_status_t s = make_map(&maps.out, c.out, c.K, c.N, c.E, 64, 32);
  if (s) return s;
  static KernelInfo info;
  int n = 0;
  MOK_CUDA(resident_clusters(grouped_weight_kernel, info, C::kThreads, C::kSmemBytes, 2, &n));
  const int pairs = items < n ? static_cast<int>(items) : n;
  MOK_CUDA(launch_clusters(grouped_weight_kernel, dim3(2 * pairs), C::kThreads, C::kSmemBytes, 2, st, maps, p));
  return MOK_OK;
}

int grouped_dz_chunk(int M, int N) {
  // about 8 blocks for each of 152 SMs, a chunk no shorter than 4 steps
  const int cols = (N + 255) / 256, want = (1216 + cols - 1) / cols;
  const long long rows = ((static_cast<long long>(M) + want - 1) / want + kDzRows - 1) / kDzRows * kDzRows;
  return rows < 4 * kDzRows ? 4 * kDzRows : static_cast<int>(rows);
}

cudaError_t launch_grouped_bias(const GroupedBias& b, const void* plan, int E, int N, cudaStream_t st) {
  const long long blocks = (static_cast<long long>(E) * N + 255) / 256;
  return launch_dependent(grouped_bias_kernel, dim3(static_cast<unsigned>(blocks < 4864 ? blocks : 4864)), dim3(256), 0, st, b,
                          static_cast<const int*>(plan), E, N);
}

}  // namespace mok
