// Launches of the dense products (linear.cuh): operand maps, the choice of
// kernel and tile, and the elementwise pass of the backward.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "api_util.h"
#include "clusters.h"
#include "internal.h"
#include "linear.cuh"

namespace mok {
namespace {

// [outer][inner] of bf16 or fp32 with a box of box_outer rows x box_inner
// elements, whose bytes (64 or 128) are the swizzle; zeros outside.
mok_status_t make_box(CUtensorMap* m, const void* base, int f32, long long inner, long long outer, int box_inner, int box_outer) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(MOK_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const int size = f32 ? 4 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(inner) * size};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_outer)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                        const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        box_inner * size == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(MOK_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d) for [%lld x %lld]", static_cast<int>(r), outer, inner);
  return MOK_OK;
}

mok_status_t operand_map(CUtensorMap* m, const void* base, long long inner, long long outer, int box_outer) {
  return make_box(m, base, 0, inner, outer, 64, box_outer);
}

__device__ int g_linear_status;   // first error since the last read

// The largest split of K, in powers of two, whose clusters are all resident
// and whose CTAs each have at least four K-blocks.
template <class K>
cudaError_t choose_split(K kern, KernelInfo& info, int threads, int smem, long long tiles, LinearParams& p) {
  p.split = 1;
  int n = 0;
  cudaError_t err = resident_clusters(kern, info, threads, smem, 1, &n);
  for (int s = 2; err == cudaSuccess && s <= 8 && p.nk / s >= 4; s *= 2) {
    err = resident_clusters(kern, info, threads, smem, s, &n);
    if (tiles > n) break;
    p.split = s;
  }
  return err;
}

// Whether the longest of the split's ranges of K is summed in chunks.
bool needs_chunks(const LinearParams& p) { return p.out_f32 && (p.nk + p.split - 1) / p.split > 2 * kChunk; }

template <bool AMN, bool BMN, int BN, bool FWD>
cudaError_t launch_split(const LinearMaps& maps, LinearParams& p, cudaStream_t st) {
  using C = SplitCfg<AMN, BMN, BN>;
  const long long lt = (p.L + 127) / 128, ct = (static_cast<long long>(p.C) + BN - 1) / BN;
  const auto launch = [&](auto kern) {
    return launch_clusters(kern, dim3(static_cast<unsigned>(lt * p.split), static_cast<unsigned>(ct)), C::kThreads, C::kSmemBytes,
                           p.split, st, maps, p);
  };
  auto kern = linear_split_kernel<AMN, BMN, BN, FWD, false>;
  static KernelInfo info;
  cudaError_t err = choose_split(kern, info, C::kThreads, C::kSmemBytes, lt * ct, p);
  if (err != cudaSuccess) return err;
  if constexpr (FWD) {
    if (needs_chunks(p)) {
      auto chunked = linear_split_kernel<AMN, BMN, BN, FWD, true>;
      static KernelInfo chunked_info;
      err = choose_split(chunked, chunked_info, C::kThreads, C::kSmemBytes, lt * ct, p);
      return err != cudaSuccess ? err : launch(chunked);
    }
  }
  return launch(kern);
}

// The largest number of pairs along K, likewise.
template <class K>
cudaError_t choose_pairs(K kern, KernelInfo& info, int threads, int smem, LinearParams& p) {
  p.split = 1;
  int n = 0;
  cudaError_t err = resident_clusters(kern, info, threads, smem, 2, &n);
  for (int s = 2; err == cudaSuccess && s <= 4 && p.nk / s >= 4; ++s) {
    err = resident_clusters(kern, info, threads, smem, 2 * s, &n);
    if (p.l_tiles * p.c_tiles > n) break;
    p.split = s;
  }
  return err;
}

template <bool AMN, bool BMN, bool FWD>
cudaError_t launch_pair_split(const LinearMaps& maps, LinearParams& p, cudaStream_t st) {
  using C = PairSplitCfg<AMN, BMN>;
  const auto launch = [&](auto kern) {
    return launch_clusters(kern, dim3(static_cast<unsigned>(2 * p.split * p.l_tiles * p.c_tiles)), C::kThreads, C::kSmemBytes,
                           2 * p.split, st, maps, p);
  };
  auto kern = linear_pair_split_kernel<AMN, BMN, FWD, false>;
  static KernelInfo info;
  cudaError_t err = choose_pairs(kern, info, C::kThreads, C::kSmemBytes, p);
  if (err != cudaSuccess) return err;
  if constexpr (FWD) {
    if (needs_chunks(p)) {
      auto chunked = linear_pair_split_kernel<AMN, BMN, FWD, true>;
      static KernelInfo chunked_info;
      err = choose_pairs(chunked, chunked_info, C::kThreads, C::kSmemBytes, p);
      return err != cudaSuccess ? err : launch(chunked);
    }
  }
  return launch(kern);
}

template <int KIND>
cudaError_t launch_pair(PairJob& job, cudaStream_t st) {
  using C = PairKindCfg<KIND>;
  auto kern = linear_pair_kernel<KIND>;
  static KernelInfo info;
  int n = 0;
  const cudaError_t err = resident_clusters(kern, info, C::kThreads, C::kSmemBytes, 2, &n);
  if (err != cudaSuccess) return err;
  const long long n0 = static_cast<long long>(job.p[0].l_tiles) * job.p[0].c_tiles;
  const long long n1 = job.problems > 1 ? static_cast<long long>(job.p[1].l_tiles) * job.p[1].c_tiles : 0;
  const int pairs = n0 + n1 < n ? static_cast<int>(n0 + n1) : n;
  job.extra = n1 > 0 && n0 % pairs ? (job.p[0].nk + job.p[1].nk / 2) / job.p[1].nk : 0;
  return launch_clusters(kern, dim3(2 * pairs), C::kThreads, C::kSmemBytes, 2, st, job);
}

// A product's operand and output maps for the pair kernels, and its tiles.
mok_status_t pair_setup(bool a_mn, bool b_mn, const LinearOperands& o, LinearParams& p, LinearMaps* maps, bool store_maps) {
  const long long lt = (p.L + 255) / 256, ct = (static_cast<long long>(p.C) + 255) / 256;
  if (lt * ct > 0x7fffffffll / 4) return fail(MOK_ERR_INVALID_ARG, "product too large");
  p.nk = static_cast<int>((o.K + kLinBK - 1) / kLinBK);
  p.l_tiles = static_cast<int>(lt);
  p.c_tiles = static_cast<int>(ct);
  p.group = 8;
  mok_status_t s = a_mn ? operand_map(&maps->a, o.a, p.L, o.K, 64) : operand_map(&maps->a, o.a, o.K, p.L, 128);
  if (!s) s = b_mn ? operand_map(&maps->b, o.b, p.C, o.K, 64) : operand_map(&maps->b, o.b, o.K, p.C, 128);
  if (!s && store_maps) s = make_box(&maps->out, p.out, p.out_f32, p.L, p.C, 32, 32);
  if (!s && store_maps && p.z) s = make_box(&maps->z, p.z, 0, p.L, p.C, 32, 32);
  return s;
}

long long pair_tiles(const LinearParams& p) {
  return (p.L + 255) / 256 * ((static_cast<long long>(p.C) + 255) / 256);
}
// Whether a product is for the pair kernels: more than 128 rows, and either
// more than 128 columns or tiles enough to fill the GPU.  Measured, split and
// pair kernel: 1 x 152064 x 4096 177 and 326 us, 128 x 28672 x 4096 44 and 49,
// 1003 x 1416 x 2056 21.5 and 14.8, 100000 x 64 x 1024 46 and 40.
bool is_paired(const LinearParams& p, int pairs) { return p.C > 128 && (p.L > 128 || pair_tiles(p) >= pairs); }

// Up to how many K-blocks the forward runs with twice the epilogue warps for one
// stage less (fp32 outputs: up to kChunk).  Measured both ways (us; 8 and 16
// epilogue warps), 8192 x 4864 outputs: K = 272 40 and 36 plain, 67 and 53 with
// bias and GELU, 79 and 65 with a residual, 50 and 44 in fp32; K = 1024 50 and
// 50, 74 and 61, 87 and 73; K = 1536 66 and 68, 79 and 73; K = 2048 85 and 87,
// 91 and 91.
constexpr int kShortK = 16;

template <int KIND>
mok_status_t run_kind(const LinearOperands& o, const LinearParams& q, int num_sms, cudaStream_t st) {
  constexpr bool FWD = KIND == LIN_FWD, AMN = KIND != LIN_FWD, BMN = KIND == LIN_DW;
  LinearParams p = q;
  const int pairs = num_sms / 2;
  if (is_paired(p, pairs)) {
    const bool fills = pair_tiles(p) >= pairs;
    PairJob job = {};
    mok_status_t s = pair_setup(AMN, BMN, o, p, &job.maps[0], fills);
    if (s) return s;
    if (fills) {
      job.p[0] = p;
      job.problems = 1;
      if (FWD && p.out_f32 && p.nk > kChunk)
        MOK_CUDA(launch_pair<FWD ? LIN_FWD_F32 : KIND>(job, st));
      else if (FWD && p.nk <= kShortK)
        MOK_CUDA(launch_pair<FWD ? LIN_FWD_SHORT : KIND>(job, st));
      else
        MOK_CUDA(launch_pair<KIND>(job, st));
    } else {
      MOK_CUDA((launch_pair_split<AMN, BMN, FWD>(job.maps[0], p, st)));
    }
    return MOK_OK;
  }
  int bn = 128;
  if (!BMN && p.C <= 16) bn = 16;
  else if (!BMN && p.C <= 32) bn = 32;
  else if (p.C <= 64) bn = 64;
  p.nk = static_cast<int>((o.K + kLinBK - 1) / kLinBK);
  LinearMaps maps;
  mok_status_t s = AMN ? operand_map(&maps.a, o.a, p.L, o.K, 64) : operand_map(&maps.a, o.a, o.K, p.L, 128);
  if (!s) s = BMN ? operand_map(&maps.b, o.b, p.C, o.K, 64) : operand_map(&maps.b, o.b, o.K, p.C, bn);
  if (s) return s;
  cudaError_t err = cudaSuccess;
  if (bn == 128) {
    err = launch_split<AMN, BMN, 128, FWD>(maps, p, st);
  } else if (bn == 64) {
    err = launch_split<AMN, BMN, 64, FWD>(maps, p, st);
  } else if constexpr (!BMN) {
    err = bn == 32 ? launch_split<AMN, BMN, 32, FWD>(maps, p, st) : launch_split<AMN, BMN, 16, FWD>(maps, p, st);
  }
  MOK_CUDA(err);
  return MOK_OK;
}

// ---------------------------------------------------------------- dz
constexpr int kDzRows = 8;   // rows in step in a block; 32 threads x 8 columns wide

// dz = dy act'(z) in bf16, the products' operand type, and per block the column
// sums of the unrounded values.  Bound by memory: 8192 x 4096 with GELU 31 us
// for its 201 MB (6.5 TB/s).
template <class DY, int ACT>
__global__ void __launch_bounds__(256) linear_dz_kernel(const DY* __restrict__ dy, const uint16_t* __restrict__ z,
                                                        long long M, int N, uint16_t* __restrict__ dz,
                                                        float* __restrict__ part) {
  __shared__ float s[kDzRows][32][9];
  griddep_wait();
  griddep_launch_dependents();
  const int col = (blockIdx.x * 32 + threadIdx.x) * 8;
  float sum[8] = {};
  if (col < N) {
    for (long long r = static_cast<long long>(blockIdx.y) * kDzRows + threadIdx.y; r < M;
         r += static_cast<long long>(gridDim.y) * kDzRows) {
      const long long at = r * N + col;
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
  if (!part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) s[threadIdx.y][threadIdx.x][i] = sum[i];
  __syncthreads();
  const int t = threadIdx.y * 32 + threadIdx.x, c = t >> 3, i = t & 7;   // one column per thread
  float v = 0.f;
#pragma unroll
  for (int r = 0; r < kDzRows; ++r) v += s[r][c][i];
  const int out = (blockIdx.x * 32 + c) * 8 + i;
  if (out < N) part[static_cast<long long>(blockIdx.y) * N + out] = v;
}

template <class DY>
cudaError_t launch_dz(const DY* dy, const uint16_t* z, int act, long long M, int N, uint16_t* dz, float* part, cudaStream_t st) {
  const dim3 grid((N + 255) / 256, dz_partials(M, N)), block(32, kDzRows);
  switch (act) {
    case LIN_RELU: return launch_dependent(linear_dz_kernel<DY, LIN_RELU>, grid, block, 0, st, dy, z, M, N, dz, part);
    case LIN_SILU: return launch_dependent(linear_dz_kernel<DY, LIN_SILU>, grid, block, 0, st, dy, z, M, N, dz, part);
    case LIN_GELU: return launch_dependent(linear_dz_kernel<DY, LIN_GELU>, grid, block, 0, st, dy, z, M, N, dz, part);
    case LIN_GELU_TANH:
      return launch_dependent(linear_dz_kernel<DY, LIN_GELU_TANH>, grid, block, 0, st, dy, z, M, N, dz, part);
    default: return launch_dependent(linear_dz_kernel<DY, LIN_NONE>, grid, block, 0, st, dy, z, M, N, dz, part);
  }
}

}  // namespace

cudaError_t linear_status_word(int** word) {
  static std::atomic<int*> at[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  *word = at[dev].load(std::memory_order_acquire);
  if (!*word) {
    void* a = nullptr;
    err = cudaGetSymbolAddress(&a, g_linear_status);
    if (err != cudaSuccess) return err;
    *word = static_cast<int*>(a);
    at[dev].store(*word, std::memory_order_release);
  }
  return cudaSuccess;
}

mok_status_t run_linear(LinKind kind, const LinearOperands& o, const LinearParams& p, int num_sms, cudaStream_t st) {
  switch (kind) {
    case LIN_FWD: return run_kind<LIN_FWD>(o, p, num_sms, st);
    case LIN_DX: return run_kind<LIN_DX>(o, p, num_sms, st);
    default: return run_kind<LIN_DW>(o, p, num_sms, st);
  }
}

mok_status_t run_linear_grads(const LinearOperands& ox, const LinearParams& px, const LinearOperands& ow, const LinearParams& pw,
                              int num_sms, cudaStream_t st) {
  const int pairs = num_sms / 2;
  if (!is_paired(px, pairs) || !is_paired(pw, pairs) || pair_tiles(px) + pair_tiles(pw) < pairs) {
    const mok_status_t s = run_linear(LIN_DW, ow, pw, num_sms, st);
    return s ? s : run_linear(LIN_DX, ox, px, num_sms, st);
  }
  PairJob job = {};
  const int w = ow.K >= ox.K ? 0 : 1, x = 1 - w;   // the longer tiles first
  job.p[w] = pw;
  job.p[x] = px;
  job.b_mn[w] = 1;
  job.problems = 2;
  mok_status_t s = pair_setup(true, true, ow, job.p[w], &job.maps[w], true);
  if (!s) s = pair_setup(true, false, ox, job.p[x], &job.maps[x], true);
  if (s) return s;
  MOK_CUDA(launch_pair<LIN_GRADS>(job, st));
  return MOK_OK;
}

int dz_partials(long long M, int N) {
  // about 8 blocks for each of 152 SMs, a block no shorter than 4 steps
  const long long want = (1216 + (N + 255) / 256 - 1) / ((N + 255) / 256);
  const long long most = (M + 4 * kDzRows - 1) / (4 * kDzRows);
  const long long n = want < most ? want : most;
  return static_cast<int>(n < 1 ? 1 : n);
}

cudaError_t launch_linear_dz(const void* dy, int dy_f32, const uint16_t* z, int act, long long M, int N, uint16_t* dz,
                             float* part, cudaStream_t st) {
  if (M == 0) return cudaSuccess;
  return dy_f32 ? launch_dz(static_cast<const float*>(dy), z, act, M, N, dz, part, st)
                : launch_dz(static_cast<const uint16_t*>(dy), z, act, M, N, dz, part, st);
}

}  // namespace mok
