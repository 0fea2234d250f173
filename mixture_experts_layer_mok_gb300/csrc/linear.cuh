// Dense matrix products on tcgen05 / TMEM / TMA with a fused epilogue, for
// mok_linear and mok_linear_bwd.
//
// All three products are written as D[c][l] = sum_k A[l][k] B[c][k], with l
// the contiguous index of the row-major output.  l runs over the tensor
// core's M (128 TMEM lanes per CTA) and c over its N, so that a warp of the
// epilogue holds 32 neighbouring elements of an output row: its loads of the
// residual and its stores are whole 64- or 128-byte segments straight from
// registers, the bias is one value per lane, and a handful of tokens costs an
// N of 16 rather than a padded M of 128.
//   forward  l = n, c = m, k = k:  A = W [N][K],            B = x [M][K]
//   dx       l = k, c = m, k = n:  A = W^T (W is [k][l]),   B = dz [M][N]
//   dW       l = k, c = n, k = m:  A = x^T (x is [k][l]),   B = dz^T (dz is [k][c])
// An operand that is stored [k][l] is read in place as an MN-major operand.
// Sums are fp32 in TMEM; every edge (l, c and k) is cut by the tensor maps,
// whose loads read zeros outside.
//
// Two kernels.  linear_pair_kernel: persistent CTA pairs (M = 256 over two
// SMs, 256 columns, two accumulator buffers), for products with enough
// 256 x 256 tiles to fill the GPU.  linear_split_kernel: one 128 x BN tile per
// CTA, K split over a cluster of up to 8 CTAs that add their parts through
// distributed shared memory in rank order, for everything smaller, where
// the bytes of A have to come in through as many SMs as there are.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "gemm.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace mok {

struct LinearMaps {
  CUtensorMap a;
  CUtensorMap b;
};

constexpr int kLinBK = 64;                 // K-block of a stage: one 128-byte swizzled row
constexpr int kLinChunk = 64 * 128;        // an MN-major 64 x 64 block
constexpr int kLinABytes = 128 * kLinBK * 2;

// ---------------------------------------------------------------- epilogue
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == LIN_RELU) return z < 0.f ? 0.f : z;   // keeps a NaN
  if constexpr (ACT == LIN_SILU) return z * __fdividef(1.f, 1.f + __expf(-z));
  if constexpr (ACT == LIN_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
  if constexpr (ACT == LIN_GELU_TANH)   // 0.5 z (1 + tanh u) = z / (1 + exp(-2u))
    return z * __fdividef(1.f, 1.f + __expf(-1.5957691216057308f * (z + 0.044715f * z * z * z)));
  return z;
}

// d act / dz
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == LIN_RELU) return z > 0.f ? 1.f : z == z ? 0.f : z;
  if constexpr (ACT == LIN_SILU) {
    const float s = __fdividef(1.f, 1.f + __expf(-z));
    return s * (1.f + z * (1.f - s));
  }
  if constexpr (ACT == LIN_GELU)
    return 0.5f * (1.f + erff(z * 0.70710678118654752f)) + z * 0.3989422804014327f * __expf(-0.5f * z * z);
  if constexpr (ACT == LIN_GELU_TANH) {   // with s = 1 / (1 + exp(-2u)): s + 2 z s (1 - s) du/dz
    const float z2 = z * z;
    const float s = __fdividef(1.f, 1.f + __expf(-1.5957691216057308f * z * (1.f + 0.044715f * z2)));
    return s + z * s * (1.f - s) * 1.5957691216057308f * (1.f + 0.134145f * z2);
  }
  return 1.f;
}

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// The output elements (row c + i, column l) for i < NC from the sums acc:
// z = acc + bias, y = act(z) + residual.  Rows past p.C are left alone.
template <int ACT, int NC>
__device__ __forceinline__ void linear_store_act(const LinearParams& p, long long l, int c, float bias, const float* acc) {
  const int n = min(NC, p.C - c);
  const long long at = static_cast<long long>(c) * p.L + l;
  float res[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    res[i] = 0.f;
    if (p.residual && i < n)
      res[i] = p.residual_f32 ? __ldg(static_cast<const float*>(p.residual) + at + static_cast<long long>(i) * p.L)
                              : bf16_value(__ldg(static_cast<const uint16_t*>(p.residual) + at + static_cast<long long>(i) * p.L));
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if (i < n) {
      const long long o = at + static_cast<long long>(i) * p.L;
      const float z = acc[i] + bias;
      if (p.z) p.z[o] = __bfloat16_as_ushort(__float2bfloat16_rn(z));
      const float y = act_value<ACT>(z) + res[i];
      if (p.out_f32)
        static_cast<float*>(p.out)[o] = y;
      else
        static_cast<uint16_t*>(p.out)[o] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
    }
  }
}

template <bool FWD, int NC>
__device__ __forceinline__ void linear_store(const LinearParams& p, long long l, int c, float bias, const float* acc) {
  if (l >= p.L || c >= p.C) return;
  if constexpr (!FWD) {
    const int n = min(NC, p.C - c);
    uint16_t* o = static_cast<uint16_t*>(p.out) + static_cast<long long>(c) * p.L + l;
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (i < n) o[static_cast<long long>(i) * p.L] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[i]));
  } else {
    switch (p.act) {
      case LIN_RELU: linear_store_act<LIN_RELU, NC>(p, l, c, bias, acc); break;
      case LIN_SILU: linear_store_act<LIN_SILU, NC>(p, l, c, bias, acc); break;
      case LIN_GELU: linear_store_act<LIN_GELU, NC>(p, l, c, bias, acc); break;
      case LIN_GELU_TANH: linear_store_act<LIN_GELU_TANH, NC>(p, l, c, bias, acc); break;
      default: linear_store_act<LIN_NONE, NC>(p, l, c, bias, acc); break;
    }
  }
}

__device__ __forceinline__ float lane_bias(const LinearParams& p, long long l) {
  if (!p.bias || l >= p.L) return 0.f;
  return p.bias_f32 ? __ldg(static_cast<const float*>(p.bias) + l) : bf16_value(__ldg(static_cast<const uint16_t*>(p.bias) + l));
}

// Descriptor of K-step kk (16 elements) of an operand block at shared address
// s: K-major rows of 128 bytes, or MN-major chunks of 64 x 64.
template <bool MN>
__device__ __forceinline__ uint64_t linear_desc(uint32_t s, int kk) {
  return MN ? smem_desc(s + kk * 16 * 128, kLinChunk, 1024, 2u) : smem_desc(s + kk * 32, 16, 1024, 2u);
}

// ---------------------------------------------------------------- split kernel
template <bool AMN, bool BMN, int BN>
struct SplitCfg {
  static constexpr int kBBytes = BN * kLinBK * 2;
  static constexpr int kStageBytes = kLinABytes + kBBytes;
  // as many stages as let two CTAs share an SM
  static constexpr int kStages = BN <= 32 ? 5 : BN == 64 ? 4 : 3;
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + 256;
  static constexpr int kTmemCols = BN < 32 ? 32 : BN;
  static constexpr int kThreads = 192;
  static constexpr uint32_t kIdesc = idesc_bf16(128, BN, AMN, BMN);
  static_assert(BN * 128 * 4 <= kStages * kStageBytes, "the partial tile fits the stages");
  static_assert(!BMN || BN % 64 == 0, "MN-major B comes in 64-wide chunks");
};

__device__ __forceinline__ float ld_shared_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// grid {S * L tiles, C tiles}, clusters of S CTAs along K.
// warp 0: TMA producer; warp 1: MMA issuer, TMEM owner; warps 2..5: epilogue.
template <bool AMN, bool BMN, int BN, bool FWD>
__global__ void __launch_bounds__(192, 2) linear_split_kernel(const __grid_constant__ LinearMaps maps, const LinearParams p) {
  using C = SplitCfg<AMN, BMN, BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;
  uint64_t* done = tfull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.split;
  const int rank = S > 1 ? static_cast<int>(cluster_rank()) : 0;
  const long long l0 = static_cast<long long>(blockIdx.x / S) * 128;
  const int c0 = blockIdx.y * BN;
  const int kb0 = static_cast<int>(static_cast<long long>(p.nk) * rank / S);
  const int kb1 = static_cast<int>(static_cast<long long>(p.nk) * (rank + 1) / S);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tmem_base = *tmem_slot;
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, fills = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&full[stage], C::kStageBytes);
        uint8_t* sA = smem + stage * C::kStageBytes;
        uint8_t* sB = sA + kLinABytes;
        const int k0 = kb * kLinBK;
        if (AMN) {
          tma_load_2d(sA, &maps.a, &full[stage], static_cast<int>(l0), k0);
          tma_load_2d(sA + kLinChunk, &maps.a, &full[stage], static_cast<int>(l0) + 64, k0);
        } else {
          tma_load_2d(sA, &maps.a, &full[stage], k0, static_cast<int>(l0));
        }
        if (BMN) {
#pragma unroll
          for (int j = 0; j < BN / 64; ++j) tma_load_2d(sB + j * kLinChunk, &maps.b, &full[stage], c0 + 64 * j, k0);
        } else {
          tma_load_2d(sB, &maps.b, &full[stage], k0, c0);
        }
        ++fills;
        if (++stage == C::kStages) stage = 0, phase ^= 1;
      }
      if (!ok) {   // no load may be in flight when the CTA ends
        const int n = min(fills, C::kStages);
        for (int i = 0; i < n; ++i) {
          if (--stage < 0) stage = C::kStages - 1, phase ^= 1;
          mbar_drain(&full[stage], phase);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&full[stage], phase, abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a0 = smem_u32(smem + stage * C::kStageBytes), b0 = a0 + kLinABytes;
#pragma unroll
        for (int kk = 0; kk < kLinBK / 16; ++kk)
          umma_bf16(tmem_base, linear_desc<AMN>(a0, kk), linear_desc<BMN>(b0, kk), C::kIdesc, (kb > kb0 || kk) ? 1u : 0u);
        umma_commit(&empty[stage]);
        if (++stage == C::kStages) stage = 0, phase ^= 1;
      }
      if (ok) umma_commit(tfull);
      umma_commit(done);   // every MMA issued here ends before TMEM is released
      mbar_drain(done, 0);
    }
  }
  __syncwarp();
  const int q = warp & 3, row = q * 32 + lane;
  const long long l = l0 + row;
  bool ready = false;
  float bias = 0.f;
  float* part = reinterpret_cast<float*>(smem);   // [BN][128], over the stages
  if (warp >= 2) {
    if (FWD) bias = lane_bias(p, l);
    int w = (lane == 0) ? (mbar_wait(tfull, 0, abort_flag, p.status) ? 1 : 0) : 0;
    ready = __shfl_sync(0xffffffffu, w, 0) != 0;
    tc_fence_after();
    if (ready) {
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < BN; c += 16) {
        float v[16];
        tmem_ld16(tb + c, v);
        if (S == 1) {
          linear_store<FWD, 16>(p, l, c0 + c, bias, v);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) part[(c + i) * 128 + row] = v[i];
        }
      }
    }
    tc_fence_before();
  }
  if (S > 1) {
    __syncwarp();
    cluster_sync();   // every CTA's part is in its shared memory
    if (warp >= 2) {
      // this CTA's share of the columns: the parts of all ranks, in rank order
      const int nc = BN / S;
      uint32_t peer[8];
#pragma unroll
      for (int s = 0; s < 8; ++s) peer[s] = s < S ? cluster_addr(part, s) : 0u;
      for (int c = rank * nc; c < (rank + 1) * nc; c += 2) {
        float v[2] = {0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          if (s < S) {
            v[0] += ld_shared_cluster(peer[s] + static_cast<uint32_t>(c * 128 + row) * 4u);
            v[1] += ld_shared_cluster(peer[s] + static_cast<uint32_t>((c + 1) * 128 + row) * 4u);
          }
        }
        linear_store<FWD, 2>(p, l, c0 + c, bias, v);
      }
    }
    __syncwarp();
    cluster_sync();   // nobody reads this CTA's shared memory any more
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// ---------------------------------------------------------------- pair kernel
template <bool AMN, bool BMN>
struct PairCfg {
  static constexpr int BN = 256;
  static constexpr int kBBytes = 128 * kLinBK * 2;   // this CTA's half of B
  static constexpr int kStageBytes = kLinABytes + kBBytes;
  static constexpr int kStages = 6;
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + 512;
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr uint32_t kIdesc = idesc_bf16(256, BN, AMN, BMN);
};

// Tile idx of the grid of L tiles x C tiles (256 x 256 each): C tiles in
// groups of p.group, L tiles inside the group's width, so that the CTAs at
// work at one time share few rows of both operands.
__device__ __forceinline__ void linear_tile(const LinearParams& p, int idx, int& lt, int& ct) {
  unit_and_col(idx, p.c_tiles, p.l_tiles, p.group, ct, lt);
}

template <bool AMN, bool BMN, bool FWD>
__global__ void __launch_bounds__(320, 1) linear_pair_kernel(const __grid_constant__ LinearMaps maps, const LinearParams p) {
  using C = PairCfg<AMN, BMN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  const int items = p.l_tiles * p.c_tiles;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * C::kEpiWarps);   // the leader's counts both CTAs' warps
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();   // both CTAs' barriers are there before any signal crosses
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tmem_base = *tmem_slot;
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      long long fills = 0;
      bool ok = true;
      for (int idx = first; idx < items && ok; idx += step) {
        int lt, ct;
        linear_tile(p, idx, lt, ct);
        const int l0 = lt * 256 + rank * 128, c0 = ct * 256 + rank * 128;
        for (int kb = 0; kb < p.nk; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * C::kStageBytes);
          uint8_t* sA = smem + stage * C::kStageBytes;
          uint8_t* sB = sA + kLinABytes;
          const uint32_t bar = cluster_addr(&full[stage], 0);   // both CTAs' loads count on the leader's
          const int k0 = kb * kLinBK;
          if (AMN) {
            tma_load_2d_pair(sA, &maps.a, bar, l0, k0);
            tma_load_2d_pair(sA + kLinChunk, &maps.a, bar, l0 + 64, k0);
          } else {
            tma_load_2d_pair(sA, &maps.a, bar, k0, l0);
          }
          if (BMN) {
            tma_load_2d_pair(sB, &maps.b, bar, c0, k0);
            tma_load_2d_pair(sB + kLinChunk, &maps.b, bar, c0 + 64, k0);
          } else {
            tma_load_2d_pair(sB, &maps.b, bar, k0, c0);
          }
          ++fills;
          if (++stage == C::kStages) stage = 0, phase ^= 1;
        }
      }
      if (!ok && rank == 0) {
        const int n = fills < C::kStages ? static_cast<int>(fills) : C::kStages;
        for (int i = 0; i < n; ++i) {
          if (--stage < 0) stage = C::kStages - 1, phase ^= 1;
          mbar_drain(&full[stage], phase);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      int stage = 0, buf = 0;
      uint32_t phase = 0, bphase = 0;
      bool ok = true;
      for (int idx = first; idx < items && ok; idx += step) {
        if (!mbar_wait(&tempty[buf], bphase ^ 1, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t acc = tmem_base + static_cast<uint32_t>(buf * C::BN);
        for (int kb = 0; kb < p.nk; ++kb) {
          if (!mbar_wait(&full[stage], phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(smem + stage * C::kStageBytes), b0 = a0 + kLinABytes;
#pragma unroll
          for (int kk = 0; kk < kLinBK / 16; ++kk)
            umma_bf16_pair(acc, linear_desc<AMN>(a0, kk), linear_desc<BMN>(b0, kk), C::kIdesc, (kb | kk) ? 1u : 0u);
          umma_commit_pair(&empty[stage], 0x3);
          if (++stage == C::kStages) stage = 0, phase ^= 1;
        }
        if (!ok) break;
        umma_commit_pair(&tfull[buf], 0x3);
        buf ^= 1;
        if (buf == 0) bphase ^= 1;
      }
      umma_commit_pair(done, 0x1);
      mbar_drain(done, 0);
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    int buf = 0;
    uint32_t bphase = 0;
    for (int idx = first; idx < items; idx += step) {
      int lt, ct;
      linear_tile(p, idx, lt, ct);
      const long long l = static_cast<long long>(lt) * 256 + rank * 128 + q * 32 + lane;
      const int c0 = ct * 256 + half * 128;
      const float bias = FWD ? lane_bias(p, l) : 0.f;
      int w = (lane == 0) ? (mbar_wait(&tfull[buf], bphase, abort_flag, p.status) ? 1 : 0) : 0;
      if (!__shfl_sync(0xffffffffu, w, 0)) break;
      tc_fence_after();
      const uint32_t tb = tmem_base + static_cast<uint32_t>(buf * C::BN + half * 128) + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        float v[32];
        tmem_ld32(tb + c, v);
        linear_store<FWD, 32>(p, l, c0 + c, bias, v);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank != 0)
          mbar_arrive_cluster(cluster_addr(&tempty[buf], 0));
        else
          mbar_arrive(&tempty[buf]);
      }
      buf ^= 1;
      if (buf == 0) bphase ^= 1;
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();   // the leader's MMAs into both TMEMs are done
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

}  // namespace mok
