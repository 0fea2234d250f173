// Dense matrix products on tcgen05 / TMEM / TMA with a fused epilogue, for
// mok_linear and mok_linear_bwd.
//
// All three products are written as D[c][l] = sum_k A[l][k] B[c][k], with l
// the contiguous index of the row-major output:
//   forward  l = n, c = m, k = k:  A = W [N][K],            B = x [M][K]
//   dx       l = k, c = m, k = n:  A = W^T (W is [k][l]),   B = dz [M][N]
//   dW       l = k, c = n, k = m:  A = x^T (x is [k][l]),   B = dz^T (dz is [k][c])
// An operand that is stored [k][l] is read in place as an MN-major operand.
// Sums are fp32 in TMEM; every edge (l, c and k) is cut by the tensor maps,
// whose loads read zeros outside and whose stores write nothing there.
//
// Three kernels, each of which sums fp32 outputs in chunks of K (kChunk).
//   linear_pair_kernel: persistent CTA pairs (M = 256 rows c over two SMs, 256
//   columns l, two accumulator buffers), for products with enough 256 x 256
//   tiles to fill the GPU.  Each thread of the epilogue holds 32 neighbouring
//   elements of an output row, which leave through TMA stores.
//   linear_pair_split_kernel: the same tile with K split over 1 to 4 pairs of a
//   cluster, which add their parts through distributed shared memory in rank
//   order, for products of fewer such tiles.  An SM takes in about 64 bytes a
//   clock from L2, which bounds these: a pair loads 32 KB per CTA for 128 x
//   256 outputs, half of what two 128 x 128 tiles would.
//   linear_split_kernel: one 128 x BN tile per CTA, K split over a cluster of
//   up to 8 CTAs joined in the same way, where one side of the output is at
//   most 128 wide.  Here l runs over the tensor core's M, so that a handful of
//   tokens costs an N of 16 rather than a padded M, and the bytes of A come in
//   through as many SMs as there are.
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
  CUtensorMap out;   // pair kernel: 32 x 32 boxes of the output and of z
  CUtensorMap z;
};

constexpr int kLinBK = 64;                 // K-block of a stage: one 128-byte swizzled row
constexpr int kLinChunk = 64 * 128;        // an MN-major 64 x 64 block
constexpr int kLinABytes = 128 * kLinBK * 2;

// ---------------------------------------------------------------- epilogue
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float logistic(float x) { return fast_rcp(1.f + fast_exp2(-kLog2e * x)); }

// 1 - Phi(|z|), Phi the normal distribution function, and e = exp(-z^2/2):
// with t = 1 / (1 + p |z| / sqrt 2) it is 1/2 poly(t) e (Abramowitz and Stegun,
// 7.1.26, whose own error is below 7.5e-8).  Evaluated in these 32-bit steps it is
// off by up to 3e-7, and GELU, measured over [-12, 12], by 3.3e-7; for negative z
// that is 3.3e-6 of the value at -2, 1.6e-3 at -5, 3.6e-3 at -6 and 4% at -8 (of
// 6e-16), where 0.5 z (1 + erf) in 32 bits is off by 1.1e-6, 6% and, from -6 on,
// all of it.  A dozen instructions without a branch, where erff takes both of
// its branches in nearly every warp.
__device__ __forceinline__ float normal_tail(float z, float& e) {
  const float t = fast_rcp(fmaf(0.3275911f * 0.70710678118654752f, fabsf(z), 1.f));
  e = fast_exp2(z * z * (-0.5f * kLog2e));
  float q = fmaf(t, 0.5f * 1.061405429f, 0.5f * -1.453152027f);
  q = fmaf(t, q, 0.5f * 1.421413741f);
  q = fmaf(t, q, 0.5f * -0.284496736f);
  q = fmaf(t, q, 0.5f * 0.254829592f);
  return q * (t * e);
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == LIN_RELU) return z < 0.f ? 0.f : z;   // keeps a NaN
  if constexpr (ACT == LIN_SILU) return z * logistic(z);
  if constexpr (ACT == LIN_GELU) {
    // z Phi(z) = max(z, 0) - |z| (1 - Phi(|z|)); the last factor is 0 from 15 on
    float e;
    const float q = normal_tail(z, e);
    return fmaf(-fminf(fabsf(z), 64.f), q, z < 0.f ? 0.f : z);
  }
  if constexpr (ACT == LIN_GELU_TANH)   // 0.5 z (1 + tanh u) = z / (1 + exp(-2u))
    return z * logistic(1.5957691216057308f * z * fmaf(0.044715f * z, z, 1.f));
  return z;
}

// d act / dz
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == LIN_RELU) return z > 0.f ? 1.f : z == z ? 0.f : z;
  if constexpr (ACT == LIN_SILU) {
    const float s = logistic(z);
    return s * fmaf(z, 1.f - s, 1.f);
  }
  if constexpr (ACT == LIN_GELU) {   // Phi(z) + z phi(z)
    float e;
    const float q = normal_tail(z, e);
    return fmaf(z * 0.3989422804014327f, e, z < 0.f ? q : 1.f - q);
  }
  if constexpr (ACT == LIN_GELU_TANH) {   // with s = 1 / (1 + exp(-2u)): s + z s (1 - s) d(2u)/dz
    const float z2 = z * z;
    const float s = logistic(1.5957691216057308f * z * fmaf(0.044715f, z2, 1.f));
    return fmaf(z * s * (1.f - s), 1.5957691216057308f * fmaf(0.134145f, z2, 1.f), s);
  }
  return 1.f;
}

template <bool READ_ONLY, class T>
__device__ __forceinline__ T load_as(const T* p) {
  if constexpr (READ_ONLY) return __ldg(p);
  return *p;
}
// NV (4 or 8) consecutive values of a bf16 or fp32 array.  READ_ONLY: nothing in
// the launch writes it, as the residual may be, whose place the output can take.
template <int NV, bool READ_ONLY = true>
__device__ __forceinline__ void load_vals(const void* base, int f32, long long at, float* f) {
  if (f32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
#pragma unroll
    for (int i = 0; i < NV / 4; ++i) {
      const float4 a = load_as<READ_ONLY>(p + i);
      f[4 * i] = a.x, f[4 * i + 1] = a.y, f[4 * i + 2] = a.z, f[4 * i + 3] = a.w;
    }
  } else {
    uint32_t w[NV / 2];
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if constexpr (NV == 8) {
      const uint4 a = load_as<READ_ONLY>(reinterpret_cast<const uint4*>(p));
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    } else {
      const uint2 a = load_as<READ_ONLY>(reinterpret_cast<const uint2*>(p));
      w[0] = a.x, w[1] = a.y;
    }
#pragma unroll
    for (int i = 0; i < NV / 2; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

// Four output elements at index `at`: z = acc + bias, y = act(z) + residual.
template <int ACT>
__device__ __forceinline__ void store_four(const LinearParams& p, long long at, const float* bias, const float* acc,
                                           const float* res) {
  float z[4], y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    z[i] = acc[i] + bias[i];
    y[i] = act_value<ACT>(z[i]) + res[i];
  }
  if (p.z) *reinterpret_cast<uint2*>(p.z + at) = make_uint2(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]));
  if (p.out_f32)
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(y[0], y[1], y[2], y[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
}

// Descriptor of an operand block at shared address s (K-major rows of 128
// bytes, or MN-major chunks of 64 x 64), and the same `bytes` further on: the
// low word holds the address in units of 16 bytes.  The issuing thread's own
// instructions are what a k-block of 512 tensor cycles has little room for
// (rebuilt descriptors cost the pair kernel a fifth of its rate), so it only
// adds constants to two low words.
template <bool MN>
__device__ __forceinline__ uint64_t linear_desc(uint32_t s) {
  return MN ? smem_desc(s, kLinChunk, 1024, 2u) : smem_desc(s, 16, 1024, 2u);
}
__device__ __forceinline__ uint64_t desc_at(uint64_t d, uint32_t bytes) {
  return (d & 0xFFFFFFFF00000000ull) | (static_cast<uint32_t>(d) + (bytes >> 4));
}
// The loops of the producer and of the MMA issuer run in whole warps, so that
// their counters, addresses and descriptors are warp-uniform values (what the
// instructions they issue take); one elected lane issues.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
// mbar_wait for a whole warp: the same answer in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status));
}

// Bytes from one K-step (16 elements) to the next.
template <bool MN>
constexpr uint32_t kStep = MN ? 16 * 128 : 32;

// 8 consecutive fp32 columns of this thread's TMEM lane, waited on.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// 16 consecutive fp32 columns of this thread's TMEM lane, not waited on.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// K-blocks that are summed in the tensor core for fp32 outputs before they are
// added to the sums that the epilogue's registers hold.  The tensor core's
// additions truncate, which shifts a sum by about 1e-9 of its size per k: in one
// go, the outputs of K = 4096 are 4.4e-6 off and those of K = 16384 1.9e-5, in
// chunks 7e-7 both, whichever kernel takes the product (bf16 outputs, rounded at
// 2e-3, have no use for it).  The split kernels sum up to two chunks in their
// two accumulators, and only longer ranges of K in registers.
constexpr int kChunk = 12;

// This thread's N columns at TMEM address t, in steps of 16 (or 8): added to
// sum, or with BACK the sums put in their place.
template <int N, bool BACK = false>
__device__ __forceinline__ void add_columns(uint32_t t, float (&sum)[N]) {
  constexpr int kStep = N % 16 == 0 ? 16 : 8;
  static_assert(N % kStep == 0 && (kStep == 16 || !BACK), "whole steps");
#pragma unroll
  for (int j = 0; j < N; j += kStep) {
    float v[kStep];
    if constexpr (kStep == 16)
      tmem_ld16(t + j, v);
    else
      tmem_ld8(t + j, v);
#pragma unroll
    for (int i = 0; i < kStep; ++i) sum[j + i] += v[i];
    if constexpr (BACK) tmem_st16(t + j, sum + j);
  }
  if (BACK) asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ---------------------------------------------------------------- split kernel
template <bool AMN, bool BMN, int BN>
struct SplitCfg {
  static constexpr int kBBytes = BN * kLinBK * 2;
  static constexpr int kStageBytes = kLinABytes + kBBytes;
  // as many stages as let two CTAs share an SM
  static constexpr int kStages = BN <= 32 ? 5 : BN == 64 ? 4 : 3;
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + 256;
  static constexpr int kTmemCols = 2 * BN;   // two accumulators, for fp32 outputs
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr uint32_t kIdesc = idesc_bf16(128, BN, AMN, BMN);
  static_assert(BN * 128 * 4 <= kStages * kStageBytes, "the partial tile fits the stages");
  static_assert(!BMN || BN % 64 == 0, "MN-major B comes in 64-wide chunks");
};

__device__ __forceinline__ float4 ld_shared_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

// float4 at byte `off` of rank s's part: this CTA's own through plain shared
// loads, which are several times as fast as through the cluster's window.
template <int S>
__device__ __forceinline__ float4 part_of(const float* mine, const uint32_t* peer, int s, int me, uint32_t off) {
  if (S == 1 || s == me) return *reinterpret_cast<const float4*>(reinterpret_cast<const char*>(mine) + off);
  return ld_shared_cluster4(peer[s] + off);
}

// The join of a tile whose parts [BN][128] lie at `part` in the shared memory
// of S CTAs: this CTA's share of the columns, summed in rank order, four
// elements of a row per thread.  Several columns at a time, their residuals
// and all ranks' parts in flight together: one at a time each would cost the
// latency of a global and of a remote load.
template <bool FWD, int ACT, int S, int BN>
__device__ __forceinline__ void join_columns(const LinearParams& p, const float* part, int rank, long long l0, int c0, int warp,
                                             int lane) {
  constexpr int kShare = BN / S, kWarps = 8, kAtOnce = 2;
  const long long l = l0 + lane * 4;
  if (l >= p.L) return;
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  if (FWD && p.bias) load_vals<4>(p.bias, p.bias_f32, l, bias);
  uint32_t peer[S];
#pragma unroll
  for (int s = 0; s < S; ++s) peer[s] = S > 1 ? cluster_addr(part, s) : smem_u32(part);
  const int c_end = min((rank + 1) * kShare, p.C - c0);
  for (int c = rank * kShare + warp; c < c_end; c += kWarps * kAtOnce) {
    float r[kAtOnce][4] = {}, v[kAtOnce][4] = {};
    float4 t[kAtOnce][S];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int cu = min(c + kWarps * u, c_end - 1);   // past the end: the last column again, not stored
      if (FWD && p.residual) load_vals<4, false>(p.residual, p.residual_f32, static_cast<long long>(c0 + cu) * p.L + l, r[u]);
#pragma unroll
      for (int s = 0; s < S; ++s) t[u][s] = part_of<S>(part, peer, s, rank, static_cast<uint32_t>(cu * 128 + lane * 4) * 4u);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
#pragma unroll
      for (int s = 0; s < S; ++s) v[u][0] += t[u][s].x, v[u][1] += t[u][s].y, v[u][2] += t[u][s].z, v[u][3] += t[u][s].w;
      const int cu = c + kWarps * u;
      if (cu < c_end) store_four<ACT>(p, static_cast<long long>(c0 + cu) * p.L + l, bias, v[u], r[u]);
    }
  }
}

template <bool FWD, int ACT, int BN>
__device__ __forceinline__ void join_split(const LinearParams& p, const float* part, int rank, long long l0, int c0, int warp,
                                           int lane) {
  switch (p.split) {
    case 1: join_columns<FWD, ACT, 1, BN>(p, part, rank, l0, c0, warp, lane); break;
    case 2: join_columns<FWD, ACT, 2, BN>(p, part, rank, l0, c0, warp, lane); break;
    case 4: join_columns<FWD, ACT, 4, BN>(p, part, rank, l0, c0, warp, lane); break;
    default: join_columns<FWD, ACT, 8, BN>(p, part, rank, l0, c0, warp, lane); break;
  }
}

// grid {S * L tiles, C tiles}, clusters of S CTAs along K.
// warp 0: TMA producer; warp 1: MMA issuer, TMEM owner; the others: epilogue, two
// warps for each quarter of the TMEM lanes.  Few rows are bound by the bytes of
// the weight: one row, 152064 x 4096, 174 us (7.2 TB/s); 7168 x 2048, 7.3 us, of
// which the launch and the first bytes take three.
// CHUNKED: fp32 outputs over more than two chunks of K to a CTA; 100 x 152064 x
// 4096 209 us so and 204 in two accumulators, 128 x 40000 x 16384 286 and 276, 1 x
// 152064 x 4096 176 and 175 (errors 7e-7, and 2.1e-6 and 9.1e-6).
template <bool AMN, bool BMN, int BN, bool FWD, bool CHUNKED>
__global__ void __launch_bounds__(SplitCfg<AMN, BMN, BN>::kThreads, 2) linear_split_kernel(const __grid_constant__ LinearMaps maps, const LinearParams p) {
  using C = SplitCfg<AMN, BMN, BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;   // (the second, and tempty: CHUNKED)
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.split;
  const int rank = S > 1 ? static_cast<int>(cluster_rank()) : 0;
  const long long l0 = static_cast<long long>(blockIdx.x / S) * 128;
  const int c0 = blockIdx.y * BN;
  const int kb0 = static_cast<int>(static_cast<long long>(p.nk) * rank / S);
  const int kb1 = static_cast<int>(static_cast<long long>(p.nk) * (rank + 1) / S);
  // fp32 outputs: the K range in two accumulators, added in the epilogue, which
  // halves the length of the tensor core's chain of truncating additions
  const bool two = FWD && !CHUNKED && p.out_f32 && kb1 - kb0 > 1;
  const int kbm = two ? (kb0 + kb1) / 2 : kb1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], C::kEpiWarps);
    }
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
    int stage = 0, fills = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!warp_wait(&empty[stage], phase ^ 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      uint8_t* sA = smem + stage * C::kStageBytes;
      uint8_t* sB = sA + kLinABytes;
      const int k0 = kb * kLinBK;
      if (elect_one()) {
        mbar_arrive_expect_tx(&full[stage], C::kStageBytes);
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
      }
      __syncwarp();
      ++fills;
      if (++stage == C::kStages) stage = 0, phase ^= 1;
    }
    if (!ok && lane == 0) {   // no load may be in flight when the CTA ends
      const int n = min(fills, C::kStages);
      for (int i = 0; i < n; ++i) {
        if (--stage < 0) stage = C::kStages - 1, phase ^= 1;
        mbar_drain(&full[stage], phase);
      }
    }
  } else if (warp == 1) {
    const uint64_t ad = linear_desc<AMN>(smem_u32(smem)), bd = linear_desc<BMN>(smem_u32(smem) + kLinABytes);
    int stage = 0, buf = 0, in = 0;   // CHUNKED: the accumulator, and the block's place in its chunk
    uint32_t phase = 0, bphase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (CHUNKED && in == 0) {
        if (!warp_wait(&tempty[buf], bphase ^ 1, abort_flag, p.status)) break;
        tc_fence_after();
      }
      if (!warp_wait(&full[stage], phase, abort_flag, p.status)) break;
      const uint32_t at = stage * C::kStageBytes, acc = tmem_base + (CHUNKED ? buf * BN : kb >= kbm ? BN : 0);
      const bool last = CHUNKED ? in == kChunk - 1 || kb == kb1 - 1 : kb == kb1 - 1;
      if (elect_one()) {
        umma_bf16(acc, desc_at(ad, at), desc_at(bd, at), C::kIdesc, CHUNKED ? in != 0 : kb != kb0 && kb != kbm);
#pragma unroll
        for (int kk = 1; kk < kLinBK / 16; ++kk)
          umma_bf16(acc, desc_at(ad, at + kk * kStep<AMN>), desc_at(bd, at + kk * kStep<BMN>), C::kIdesc, 1u);
        umma_commit(&empty[stage]);
        if (last) umma_commit(&tfull[CHUNKED ? buf : 0]);
      }
      __syncwarp();
      if (CHUNKED && ++in == kChunk) {
        in = 0;
        buf ^= 1;
        if (buf == 0) bphase ^= 1;
      }
      if (++stage == C::kStages) stage = 0, phase ^= 1;
    }
    if (elect_one()) {
      umma_commit(done);   // every MMA issued here ends before TMEM is released
      mbar_drain(done, 0);
    }
  }
  __syncwarp();
  float* part = reinterpret_cast<float*>(smem);   // [BN][128], over the stages
  if (warp >= 2) {
    const int q = warp & 3, row = q * 32 + lane, col0 = ((warp - 2) >> 2) * (BN / 2);
    if (FWD && p.residual) {   // this CTA's share of it into L2 while the accumulator fills
      const int size = p.residual_f32 ? 4 : 2, c1 = min((rank + 1) * (BN / S), p.C - c0);
      const long long cols = p.L - l0 < 128 ? p.L - l0 : 128;
      for (int c = rank * (BN / S) + warp - 2; c < c1; c += C::kEpiWarps)
        if (lane * 128 < cols * size)
          prefetch_l2(static_cast<const char*>(p.residual) + (static_cast<long long>(c0 + c) * p.L + l0) * size + lane * 128);
    }
    const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    const auto wait_full = [&](uint64_t* bar, uint32_t parity) {
      const int w = lane == 0 ? (mbar_wait(bar, parity, abort_flag, p.status) ? 1 : 0) : 0;
      const bool got = __shfl_sync(0xffffffffu, w, 0) != 0;
      tc_fence_after();
      return got;
    };
    if constexpr (CHUNKED) {
      float sum[BN / 2] = {};
      bool ok = true;
      int buf = 0;
      uint32_t bphase = 0;
      for (int first = kb0; first < kb1; first += kChunk) {
        if (!(ok = wait_full(&tfull[buf], bphase))) break;
        add_columns<BN / 2>(tb + buf * BN + col0, sum);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[buf]);
        buf ^= 1;
        if (buf == 0) bphase ^= 1;
      }
      if (ok) {
#pragma unroll
        for (int c = 0; c < BN / 2; ++c) part[(col0 + c) * 128 + row] = sum[c];
      }
    } else if (wait_full(tfull, 0)) {
#pragma unroll 1
      for (int c = col0; c < col0 + BN / 2; c += 8) {
        float v[8];
        tmem_ld8(tb + c, v);
        if (two) {
          float u[8];
          tmem_ld8(tb + BN + c, u);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += u[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) part[(c + i) * 128 + row] = v[i];
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  // every CTA's part is in its shared memory; each now finishes its share of
  // the columns, four elements of a row per thread
  if (S > 1)
    cluster_sync();
  else
    __syncthreads();
  if (warp >= 2) switch (FWD ? p.act : LIN_NONE) {
    case LIN_RELU: join_split<FWD, FWD ? LIN_RELU : LIN_NONE, BN>(p, part, rank, l0, c0, warp - 2, lane); break;
    case LIN_SILU: join_split<FWD, FWD ? LIN_SILU : LIN_NONE, BN>(p, part, rank, l0, c0, warp - 2, lane); break;
    case LIN_GELU: join_split<FWD, FWD ? LIN_GELU : LIN_NONE, BN>(p, part, rank, l0, c0, warp - 2, lane); break;
    case LIN_GELU_TANH: join_split<FWD, FWD ? LIN_GELU_TANH : LIN_NONE, BN>(p, part, rank, l0, c0, warp - 2, lane); break;
    default: join_split<FWD, LIN_NONE, BN>(p, part, rank, l0, c0, warp - 2, lane); break;
  }
  __syncwarp();
  if (S > 1) cluster_sync();   // nobody reads this CTA's shared memory any more
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// ---------------------------------------------------------------- pair kernel
// SHORT: the forward over few K-blocks, whose epilogue takes longer than its
// products: twice the epilogue warps, for one stage less.
template <bool AMN, bool BMN, bool SHORT = false>
struct PairCfg {
  static constexpr int BN = 256;
  static constexpr int kBBytes = 128 * kLinBK * 2;   // this CTA's half of B
  static constexpr int kStageBytes = kLinABytes + kBBytes;
  static constexpr int kStages = SHORT ? 5 : 6;
  static constexpr int kEpiWarps = SHORT ? 16 : 8;
  static constexpr int kOutBytes = 4096;   // per epilogue warp: see output_block
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kEpiWarps * kOutBytes + 512;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr uint32_t kIdesc = idesc_bf16(256, BN, BMN, AMN);
};

// Tile idx of the grid of L tiles x C tiles (256 x 256 each): C tiles in
// groups of p.group, L tiles inside the group's width, so that the CTAs at
// work at one time share few rows of both operands.
__device__ __forceinline__ void linear_tile(const LinearParams& p, int idx, int& lt, int& ct) {
  unit_and_col(idx, p.c_tiles, p.l_tiles, p.group, ct, lt);
}

// 16-byte piece j of this lane's row in a staged 32 x 32 block, in the
// swizzled layout of its tensor map: rows of 64 bytes (bf16) or 128 (fp32).
template <bool F32>
__device__ __forceinline__ uint4* stage_piece(uint8_t* block, int lane, int j) {
  return reinterpret_cast<uint4*>(block) + (F32 ? lane * 8 + (j ^ (lane & 7)) : lane * 4 + (j ^ ((lane >> 1) & 3)));
}

// One 32 x 32 block of the outputs: this lane's row c, columns l .. l + 31, the
// sums at TMEM address t.  16 columns at a time they become z and y in the
// warp's stage, and leave by TMA stores of the whole block.  The stage's 4 KB
// hold two bf16 blocks, either one after the other (a block is computed while
// the one before it is read) or y and z of one, or one fp32 block.
template <bool FWD, int ACT, bool F32>
__device__ __forceinline__ void output_block(const LinearParams& p, const LinearMaps& maps, uint32_t t, int l, long long c,
                                             int row0, uint8_t* stage, int& buf, int lane, bool has_z) {
  const bool single = F32 || has_z;
  uint8_t* y_block = stage + (single ? 0 : buf * 2048);
  uint8_t* z_block = stage + 2048;
  if (lane == 0) {   // the copies that last read this buffer are done reading
    if (single)
      bulk_wait_read<0>();
    else
      bulk_wait_read<1>();
  }
  __syncwarp();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[16];
    tmem_ld16(t + 16 * h, v);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float* z = v + 8 * j;
      const int lj = l + 16 * h + 8 * j;
      if constexpr (FWD) {
        if (p.bias && lj < p.L) {
          float b[8];
          load_vals<8>(p.bias, p.bias_f32, lj, b);
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] += b[i];
        }
        if (has_z)
          *stage_piece<false>(z_block, lane, 2 * h + j) =
              make_uint4(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]), pack_bf16(z[4], z[5]), pack_bf16(z[6], z[7]));
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = act_value<ACT>(z[i]);
        if (p.residual && lj < p.L && c < p.C) {
          float r[8];
          load_vals<8, false>(p.residual, p.residual_f32, c * p.L + lj, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] += r[i];
        }
      }
      if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          *stage_piece<true>(y_block, lane, 4 * h + 2 * j + i) =
              make_uint4(__float_as_uint(z[4 * i]), __float_as_uint(z[4 * i + 1]), __float_as_uint(z[4 * i + 2]),
                         __float_as_uint(z[4 * i + 3]));
      } else {
        *stage_piece<false>(y_block, lane, 2 * h + j) =
            make_uint4(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]), pack_bf16(z[4], z[5]), pack_bf16(z[6], z[7]));
      }
    }
  }
  fence_proxy_async_smem();   // generic-proxy writes, then the async-proxy reads
  __syncwarp();
  if (lane == 0) {
    if (has_z) tma_store_2d(&maps.z, z_block, l, row0);
    tma_store_2d(&maps.out, y_block, l, row0);
    bulk_commit();
  }
  buf ^= 1;
}

// The pre-activations of one block alone.
__device__ __forceinline__ void z_only_block(const LinearParams& p, const LinearMaps& maps, uint32_t t, int l, int row0,
                                             uint8_t* stage, int lane) {
  if (lane == 0) bulk_wait_read<0>();
  __syncwarp();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[16];
    tmem_ld16(t + 16 * h, v);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float* z = v + 8 * j;
      const int lj = l + 16 * h + 8 * j;
      if (p.bias && lj < p.L) {
        float b[8];
        load_vals<8>(p.bias, p.bias_f32, lj, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] += b[i];
      }
      *stage_piece<false>(stage, lane, 2 * h + j) =
          make_uint4(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]), pack_bf16(z[4], z[5]), pack_bf16(z[6], z[7]));
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(&maps.z, stage, l, row0);
    bulk_commit();
  }
}

template <int ACT>
__device__ __forceinline__ void forward_block(const LinearParams& p, const LinearMaps& maps, uint32_t t, int l, long long c,
                                              int row0, uint8_t* stage, int& buf, int lane) {
  if (!p.out_f32) {
    output_block<true, ACT, false>(p, maps, t, l, c, row0, stage, buf, lane, p.z != nullptr);
    return;
  }
  if (p.z) z_only_block(p, maps, t, l, row0, stage, lane);   // the stage does not hold both
  output_block<true, ACT, true>(p, maps, t, l, c, row0, stage, buf, lane, false);
}

// ---------------------------------------------------------------- pair split kernel
template <bool AMN, bool BMN>
struct PairSplitCfg {
  static constexpr int kStageBytes = PairCfg<AMN, BMN>::kStageBytes;
  static constexpr int kStages = 6;
  static constexpr int kSmemBytes = 1024 + kStages * kStageBytes + 256;
  // the epilogue and the join wait on latencies: 16 warps of them
  static constexpr int kEpiWarps = 16;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr uint32_t kIdesc = PairCfg<AMN, BMN>::kIdesc;
  static_assert(128 * 256 * 4 <= kStages * kStageBytes, "the partial tile fits the stages");
};

// Where float4 column c4 of row r of a part [128][256] lies (in units of 16
// bytes): neighbouring rows' same column falls into different banks.
__device__ __forceinline__ int part_at(int r, int c4) { return r * 64 + (c4 ^ (r & 7)); }

// The join of a pair tile: this CTA's share of its 128 rows, from the S CTAs
// that hold parts of the same rows, in rank order.
template <bool FWD, int ACT, int S>
__device__ __forceinline__ void join_rows(const LinearParams& p, const float* part, int rank, long long l0, int c0, int warp,
                                          int lane) {
  constexpr int kWarps = 16, kAtOnce = S <= 2 ? 4 : 2;
  const int share = rank >> 1, r0 = 128 * share / S, rows = min(128 * (share + 1) / S, p.C - c0) - r0;
  uint32_t peer[S];
#pragma unroll
  for (int s = 0; s < S; ++s) peer[s] = cluster_addr(part, 2 * s + (rank & 1));
  // a warp's tasks: halves (128 columns) of rows, a fixed half for each warp
  const int h = warp & 1;
  const long long l = l0 + h * 128 + lane * 4;
  if (l >= p.L) return;
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  if (FWD && p.bias) load_vals<4>(p.bias, p.bias_f32, l, bias);
  for (int r = warp >> 1; r < rows; r += kWarps / 2 * kAtOnce) {
    float res[kAtOnce][4] = {}, v[kAtOnce][4] = {};
    float4 t[kAtOnce][S];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int ru = r0 + min(r + kWarps / 2 * u, rows - 1);   // past the end: the last row again, not stored
      if (FWD && p.residual) load_vals<4, false>(p.residual, p.residual_f32, static_cast<long long>(c0 + ru) * p.L + l, res[u]);
#pragma unroll
      for (int s = 0; s < S; ++s)
        t[u][s] = part_of<S>(part, peer, s, share, static_cast<uint32_t>(part_at(ru, h * 32 + lane)) * 16u);
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
#pragma unroll
      for (int s = 0; s < S; ++s) v[u][0] += t[u][s].x, v[u][1] += t[u][s].y, v[u][2] += t[u][s].z, v[u][3] += t[u][s].w;
      const int ru = r + kWarps / 2 * u;
      if (ru < rows) store_four<ACT>(p, static_cast<long long>(c0 + r0 + ru) * p.L + l, bias, v[u], res[u]);
    }
  }
}

template <bool FWD, int ACT>
__device__ __forceinline__ void join_pairs(const LinearParams& p, const float* part, int rank, long long l0, int c0, int warp,
                                           int lane) {
  switch (p.split) {
    case 1: join_rows<FWD, ACT, 1>(p, part, rank, l0, c0, warp, lane); break;
    case 2: join_rows<FWD, ACT, 2>(p, part, rank, l0, c0, warp, lane); break;
    case 3: join_rows<FWD, ACT, 3>(p, part, rank, l0, c0, warp, lane); break;
    default: join_rows<FWD, ACT, 4>(p, part, rank, l0, c0, warp, lane); break;
  }
}

// grid {2 S x tiles}, clusters of S pairs along K.  4096 x 256 x 7168 in fp32:
// 20.6 us, of which the products take 12 on the 96 SMs that clusters of six
// fill, and the join 4; 1003 x 1416 x 2056 14.8 us.
// CHUNKED: as for linear_split_kernel; 4096 x 256 x 7168 20.9 us so and 20.5 in two
// accumulators, 1800 x 1800 x 4096 26.1 and 25.7.
template <bool AMN, bool BMN, bool FWD, bool CHUNKED>
__global__ void __launch_bounds__(PairSplitCfg<AMN, BMN>::kThreads, 1) linear_pair_split_kernel(const __grid_constant__ LinearMaps maps, const LinearParams p) {
  using C = PairSplitCfg<AMN, BMN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kStages * C::kStageBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;   // (the second, and tempty: CHUNKED)
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.split, rank = static_cast<int>(cluster_rank()), lead = rank & ~1;
  const int tile = blockIdx.x / (2 * S), lt = tile % p.l_tiles, ct = tile / p.l_tiles;
  const long long l0 = static_cast<long long>(lt) * 256;
  const int c0 = ct * 256 + (rank & 1) * 128;   // this CTA's rows
  const int kb0 = static_cast<int>(static_cast<long long>(p.nk) * (rank >> 1) / S);
  const int kb1 = static_cast<int>(static_cast<long long>(p.nk) * ((rank >> 1) + 1) / S);
  // fp32 outputs: the K range in two accumulators (see linear_split_kernel)
  const bool two = FWD && !CHUNKED && p.out_f32 && kb1 - kb0 > 1;
  const int kbm = two ? (kb0 + kb1) / 2 : kb1;
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
  cluster_sync();   // all barriers are there before any signal crosses
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tmem_base = *tmem_slot;
  if (warp == 0) {
    int stage = 0, fills = 0;
    uint32_t phase = 0;
    bool ok = true;
    const uint32_t lead_full = cluster_addr(full, lead);
    const int la = static_cast<int>(l0) + (rank & 1) * 128;   // this CTA's half of the columns' operand
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!warp_wait(&empty[stage], phase ^ 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      uint8_t* sB = smem + stage * C::kStageBytes;
      uint8_t* sA = sB + kLinABytes;
      const uint32_t bar = lead_full + stage * 8;
      const int k0 = kb * kLinBK;
      if (elect_one()) {
        if (rank == lead) mbar_arrive_expect_tx(&full[stage], 2 * C::kStageBytes);
        if (AMN) {
          tma_load_2d_pair(sA, &maps.a, bar, la, k0);
          tma_load_2d_pair(sA + kLinChunk, &maps.a, bar, la + 64, k0);
        } else {
          tma_load_2d_pair(sA, &maps.a, bar, k0, la);
        }
        if (BMN) {
          tma_load_2d_pair(sB, &maps.b, bar, c0, k0);
          tma_load_2d_pair(sB + kLinChunk, &maps.b, bar, c0 + 64, k0);
        } else {
          tma_load_2d_pair(sB, &maps.b, bar, k0, c0);
        }
      }
      __syncwarp();
      ++fills;
      if (++stage == C::kStages) stage = 0, phase ^= 1;
    }
    if (!ok && rank == lead && lane == 0) {   // no load may be in flight when the CTA ends
      const int n = min(fills, C::kStages);
      for (int i = 0; i < n; ++i) {
        if (--stage < 0) stage = C::kStages - 1, phase ^= 1;
        mbar_drain(&full[stage], phase);
      }
    }
  } else if (warp == 1) {
    if (rank == lead) {
      const uint64_t bd = linear_desc<BMN>(smem_u32(smem)), ad = linear_desc<AMN>(smem_u32(smem) + kLinABytes);
      const uint16_t both = static_cast<uint16_t>(3u << lead), me = static_cast<uint16_t>(1u << lead);
      int stage = 0, buf = 0, in = 0;   // CHUNKED: the accumulator, and the block's place in its chunk
      uint32_t phase = 0, bphase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (CHUNKED && in == 0) {
          if (!warp_wait(&tempty[buf], bphase ^ 1, abort_flag, p.status)) break;
          tc_fence_after();
        }
        if (!warp_wait(&full[stage], phase, abort_flag, p.status)) break;
        const uint32_t at = stage * C::kStageBytes, acc = tmem_base + (CHUNKED ? buf * 256 : kb >= kbm ? 256 : 0);
        const bool last = CHUNKED ? in == kChunk - 1 || kb == kb1 - 1 : kb == kb1 - 1;
        if (elect_one()) {
          umma_bf16_pair(acc, desc_at(bd, at), desc_at(ad, at), C::kIdesc, CHUNKED ? in != 0 : kb != kb0 && kb != kbm);
#pragma unroll
          for (int kk = 1; kk < kLinBK / 16; ++kk)
            umma_bf16_pair(acc, desc_at(bd, at + kk * kStep<BMN>), desc_at(ad, at + kk * kStep<AMN>), C::kIdesc, 1u);
          umma_commit_pair(&empty[stage], both);
          if (last) umma_commit_pair(&tfull[CHUNKED ? buf : 0], both);
        }
        __syncwarp();
        if (CHUNKED && ++in == kChunk) {
          in = 0;
          buf ^= 1;
          if (buf == 0) bphase ^= 1;
        }
        if (++stage == C::kStages) stage = 0, phase ^= 1;
      }
      if (elect_one()) {
        umma_commit_pair(done, me);
        mbar_drain(done, 0);
      }
    }
  } else {
    constexpr int kCols = 256 * 4 / C::kEpiWarps;   // this warp's columns
    const int q = warp & 3, col0 = ((warp - 2) >> 2) * kCols, row = q * 32 + lane;
    if (FWD && p.residual) {   // this CTA's share of it into L2 while the accumulator fills
      const int size = p.residual_f32 ? 4 : 2, r1 = min(128 * ((rank >> 1) + 1) / S, p.C - c0);
      const long long cols = p.L - l0 < 256 ? p.L - l0 : 256;
      for (int r = 128 * (rank >> 1) / S + warp - 2; r < r1; r += C::kEpiWarps)
        for (long long o = lane * 128; o < cols * size; o += 32 * 128)
          prefetch_l2(static_cast<const char*>(p.residual) + (static_cast<long long>(c0 + r) * p.L + l0) * size + o);
    }
    const uint32_t tb = tmem_base + col0 + (static_cast<uint32_t>(q * 32) << 16);
    float4* part = reinterpret_cast<float4*>(smem);
    const auto wait_full = [&](uint64_t* bar, uint32_t parity) {
      const int w = lane == 0 ? (mbar_wait(bar, parity, abort_flag, p.status) ? 1 : 0) : 0;
      const bool got = __shfl_sync(0xffffffffu, w, 0) != 0;
      tc_fence_after();
      return got;
    };
    if constexpr (CHUNKED) {
      float sum[kCols] = {};
      bool ok = true;
      int buf = 0;
      uint32_t bphase = 0;
      for (int first = kb0; first < kb1; first += kChunk) {
        if (!(ok = wait_full(&tfull[buf], bphase))) break;
        add_columns<kCols>(tb + buf * 256, sum);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank != lead)
            mbar_arrive_cluster(cluster_addr(&tempty[buf], lead));
          else
            mbar_arrive(&tempty[buf]);
        }
        buf ^= 1;
        if (buf == 0) bphase ^= 1;
      }
      if (ok) {
#pragma unroll
        for (int c = 0; c < kCols; c += 4)
          part[part_at(row, (col0 + c) / 4)] = make_float4(sum[c], sum[c + 1], sum[c + 2], sum[c + 3]);
      }
    } else if (wait_full(tfull, 0)) {
#pragma unroll 1
      for (int c = 0; c < kCols; c += 16) {
        float v[16];
        tmem_ld16(tb + c, v);
        if (two) {
          float u[16];
          tmem_ld16(tb + 256 + c, u);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] += u[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          part[part_at(row, (col0 + c) / 4 + i)] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  cluster_sync();   // every CTA's part is in its shared memory
  const float* part = reinterpret_cast<const float*>(smem);
  if (warp >= 2) switch (FWD ? p.act : LIN_NONE) {
    case LIN_RELU: join_pairs<FWD, FWD ? LIN_RELU : LIN_NONE>(p, part, rank, l0, c0, warp - 2, lane); break;
    case LIN_SILU: join_pairs<FWD, FWD ? LIN_SILU : LIN_NONE>(p, part, rank, l0, c0, warp - 2, lane); break;
    case LIN_GELU: join_pairs<FWD, FWD ? LIN_GELU : LIN_NONE>(p, part, rank, l0, c0, warp - 2, lane); break;
    case LIN_GELU_TANH: join_pairs<FWD, FWD ? LIN_GELU_TANH : LIN_NONE>(p, part, rank, l0, c0, warp - 2, lane); break;
    default: join_pairs<FWD, LIN_NONE>(p, part, rank, l0, c0, warp - 2, lane); break;
  }
  __syncwarp();
  cluster_sync();   // nobody reads this CTA's shared memory or writes its TMEM any more
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// ---------------------------------------------------------------- persistent pair kernel
// Bound by the tensor core: 16384 x 8192 x 2048 281 us (1.96 PFLOP/s), with GELU
// and z kept 320 us, 8192 x 8192 x 8192 580 to 600 us (the power limit); both
// gradients of 8192 x 4096 x 2048 141 us, tensor pipe active 93% of cycles.
//
// The products of one launch: one, or the backward's two (the one with the
// longer tiles first).
struct PairJob {
  LinearMaps maps[2];
  LinearParams p[2];
  int b_mn[2];    // the products' B is MN-major (LIN_GRADS)
  int problems;
  int extra;      // see pair_item
};

struct PairItem {
  int w;       // the product
  int lt, ct;  // its tile
};

// Work item s of pair `pair`.  The first product's n0 tiles go round the pairs
// in turn, which leaves h = n0 % pairs of them a tile ahead.  Two products: the
// other pairs first take `extra` tiles of the second, about as long as one of
// the first, and what then remains goes round all pairs again, so that all end
// together (two launches each end with pairs that stand still).
__device__ __forceinline__ bool pair_item(const PairJob& job, int s, int pair, int pairs, PairItem& it) {
  const int n0 = job.p[0].l_tiles * job.p[0].c_tiles;
  int idx = pair + s * pairs;
  it.w = 0;
  if (idx >= n0) {
    if (job.problems == 1) return false;
    const int h = n0 % pairs, s2 = s - (n0 / pairs + (pair < h ? 1 : 0)), mine = pair < h ? 0 : job.extra;
    idx = s2 < mine ? s2 * (pairs - h) + pair - h : job.extra * (pairs - h) + (s2 - mine) * pairs + pair;
    if (idx >= job.p[1].l_tiles * job.p[1].c_tiles) return false;
    it.w = 1;
  }
  linear_tile(job.p[it.w], idx, it.lt, it.ct);
  return true;
}

// KIND: the forward as LIN_FWD, LIN_FWD_SHORT (over few K-blocks) or
// LIN_FWD_F32 (over more than kChunk of them into fp32), or a gradient.
template <int KIND>
constexpr bool kIsForward = KIND == LIN_FWD || KIND == LIN_FWD_SHORT || KIND == LIN_FWD_F32;
template <int KIND>
using PairKindCfg = PairCfg<!kIsForward<KIND>, false, KIND == LIN_FWD_SHORT>;

// What the chunks cost here: while a tile's outputs are made, the products are at
// most a chunk ahead; 8192 x 4864 outputs, in one go and in chunks, K = 1024 61
// and 69 us, K = 2048 91 and 103, K = 4096 168 and 183; 4096 x 8192 x 7168 271 to
// 298 and 279 to 289.  Sixteen epilogue warps: 73, 109 and 195 us.
template <int KIND>
__global__ void __launch_bounds__(PairKindCfg<KIND>::kThreads, 1) linear_pair_kernel(const __grid_constant__ PairJob job) {
  constexpr bool FWD = kIsForward<KIND>, AMN = !FWD, CHUNKED = KIND == LIN_FWD_F32;
  using C = PairKindCfg<KIND>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* out_stage = smem + C::kStages * C::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(out_stage + C::kEpiWarps * C::kOutBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  int* const status = job.p[0].status;
  const auto b_is_mn = [&](int w) { return KIND == LIN_GRADS ? job.b_mn[w] != 0 : KIND == LIN_DW; };
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
    tma_prefetch_desc(&job.maps[0].a);
    tma_prefetch_desc(&job.maps[0].b);
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
    int stage = 0;
    uint32_t phase = 0;
    long long fills = 0;
    bool ok = true;
    const uint32_t lead_full = cluster_addr(full, 0);   // both CTAs' loads count on the leader's barriers
    PairItem it;
    for (int s = 0; ok && pair_item(job, s, pair, pairs, it); ++s) {
      const LinearMaps& maps = job.maps[it.w];
      const bool b_mn = b_is_mn(it.w);
      const int l0 = it.lt * 256 + rank * 128, c0 = it.ct * 256 + rank * 128, nk = job.p[it.w].nk;
      for (int kb = 0; kb < nk; ++kb) {
        if (!warp_wait(&empty[stage], phase ^ 1, abort_flag, status)) {
          ok = false;
          break;
        }
        // the tensor core's rows are c: its first operand is b
        uint8_t* sB = smem + stage * C::kStageBytes;
        uint8_t* sA = sB + kLinABytes;
        const uint32_t bar = lead_full + stage * 8;
        const int k0 = kb * kLinBK;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * C::kStageBytes);
          if (AMN) {
            tma_load_2d_pair(sA, &maps.a, bar, l0, k0);
            tma_load_2d_pair(sA + kLinChunk, &maps.a, bar, l0 + 64, k0);
          } else {
            tma_load_2d_pair(sA, &maps.a, bar, k0, l0);
          }
          if (b_mn) {
            tma_load_2d_pair(sB, &maps.b, bar, c0, k0);
            tma_load_2d_pair(sB + kLinChunk, &maps.b, bar, c0 + 64, k0);
          } else {
            tma_load_2d_pair(sB, &maps.b, bar, k0, c0);
          }
        }
        __syncwarp();
        ++fills;
        if (++stage == C::kStages) stage = 0, phase ^= 1;
      }
    }
    if (!ok && rank == 0 && lane == 0) {   // no load may be in flight when the CTA ends
      const int n = fills < C::kStages ? static_cast<int>(fills) : C::kStages;
      for (int i = 0; i < n; ++i) {
        if (--stage < 0) stage = C::kStages - 1, phase ^= 1;
        mbar_drain(&full[stage], phase);
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const uint64_t ad = linear_desc<AMN>(smem_u32(smem) + kLinABytes);
      int stage = 0, buf = 0;
      uint32_t phase = 0, bphase = 0;
      bool ok = true;
      PairItem it;
      for (int s = 0; ok && pair_item(job, s, pair, pairs, it); ++s) {
        const bool b_mn = b_is_mn(it.w);
        const uint64_t bd = b_mn ? linear_desc<true>(smem_u32(smem)) : linear_desc<false>(smem_u32(smem));
        const uint32_t b_step = b_mn ? kStep<true> : kStep<false>;
        const uint32_t idesc = b_mn ? idesc_bf16(256, C::BN, true, AMN) : idesc_bf16(256, C::BN, false, AMN);
        const int nk = job.p[it.w].nk;
        for (int first = 0; ok && first < nk; first += CHUNKED ? kChunk : nk) {
          if (!warp_wait(&tempty[buf], bphase ^ 1, abort_flag, status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int end = CHUNKED ? min(first + kChunk, nk) : nk;
          const uint32_t acc = tmem_base + static_cast<uint32_t>(buf * C::BN);
          for (int kb = first; kb < end; ++kb) {
            if (!warp_wait(&full[stage], phase, abort_flag, status)) {
              ok = false;
              break;
            }
            const uint32_t at = stage * C::kStageBytes;
            if (elect_one()) {
              umma_bf16_pair(acc, desc_at(bd, at), desc_at(ad, at), idesc, kb != first);
#pragma unroll
              for (int kk = 1; kk < kLinBK / 16; ++kk)
                umma_bf16_pair(acc, desc_at(bd, at + kk * b_step), desc_at(ad, at + kk * kStep<AMN>), idesc, 1u);
              umma_commit_pair(&empty[stage], 0x3);
              if (kb == end - 1) umma_commit_pair(&tfull[buf], 0x3);
            }
            __syncwarp();
            if (++stage == C::kStages) stage = 0, phase ^= 1;
          }
          buf ^= 1;
          if (buf == 0) bphase ^= 1;
        }
      }
      if (elect_one()) {
        umma_commit_pair(done, 0x1);
        mbar_drain(done, 0);
      }
    }
  } else {
    constexpr int kCols = C::BN * 4 / C::kEpiWarps;   // this warp's columns
    const int q = warp & 3, col0 = ((warp - 2) >> 2) * kCols;
    uint8_t* stage = out_stage + (warp - 2) * C::kOutBytes;
    int buf = 0, slot = 0;
    uint32_t bphase = 0;
    PairItem it;
    for (int s = 0; pair_item(job, s, pair, pairs, it); ++s) {
      const LinearMaps& maps = job.maps[it.w];
      const LinearParams& p = job.p[it.w];
      const int l0 = it.lt * 256 + col0, row0 = it.ct * 256 + rank * 128 + q * 32;
      const long long c = static_cast<long long>(row0) + lane;
      if (FWD && p.residual && c < p.C) {   // into L2 while the accumulator fills
        const long long size = p.residual_f32 ? 4 : 2, end = p.L - l0 < kCols ? p.L - l0 : kCols;
        const char* r = static_cast<const char*>(p.residual) + (c * p.L + l0) * size;
        for (long long o = 0; o < end * size; o += 128) prefetch_l2(r + o);
      }
      const auto wait_full = [&]() {
        const int w = lane == 0 ? (mbar_wait(&tfull[buf], bphase, abort_flag, status) ? 1 : 0) : 0;
        const bool got = __shfl_sync(0xffffffffu, w, 0) != 0;
        tc_fence_after();
        return got;
      };
      const auto release = [&]() {
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
      };
      const auto own_columns = [&]() {
        return tmem_base + static_cast<uint32_t>(buf * C::BN + col0) + (static_cast<uint32_t>(q * 32) << 16);
      };
      if constexpr (CHUNKED) {
        // all chunks but the last in registers, then onto the last one's, in
        // TMEM, from where the outputs are made
        float sum[kCols] = {};
        bool ok = true;
        for (int first = 0; first + kChunk < p.nk; first += kChunk) {
          if (!(ok = wait_full())) break;
          add_columns<kCols>(own_columns(), sum);
          release();
        }
        if (!ok || !wait_full()) break;
        add_columns<kCols, true>(own_columns(), sum);
      } else {
        if (!wait_full()) break;
      }
      const uint32_t tb = own_columns();
#pragma unroll 1
      for (int k = 0; k < kCols && l0 + k < p.L && row0 < p.C; k += 32) {
        if constexpr (FWD) {
          switch (p.act) {
            case LIN_RELU: forward_block<LIN_RELU>(p, maps, tb + k, l0 + k, c, row0, stage, slot, lane); break;
            case LIN_SILU: forward_block<LIN_SILU>(p, maps, tb + k, l0 + k, c, row0, stage, slot, lane); break;
            case LIN_GELU: forward_block<LIN_GELU>(p, maps, tb + k, l0 + k, c, row0, stage, slot, lane); break;
            case LIN_GELU_TANH: forward_block<LIN_GELU_TANH>(p, maps, tb + k, l0 + k, c, row0, stage, slot, lane); break;
            default: forward_block<LIN_NONE>(p, maps, tb + k, l0 + k, c, row0, stage, slot, lane); break;
          }
        } else {
          output_block<false, LIN_NONE, false>(p, maps, tb + k, l0 + k, c, row0, stage, slot, lane, false);
        }
      }
      release();
    }
    if (lane == 0) bulk_wait<0>();   // this warp's stores are complete before the CTA ends
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
