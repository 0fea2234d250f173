// Products with 4-bit weights (int4.cu has the layout) on tcgen05: one matrix, its
// rows 128 to a CTA.
//
//   y[c][n] = act(sum over groups of scale[n][group] (sum_k (q - zero)[n][k] x[c][k]) + bias[n])
//
// A thread has a row of w.  It makes the row's codes, less the zero, whole numbers
// in bf16 and puts them into TMEM as the tensor core's left operand; the right one
// is x in shared memory, with the tokens (16, 32 or 64) as columns.  The sums of a
// group are exact products added in fp32; another thread of the same row reads
// them back, scales them and adds them up, so that no weight is rounded.
// What it costs is the instructions of the codes: 3 shifts, 4 masks and 4
// additions for 8 of them, whatever the number of tokens; the products of mma.sync
// would cost as much again for every 8 tokens.  32 tokens times 152064 x 4096: 97
// us (mma.sync 135), issue slots 66% busy, DRAM 43%, the tensor core's pipe 23%.
//
// Two pipelines take a CTA's blocks of K in turn, each with an issuer, sums, and
// buffers of its own: from one block to the next of a pipeline there are four
// waits in a row (codes, products, sums, buffer) of some hundred cycles each,
// and the products themselves take few.  Their sums are added at the end.
// Few rows of w: K is split over a cluster, whose parts are added in rank order.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "api_util.h"
#include "clusters.h"
#include "experts.h"
#include "gemm.cuh"
#include "internal.h"
#include "linear.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace mok {
namespace {

// Warps: the codes' (four for both pipelines, or with 64 tokens, whose sums leave
// room for one CTA only, four for each), four for the sums of each, two issuers.
template <int NT, int GPB, bool ZEROS>
struct Int4TcCfg {
  static constexpr int kRows = 128, kCtas = NT == 64 ? 1 : 2;       // kCtas: on an SM
  static constexpr int kCodeWarps = NT == 64 ? 8 : 4, kSumWarp = kCodeWarps, kMmaWarp = kSumWarp + 8;
  static constexpr int kThreads = 32 * (kMmaWarp + 2);
  static constexpr int kXStages = 2, kXBytes = NT * 256;            // of a pipeline; a block of x: two chunks of 64 columns
  static constexpr int kCodeStages = 6, kZeroBytes = ZEROS ? 32 * GPB : 0;
  static constexpr int kCodeBytes = 32 * 64 + kZeroBytes;           // a warp's 32 rows of a block
  static constexpr int kScaleStages = 4, kScaleBytes = 64 * GPB;    // likewise
  static constexpr int kSums = NT == 64 ? 1 : 2;                    // groups' sums of a pipeline in TMEM
  static constexpr int kTmemCols = 256;                             // two blocks of codes (64 each), then the sums
  static constexpr int kPartBytes = NT * kRows * 4;                 // sums of the CTA, over the stages of x and codes
  static constexpr int kUsedBytes = 2 * kXStages * kXBytes + kCodeWarps * kCodeStages * kCodeBytes + 8 * kScaleStages * kScaleBytes;
  // enough that the SM holds no more CTAs than TMEM does: one that waits for TMEM while others of its cluster hold some
  // could wait for ever
  static constexpr int kLeast = 77 * 1024;
  static constexpr int kSmemBytes = kUsedBytes + 1280 < kLeast ? kLeast : kUsedBytes + 1280;
  static_assert(128 + 2 * kSums * NT <= kTmemCols, "TMEM");
  static_assert(kPartBytes <= 2 * kXStages * kXBytes + kCodeWarps * kCodeStages * kCodeBytes, "the part fits the stages");
  static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "shared memory");
};

struct Int4TcParams {
  Int4LinearArgs a;
  int split;   // CTAs of a cluster along K
};

// The codes of columns 2 i, 2 i + 1 of a word less the zero, as bf16: z holds
// -(128 + zero) twice.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i, uint32_t z) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w >> (4 * i)), "r"(0x000F000Fu), "r"(0x43004300u));   // (a & b) | c
  asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(z));
  return v;
}

// 32 registers into 32 columns of this thread's TMEM lane, not waited on.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]^T, bf16, fp32 accumulate: A's lane is its row, a
// column holds two neighbours along K.
__device__ __forceinline__ void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// a0 += s v0, a1 += s v1 in one instruction.
__device__ __forceinline__ void fma_pair(float& a0, float& a1, float s, float v0, float v1) {
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmov.b64 c, {%3, %4};\n\t"
      "fma.rn.f32x2 a, b, c, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(s), "f"(v0), "f"(v1));
}

template <int ACT>
__device__ __forceinline__ void store_act(const Int4LinearArgs& a, long long row, int n, float v) {
  const long long at = row * a.w.N + n;
  v = act_value<ACT>(v);
  if (a.out_f32)
    static_cast<float*>(a.y)[at] = v;
  else
    static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ float row_bias(const Int4LinearArgs& a, int n) {
  if (!a.bias) return 0.f;
  return a.bias_f32 ? __ldg(static_cast<const float*>(a.bias) + n)
                    : __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(a.bias) + n)) << 16);
}

// grid {S x groups of 128 rows of w, rows of x in steps of NT}, clusters of S.
template <int NT, int GPB, bool ZEROS>
__global__ void __launch_bounds__(Int4TcCfg<NT, GPB, ZEROS>::kThreads, Int4TcCfg<NT, GPB, ZEROS>::kCtas) int4_tc_kernel(const __grid_constant__ CUtensorMap xmap, const Int4TcParams p) {
  using C = Int4TcCfg<NT, GPB, ZEROS>;
  const Int4LinearArgs& a = p.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* code_ring = smem + 2 * C::kXStages * C::kXBytes;
  uint8_t* scale_ring = code_ring + C::kCodeWarps * C::kCodeStages * C::kCodeBytes;
  // per pipeline and stage of x, for the block that is in it: its codes and its x are there; its products are made
  uint64_t* ready = reinterpret_cast<uint64_t*>(scale_ring + 8 * C::kScaleStages * C::kScaleBytes);
  uint64_t* made = ready + 2 * C::kXStages;
  // per pipeline and buffer of sums: a group's are there (of a block's last group made says so); they have been read
  uint64_t* d_full = made + 2 * C::kXStages;
  uint64_t* d_empty = d_full + 2 * C::kSums;
  uint64_t* done = d_empty + 2 * C::kSums;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.split, rank = S > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int nb = a.w.blocks(), row_tiles = static_cast<int>(a.w.row_tiles());
  const int tile = blockIdx.x / S, c0 = blockIdx.y * NT, cols = min(NT, a.rows - c0);
  const int kb0 = static_cast<int>(static_cast<long long>(nb) * rank / S), kb1 = static_cast<int>(static_cast<long long>(nb) * (rank + 1) / S);
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2 * C::kXStages; ++s) {
      mbar_init(&ready[s], 5);   // four warps' codes, and the copy of x
      mbar_init(&made[s], 1);
    }
    for (int b = 0; b < 2 * C::kSums; ++b) {
      mbar_init(&d_full[b], 1);
      mbar_init(&d_empty[b], 4);
    }
    for (int w = 0; w < 2; ++w) mbar_init(&done[w], 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&xmap);
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  // the row tiles of a warp of 32 rows (behind the last one: that one again, not stored)
  const int q = warp & 3;
  const auto warp_tile = [&](int h) { return static_cast<long long>(min(tile * 8 + 2 * q + h, row_tiles - 1)) * nb; };
  // block number n of pipeline w is the CTA's block 2 n + w; its stage and parity of x, and those of its group d's sums
  const int blocks = kb1 - kb0;
  const auto x_stage = [](int w, int n) { return w * C::kXStages + n % C::kXStages; };
  const auto x_phase = [](int n) { return static_cast<uint32_t>(n / C::kXStages) & 1u; };
  const auto d_buffer = [](int w, int d) { return w * C::kSums + d % C::kSums; };
  const auto d_phase = [](int d) { return static_cast<uint32_t>(d / C::kSums) & 1u; };
  float acc[NT];
#pragma unroll
  for (int c = 0; c < NT; ++c) acc[c] = 0.f;
  if (warp < C::kCodeWarps) {
    // ---- codes: a row's 64 bytes of a block, 16-byte pieces t at t ^ (row / 2) % 4, so that eight rows meet all banks
    uint8_t* ring = code_ring + warp * (C::kCodeStages * C::kCodeBytes);
    // this lane's copies: pieces lane, lane + 32 of each tile (row piece / 4, t = piece % 4), and of zeros one or none
    constexpr int kStep = C::kCodeWarps / 4;   // it makes every block, or every other one from its own on
    const int first = kStep == 2 ? warp >> 2 : 0;
    const uint8_t* src[2];
    uint32_t dst[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      src[h] = a.codes + (warp_tile(h) + kb0 + first) * kInt4TileBytes + lane * 16;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = h * 16 + u * 8 + (lane >> 2);
        dst[h][u] = row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4);
      }
    }
    const uint8_t* zsrc = nullptr;
    if (ZEROS && lane < 2 * GPB) zsrc = a.zeros + (warp_tile(lane / GPB) + kb0 + first) * (16 * GPB) + lane % GPB * 16;
    int to = 0, left = blocks - first;
    const auto fetch = [&]() {
      if (left > 0) {
        uint8_t* st = ring + to * C::kCodeBytes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          cp_async16(st + dst[h][0], src[h], 16);
          cp_async16(st + dst[h][1], src[h] + 512, 16);
          src[h] += kStep * kInt4TileBytes;
        }
        if (ZEROS && lane < 2 * GPB) {
          cp_async16(st + 2048 + lane * 16, zsrc, 16);
          zsrc += kStep * 16 * GPB;
        }
        left -= kStep;
        if (++to == C::kCodeStages) to = 0;
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < C::kCodeStages - 1; ++i) fetch();
    int at = 0;
    for (int i = first; i < blocks; i += kStep) {
      cp_async_wait<C::kCodeStages - 2>();
      __syncwarp();   // every lane's copies are there, and the stage that is filled next has been read
      fetch();
      const uint8_t* st = ring + at * C::kCodeBytes;
      uint4 w[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) w[t] = *reinterpret_cast<const uint4*>(st + lane * 64 + ((t ^ ((lane >> 1) & 3)) << 4));
      uint32_t z = 0;
      if constexpr (ZEROS) {
        if constexpr (GPB == 4)
          z = *reinterpret_cast<const uint32_t*>(st + 2048 + lane * 4);
        else if constexpr (GPB == 2)
          z = *reinterpret_cast<const uint16_t*>(st + 2048 + lane * 2);
        else
          z = st[2048 + lane];
      }
      const int w2 = i & 1, n2 = i >> 1;   // the pipeline, whose TMEM the last of its blocks has left
      if (n2 > 0 && !warp_wait(&made[x_stage(w2, n2 - 1)], x_phase(n2 - 1), abort_flag, a.status)) break;
      tc_fence_after();
      const uint32_t to_tmem = tmem + w2 * 64 + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
      for (int h = 0; h < 2; ++h) {   // words j = 2 h, 2 h + 1 of each piece: columns 64 h .. + 63
        uint32_t r[32];
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
          const int j = 2 * h + jj, gr = j * GPB / 4;
          const uint32_t zero = ZEROS ? __byte_perm(z, 0xC3u, 0x4040u + 0x0101u * gr) : 0xC308C308u;
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint32_t word = j == 0 ? w[t].x : j == 1 ? w[t].y : j == 2 ? w[t].z : w[t].w;
#pragma unroll
            for (int u = 0; u < 4; ++u) r[16 * jj + 4 * t + u] = code_pair(word, u, zero);
          }
        }
        tmem_st32(to_tmem + 32 * h, r);
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ready[x_stage(w2, n2)]);
      if (++at == C::kCodeStages) at = 0;
    }
    cp_async_wait<0>();
  } else if (warp < C::kMmaWarp) {
    // ---- sums, and the pipeline's x
    const int w = (warp - C::kSumWarp) >> 2, mine = (blocks - w + 1) / 2;
    uint8_t* ring = scale_ring + (warp - C::kSumWarp) * (C::kScaleStages * C::kScaleBytes);
    const uint8_t* src = nullptr;   // this lane's piece of the scales, or none
    if (lane < 4 * GPB)
      src = reinterpret_cast<const uint8_t*>(a.scales) + (warp_tile(lane / (2 * GPB)) + kb0 + w) * (32 * GPB) + lane % (2 * GPB) * 16;
    int fetched = 0, loaded = 0;
    const auto fetch = [&]() {
      if (fetched < mine) {
        if (lane < 4 * GPB) {
          cp_async16(ring + fetched % C::kScaleStages * C::kScaleBytes + lane * 16, src, 16);
          src += 64 * GPB;
        }
        ++fetched;
      }
      cp_async_commit();
    };
    // x, by the first of the warps: the first blocks, and then one for each that has been made
    const auto load_x = [&]() {
      if (q == C::kSumWarp % 4 && loaded < mine) {
        const int s = x_stage(w, loaded), k = (kb0 + 2 * loaded + w) * kInt4Block;
        if (elect_one()) {
          mbar_arrive_expect_tx(&ready[s], C::kXBytes);
          tma_load_2d(smem + s * C::kXBytes, &xmap, &ready[s], k, c0);
          tma_load_2d(smem + s * C::kXBytes + NT * 128, &xmap, &ready[s], k + 64, c0);
        }
        __syncwarp();
        ++loaded;
      }
    };
    for (int i = 0; i < C::kXStages; ++i) load_x();
#pragma unroll
    for (int i = 0; i < C::kScaleStages - 1; ++i) fetch();
    bool ok = true;
    for (int i = 0; ok && i < mine; ++i) {
      cp_async_wait<C::kScaleStages - 2>();
      __syncwarp();   // the scales are there, and the stage that is filled next has been read
      fetch();
      const uint16_t* sc = reinterpret_cast<const uint16_t*>(ring + i % C::kScaleStages * C::kScaleBytes) + lane * GPB;
#pragma unroll
      for (int gr = 0; gr < GPB; ++gr) {
        const float s = __uint_as_float(static_cast<uint32_t>(sc[gr]) << 16);
        if (gr < GPB - 1) {
          const int f = i * (GPB - 1) + gr;   // the group's number among those but the last of their blocks
          if (!(ok = warp_wait(&d_full[d_buffer(w, f)], d_phase(f), abort_flag, a.status))) break;
        } else {
          if (!(ok = warp_wait(&made[x_stage(w, i)], x_phase(i), abort_flag, a.status))) break;
          load_x();
        }
        tc_fence_after();
        const int db = d_buffer(w, i * GPB + gr);
        const uint32_t from = tmem + 128 + db * NT + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
          float v[16];
          tmem_ld16(from + c, v);
#pragma unroll
          for (int u = 0; u < 16; u += 2) fma_pair(acc[c + u], acc[c + u + 1], s, v[u], v[u + 1]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&d_empty[db]);
      }
    }
    cp_async_wait<0>();
    if (!ok && q == C::kSumWarp % 4 && lane == 0) {   // no load may be in flight when the CTA ends (where codes are missing: the wait's limit)
      for (int i = loaded < C::kXStages ? 0 : loaded - C::kXStages; i < loaded; ++i) mbar_drain(&ready[x_stage(w, i)], x_phase(i));
    }
  } else {
    // ---- products
    constexpr uint32_t idesc = idesc_bf16(128, NT, false, false);
    constexpr int kSteps = 8 / GPB;   // of 16 columns, to a group
    const uint64_t xd = linear_desc<false>(smem_u32(smem));
    const int w = warp - C::kMmaWarp, mine = (blocks - w + 1) / 2;
    bool ok = true;
#pragma unroll 1
    for (int i = 0; ok && i < mine; ++i) {
      const int stage = x_stage(w, i);
      if (!warp_wait(&ready[stage], x_phase(i), abort_flag, a.status)) break;
#pragma unroll
      for (int gr = 0; gr < GPB; ++gr) {
        const int d = i * GPB + gr, db = d_buffer(w, d);
        if (!(ok = warp_wait(&d_empty[db], d_phase(d) ^ 1, abort_flag, a.status))) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int u = 0; u < kSteps; ++u) {
            const int k = gr * kSteps + u;   // step of the block: chunk k / 4, 32 bytes each inside
            umma_bf16_ta(tmem + 128 + db * NT, tmem + w * 64 + k * 8,
                         desc_at(xd, stage * C::kXBytes + (k >> 2) * (NT * 128) + (k & 3) * 32), idesc, u != 0);
          }
          umma_commit(gr < GPB - 1 ? &d_full[d_buffer(w, i * (GPB - 1) + gr)] : &made[stage]);
        }
        __syncwarp();
      }
    }
    if (elect_one()) {
      umma_commit(&done[w]);   // every MMA issued here ends before TMEM is released
      mbar_drain(&done[w], 0);
    }
  }
  __syncwarp();
  // the second pipeline's sums to the first's warps
  float* part = reinterpret_cast<float*>(smem) + q * 32 + lane;   // [NT][128], this thread's row of w
  const bool sums = warp >= C::kSumWarp && warp < C::kMmaWarp, second = warp >= C::kSumWarp + 4;
  __syncthreads();   // the stages are read and filled no more
  if (sums && second) {
#pragma unroll
    for (int c = 0; c < NT; ++c) part[c * C::kRows] = acc[c];
  }
  __syncthreads();
  if (sums && !second) {
#pragma unroll
    for (int c = 0; c < NT; ++c) acc[c] += part[c * C::kRows];
  }
  const int n = tile * C::kRows + q * 32 + lane;
  if (S == 1) {
    if (sums && !second && n < a.w.N) {
      const float bias = row_bias(a, n);
      const auto store = [&](auto act) {
#pragma unroll
        for (int c = 0; c < NT; ++c)
          if (c < cols) store_act<decltype(act)::value>(a, c0 + c, n, acc[c] + bias);
      };
      switch (a.act) {
        case LIN_RELU: store(std::integral_constant<int, LIN_RELU>()); break;
        case LIN_SILU: store(std::integral_constant<int, LIN_SILU>()); break;
        case LIN_GELU: store(std::integral_constant<int, LIN_GELU>()); break;
        case LIN_GELU_TANH: store(std::integral_constant<int, LIN_GELU_TANH>()); break;
        default: store(std::integral_constant<int, LIN_NONE>()); break;
      }
    }
    tc_fence_before();
    __syncthreads();
  } else {
    if (sums && !second) {
#pragma unroll
      for (int c = 0; c < NT; ++c) part[c * C::kRows] = acc[c];
    }
    __syncwarp();
    cluster_sync();   // every CTA's part is there
    // this CTA's share of the columns, a row of w to a thread
    if (warp < 12) {
      const int r = threadIdx.x & 127, row = tile * C::kRows + r;
      if (row < a.w.N) {
        const float* at = reinterpret_cast<const float*>(smem) + r;
        const float bias = row_bias(a, row);
        const int end = min(cols, (rank + 1) * NT / S);
        for (int c = rank * NT / S + (threadIdx.x >> 7); c < end; c += 3) {
          float v = 0.f;
          for (int s = 0; s < S; ++s) {
            float u;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(u) : "r"(cluster_addr(at + c * C::kRows, s)));
            v += u;
          }
          v += bias;
          switch (a.act) {
            case LIN_RELU: store_act<LIN_RELU>(a, c0 + c, row, v); break;
            case LIN_SILU: store_act<LIN_SILU>(a, c0 + c, row, v); break;
            case LIN_GELU: store_act<LIN_GELU>(a, c0 + c, row, v); break;
            case LIN_GELU_TANH: store_act<LIN_GELU_TANH>(a, c0 + c, row, v); break;
            default: store_act<LIN_NONE>(a, c0 + c, row, v); break;
          }
        }
      }
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();   // nobody reads this CTA's shared memory any more
  }
  if (warp == C::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int NT, int GPB, bool ZEROS>
mok_status_t tc_launch(const CUtensorMap& xmap, const Int4LinearArgs& a, cudaStream_t st) {
  using C = Int4TcCfg<NT, GPB, ZEROS>;
  auto kern = int4_tc_kernel<NT, GPB, ZEROS>;
  static KernelInfo info;
  Int4TcParams p = {a, 1};
  const long long tiles = (static_cast<long long>(a.w.N) + C::kRows - 1) / C::kRows, ct = (a.rows + NT - 1) / NT;
  int n = 0;
  MOK_CUDA(resident_clusters(kern, info, C::kThreads, C::kSmemBytes, 1, &n));
  // the split of K for which the waves of CTAs take the fewest blocks of K, a CTA's start and end counted as 16 (as 3, 8 and 16:
  // 32 rows times 40960 x 4096 53, 47 and 44 us, times 16384 x 8192 32 us each)
  constexpr double kFixed = 16;
  double least = 0.0;
  for (int s = 1; s <= 8 && a.w.blocks() / s >= 2; s *= 2) {
    MOK_CUDA(resident_clusters(kern, info, C::kThreads, C::kSmemBytes, s, &n));
    n *= C::kCtas;   // (the query counts one CTA to an SM)
    const double t = static_cast<double>((tiles * ct + n - 1) / n) * ((a.w.blocks() + s - 1) / s + kFixed);
    if (s == 1 || t < least) least = t, p.split = s;
  }
  MOK_CUDA(launch_clusters(kern, dim3(static_cast<unsigned>(tiles * p.split), static_cast<unsigned>(ct)), C::kThreads, C::kSmemBytes, p.split, st,
                           xmap, p));
  return MOK_OK;
}

template <int NT>
mok_status_t tc_columns(const Int4LinearArgs& a, cudaStream_t st) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(MOK_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  CUtensorMap m;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.w.K), static_cast<cuuint64_t>(a.rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.w.K) * 2};
  const cuuint32_t box[2] = {64, NT}, estr[2] = {1, 1};
  const CUresult r = fn(&m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(a.x), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(MOK_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d) for [%d x %d]", static_cast<int>(r), a.rows, a.w.K);
  const bool z = a.zeros != nullptr;
  if (a.w.group == 32) return z ? tc_launch<NT, 4, true>(m, a, st) : tc_launch<NT, 4, false>(m, a, st);
  if (a.w.group == 64) return z ? tc_launch<NT, 2, true>(m, a, st) : tc_launch<NT, 2, false>(m, a, st);
  return z ? tc_launch<NT, 1, true>(m, a, st) : tc_launch<NT, 1, false>(m, a, st);
}

}  // namespace

mok_status_t run_int4_tc(const Int4LinearArgs& a, cudaStream_t st) {
  if (a.rows <= 16) return tc_columns<16>(a, st);
  if (a.rows <= 32) return tc_columns<32>(a, st);
  return tc_columns<64>(a, st);
}

}  // namespace mok
