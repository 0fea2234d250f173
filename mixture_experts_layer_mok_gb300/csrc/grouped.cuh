// Matrix products grouped by expert on tcgen05 / TMEM / TMA: the rows of each
// group lie one after the other, without padding, and their counts are on the
// device.
//
//   rows kernel    D[l][c] = sum_k A[l][k] B[c][k], c the rows of one group:
//     forward  l = n, k = k:  A = W_e [N][K],                B = x rows
//     dx       l = k, k = n:  A = W_e^T (W_e is [k][l]),     B = dz rows
//   weight kernel  D[c][l] = sum_m dz[m][c] x[m][l], m the rows of one group.
//
// Measured, the rows kernel in short graph replays: 32768 rows of 64 groups of 1024
// x 2048 with SiLU and z 106 us (DRAM and tensor pipe 58% busy each), 131072 of 2048
// x 4096 1200 to 1240, 512 rows of 256 groups of 2048 x 7168 780 (the weights' bytes).
// Calls in a long loop take 118 to 120, 1400 to 1413 (the power limit) and 785 to 833.
//
// Both are persistent CTA pairs with two accumulator buffers.  In the rows
// kernel the weights run over the tensor core's M (256 over two SMs) and a
// group's rows over its N, which is any multiple of 32 up to 256: a group of 300
// rows costs 320, not 512, and a group of two costs 32; one kernel serves the
// decoded token, bound by the weights' bytes, and the long batch, bound by the
// tensor core.  A group's rows are cut evenly into tiles of at most 256.
// Rows that a tile's loads bring in from the next group fill columns that are
// not stored.  The weight kernel contracts over the rows, where a neighbour's
// row must not come in: it reads through tensor maps that end with the group
// (grouped_plan_kernel writes them), so that the hardware fills in zeros.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "experts.h"
#include "gemm.cuh"
#include "linear.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace mok {

constexpr int kGroupedStageBytes = 2 * kLinABytes;   // 128 x 64 of A, up to 128 x 64 of B

// ---------------------------------------------------------------- the groups
struct GroupTable {
  int start[kMaxGroups + 1];   // first row of each group, and the end of the last
  int tile[kMaxGroups + 1];    // row tiles before each group, and all of them
  int full, last, parts;       // items that are not cut, the rest, and into how many parts these are
};

// By one warp: the table from the counts.  Counts below 0 count as 0 and rows
// behind M as none; returns whether there were any.
__device__ __forceinline__ bool scan_groups(const int* counts, int E, int M, int* start, int* tile, int lane) {
  const int each = (E + 31) / 32, e0 = min(lane * each, E), e1 = min(e0 + each, E);
  long long sum = 0;
  bool bad = false;
  for (int e = e0; e < e1; ++e) {
    const int c = __ldg(counts + e);
    bad |= c < 0;
    sum += max(c, 0);
  }
  long long before = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  bad |= before > M;
  before -= sum;
  int tiles = 0;
  long long at = before;
  for (int e = e0; e < e1; ++e) {
    const int s = static_cast<int>(min(at, static_cast<long long>(M)));
    at += max(__ldg(counts + e), 0);
    const int n = static_cast<int>(min(at, static_cast<long long>(M))) - s;
    start[e] = s;
    tiles += (n + 255) / 256;
  }
  if (e1 == E && e0 < e1) start[E] = static_cast<int>(min(at, static_cast<long long>(M)));
  if (tile) {
    int t = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += v;
    }
    t -= tiles;
    __syncwarp();
    for (int e = e0; e < e1; ++e) {
      tile[e] = t;
      t += ((e + 1 < e1 ? start[e + 1] : static_cast<int>(min(at, static_cast<long long>(M)))) - start[e] + 255) / 256;
    }
    if (e1 == E && e0 < e1) tile[E] = t;
  }
  __syncwarp();
  return __any_sync(0xffffffffu, bad);
}

// The last e with tab[e] <= q, for tab ascending with tab[0] = 0, by a warp.
__device__ __forceinline__ int find_group(const int* tab, int E, int q, int lane) {
  const int far = lane * 32;
  const int seg = __popc(__ballot_sync(0xffffffffu, far < E && tab[far] <= q)) - 1;
  const int near = seg * 32 + lane;
  return seg * 32 + __popc(__ballot_sync(0xffffffffu, near < E && tab[near] <= q)) - 1;
}

// ---------------------------------------------------------------- rows kernel
struct GroupedRowsMaps {
  CUtensorMap w;      // [E][L][K], boxes 64 x 128, or [E][K][L], boxes 64 x 64
  CUtensorMap x[4];   // [M][K], boxes of 64 x 16, 32, 64 and 128
};

// fp32 outputs leave from registers: room for twice the epilogue warps, whose
// activations and stores are what the last tile of a pair ends with.
template <bool F32>
struct GroupedRowsCfg {
  static constexpr int kStages = 6, kEpiWarps = F32 ? 16 : 8, kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kStageOut = F32 ? 0 : 2048;   // an epilogue warp's 32 rows x 32 columns in bf16
  static constexpr int kSmemBytes =
      1024 + kStages * kGroupedStageBytes + kEpiWarps * kStageOut + static_cast<int>(sizeof(GroupTable)) + 256;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

// A length cut evenly into parts, in steps of 32: a part's length (count + parts
// may pass 2^31).
__host__ __device__ constexpr int even_part(int count, int parts) { return ((count - 1) / parts + 32) & ~31; }
static_assert(even_part(1, 1) == 32 && even_part(257, 2) == 160 && even_part(224, 3) == 96, "rounded up");
static_assert(even_part(0x7fffffff - 512, (0x7fffffff - 512 + 255) / 256) == 256, "the largest group");

struct RowsItem {
  int e, l0, m0, rows, n;   // group, first l, first row, rows, and the tensor core's N
};
// Item idx of tile[E] x l_tiles: a group's items are neighbours, and inside a
// group of 4 of its row tiles l goes on outside the rows, so that the CTAs at
// work at one time share few rows of both operands.  The last round's items,
// where half the pairs or more would have none, are cut by rows into up to 4
// parts, for each of which the tensor core takes less time: as many as a tile has
// whole 64s of rows, of equal length in steps of 32, so that the last may be short
// (200 rows: 96, 96 and 8).  256 rows of one group of 1024 x 4096 18 us, and 25 whole; 32768 rows of 64 groups 2 us
// less of 108; 16 rows of 8 groups, which are not cut, 0.2 us more of 8.
__device__ __forceinline__ bool rows_item(const GroupedRowsParams& p, const GroupTable& g, int idx, int lane, RowsItem& it) {
  int part = 0, parts = 1;
  if (idx >= g.full) {
    parts = g.parts;
    for (idx -= g.last; idx >= g.full; idx -= g.last)   // (parts times last are no more than the pairs, so that a pair has one of them)
      if (++part >= parts) return false;
    idx += g.last;
  }
  const int q = idx / p.l_tiles;
  it.e = find_group(g.tile, p.E, q, lane);
  const int t0 = g.tile[it.e], tiles = g.tile[it.e + 1] - t0, first = g.start[it.e], count = g.start[it.e + 1] - first;
  int ct, lt;
  unit_and_col(idx - t0 * p.l_tiles, tiles, p.l_tiles, 4, ct, lt);
  const int each = even_part(count, tiles);
  it.l0 = lt * 256;
  it.m0 = first + ct * each;
  it.rows = min(each, count - ct * each);
  if (parts > 1) {
    parts = max(min(parts, it.rows / 64), 1);
    const int rows = even_part(it.rows, parts);
    it.m0 += part * rows;
    it.rows = min(rows, it.rows - part * rows);
    if (it.rows <= 0) return false;
  }
  it.n = (it.rows + 31) & ~31;
  return true;
}

__device__ __forceinline__ void tma_load_rows_pair(uint8_t* dst, const CUtensorMap* maps, uint32_t bar, int k0, int row, int rows) {
#pragma unroll
  for (int b = 3; b >= 0; --b) {   // 128, 64, 32, 16: the bits of rows
    const int box = 16 << b;
    if (rows & box) {
      tma_load_2d_pair(dst, &maps[b], bar, k0, row);
      dst += box * 128;
      row += box;
    }
  }
}

// 16 TMEM lanes x 8 N columns in the fragment layout: register 4 i + {0, 1}:
// lane g = thread / 4, columns 8 i + 2 (thread % 4) + {0, 1}; + {2, 3}: lane g + 8.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Four 8 x 8 blocks of bf16 from the fragment layout, each transposed; lane 8 i +
// j names the address of block i's row j.
__device__ __forceinline__ void st_matrix_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ float bias_at(const GroupedRowsParams& p, int e, int l) {
  if (!p.bias || l >= p.L) return 0.f;
  const long long at = static_cast<long long>(e) * p.L + l;
  return p.bias_f32 ? __ldg(static_cast<const float*>(p.bias) + at)
                    : __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(p.bias) + at)) << 16);
}

// A staged block (32 rows of 64 bytes, 16-byte pieces swizzled) to rows row ..
// row + rows - 1 of out, columns l .. l + 31 as far as there are: 64 bytes of a
// row by four lanes.
__device__ __forceinline__ void store_block(const uint8_t* stage, uint16_t* out, int L, int l, long long row, int rows, int lane) {
  const int piece = lane & 3;
  if (l + piece * 8 >= L) return;   // L % 8 == 0
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2);
    const uint4 v = reinterpret_cast<const uint4*>(stage)[r * 4 + (piece ^ ((r >> 1) & 3))];
    if (r < rows) *reinterpret_cast<uint4*>(out + (row + r) * L + l + piece * 8) = v;
  }
}

// 32 rows x 32 l's in bf16 from TMEM at taddr (this warp's lanes, 32 columns):
// the fragments take bias and activation, and are transposed into the stage.
template <int ACT>
__device__ __forceinline__ void rows_block(const GroupedRowsParams& p, uint32_t taddr, const float (&bias)[4], int l, long long row,
                                           int rows, uint8_t* stage, int lane) {
  uint32_t r[2][16];
  tmem_ld_16x256b_x4(taddr, r[0]);
  tmem_ld_16x256b_x4(taddr + (16u << 16), r[1]);
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  float v[2][16];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      asm volatile("" : "+r"(r[h][i]));   // no use before the wait
      v[h][i] = __uint_as_float(r[h][i]) + bias[2 * h + ((i >> 1) & 1)];
    }
  // block (rows 8 i .., l's 16 h + 8 u ..) holds registers 4 i + 2 u, 4 i + 2 u + 1 of half h; this lane's
  // address: row 8 i + lane % 8 of the piece 2 h + u = lane / 8
  const uint32_t at = smem_u32(stage);
  const auto put = [&](auto value) {
    __syncwarp();   // the stage's last readers are done
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int h = b >> 1, u = b & 1;
        w[b] = pack_bf16(value(v[h][4 * i + 2 * u]), value(v[h][4 * i + 2 * u + 1]));
      }
      const int rr = 8 * i + (lane & 7), piece = lane >> 3;
      st_matrix_trans(at + rr * 64 + ((piece ^ ((rr >> 1) & 3)) << 4), w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
  };
  if (p.z) {
    put([](float x) { return x; });
    store_block(stage, p.z, p.L, l, row, rows, lane);
  }
  put([](float x) { return act_value<ACT>(x); });
  store_block(stage, static_cast<uint16_t*>(p.out), p.L, l, row, rows, lane);
}

// 32 columns of this lane's l, in fp32: a warp's 32 l's of a row are 128 bytes.
template <int ACT>
__device__ __forceinline__ void rows_block_f32(const GroupedRowsParams& p, const float* v, float bias, int l, long long row, int rows) {
  if (l >= p.L) return;
  float* out = static_cast<float*>(p.out);
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if (i >= rows) break;
    const float z = v[i] + bias;
    if (p.z) p.z[(row + i) * p.L + l] = static_cast<uint16_t>(pack_bf16(z, 0.f) & 0xffffu);
    out[(row + i) * p.L + l] = act_value<ACT>(z);
  }
}

// AMN: A is stored [k][l] (dx).  F32: fp32 outputs, whose sums over more than
// kChunk K-blocks are added in registers (linear.cuh).
template <bool AMN, bool F32>
__global__ void __launch_bounds__(GroupedRowsCfg<F32>::kThreads, 1) grouped_rows_kernel(const __grid_constant__ GroupedRowsMaps maps, const GroupedRowsParams p) {
  using C = GroupedRowsCfg<F32>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* out_stage = smem + C::kStages * kGroupedStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(out_stage + C::kEpiWarps * C::kStageOut);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  GroupTable& table = *reinterpret_cast<GroupTable*>(tmem_slot + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  int* const status = p.status;
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
    tma_prefetch_desc(&maps.w);
    for (int b = 0; b < 4; ++b) tma_prefetch_desc(&maps.x[b]);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  if (!p.beside_last) griddep_wait();
  griddep_launch_dependents();
  if (warp == 2) {
    const bool bad = scan_groups(p.counts, p.E, p.M, table.start, table.tile, lane);
    if (lane == 0) {
      const int all = table.tile[p.E] * p.l_tiles, last = all < pairs ? all : all % pairs;
      table.parts = 4 * last <= pairs ? 4 : 3 * last <= pairs ? 3 : 2 * last <= pairs ? 2 : 1;
      table.full = table.parts > 1 ? all - last : all;
      table.last = table.parts > 1 ? last : 0;
    }
    if (bad && blockIdx.x == 0 && lane == 0) atomicCAS(status, 0, MOK_ERR_INDEX);
  }
  tc_fence_before();
  cluster_sync();   // both CTAs' barriers and tables are there before any signal crosses
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if (warp == 0) {
    int stage = 0;
    uint32_t phase = 0;
    long long fills = 0;
    bool ok = true;
    const uint32_t lead_full = cluster_addr(full, 0);   // both CTAs' loads count on the leader's barriers
    RowsItem it;
    for (int idx = pair; ok && rows_item(p, table, idx, lane, it); idx += pairs) {
      const int l0 = it.l0 + rank * 128, half = it.n >> 1, m0 = it.m0 + rank * half;
      const uint32_t bytes = 2 * kLinABytes + it.n * 128;
      for (int kb = 0; kb < p.nk; ++kb) {
        if (!warp_wait(&empty[stage], phase ^ 1, abort_flag, status)) {
          ok = false;
          break;
        }
        uint8_t* sA = smem + stage * kGroupedStageBytes;
        const uint32_t bar = lead_full + stage * 8;
        const int k0 = kb * kLinBK;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], bytes);
          if (AMN) {
            tma_load_3d_pair(sA, &maps.w, bar, l0, k0, it.e);
            tma_load_3d_pair(sA + kLinChunk, &maps.w, bar, l0 + 64, k0, it.e);
          } else {
            tma_load_3d_pair(sA, &maps.w, bar, k0, l0, it.e);
          }
          tma_load_rows_pair(sA + kLinABytes, maps.x, bar, k0, m0, half);
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
      const uint64_t ad = linear_desc<AMN>(smem_u32(smem)), bd = linear_desc<false>(smem_u32(smem) + kLinABytes);
      int stage = 0, buf = 0;
      uint32_t phase = 0, bphase = 0;
      bool ok = true;
      RowsItem it;
      for (int idx = pair; ok && rows_item(p, table, idx, lane, it); idx += pairs) {
        const uint32_t idesc = idesc_bf16(256, it.n, AMN, false);
        for (int first = 0; ok && first < p.nk; first += F32 ? kChunk : p.nk) {
          if (!warp_wait(&tempty[buf], bphase ^ 1, abort_flag, status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int end = F32 ? min(first + kChunk, p.nk) : p.nk;
          const uint32_t acc = tmem_base + static_cast<uint32_t>(buf * 256);
          for (int kb = first; kb < end; ++kb) {
            if (!warp_wait(&full[stage], phase, abort_flag, status)) {
              ok = false;
              break;
            }
            const uint32_t at = stage * kGroupedStageBytes;
            if (elect_one()) {
              umma_bf16_pair(acc, desc_at(ad, at), desc_at(bd, at), idesc, kb != first);
#pragma unroll
              for (int kk = 1; kk < kLinBK / 16; ++kk)
                umma_bf16_pair(acc, desc_at(ad, at + kk * kStep<AMN>), desc_at(bd, at + kk * kStep<false>), idesc, 1u);
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
    // a quarter of the TMEM lanes, and of each kEpiWarps / 4 blocks of 32 columns one
    constexpr int kSide = C::kEpiWarps / 4, kBlocks = 8 / kSide;
    const int q = warp & 3, side = (warp - 2) >> 2;
    uint8_t* stage = out_stage + (warp - 2) * C::kStageOut;
    int buf = 0;
    uint32_t bphase = 0;
    bool ok = true;
    RowsItem it;
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
    for (int idx = pair; rows_item(p, table, idx, lane, it); idx += pairs) {
      const int l = it.l0 + rank * 128 + q * 32;   // this warp's l's
      const auto lanes = [&]() { return tmem_base + static_cast<uint32_t>(buf * 256) + (static_cast<uint32_t>(q * 32) << 16); };
      if constexpr (F32) {
        float sum[kBlocks][32] = {};
        for (int first = 0; first < p.nk; first += kChunk) {
          if (!(ok = wait_full())) break;
#pragma unroll
          for (int b = 0; b < kBlocks; ++b)
            if ((kSide * b + side) * 32 < it.n) add_columns<32>(lanes() + (kSide * b + side) * 32, sum[b]);
          release();
        }
        if (!ok) break;
        const float bias = bias_at(p, it.e, l + lane);
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          const int c = (kSide * b + side) * 32, rows = it.rows - c;
          if (rows <= 0) continue;
          const long long row = it.m0 + c;
          switch (p.act) {
            case LIN_RELU: rows_block_f32<LIN_RELU>(p, sum[b], bias, l + lane, row, rows); break;
            case LIN_SILU: rows_block_f32<LIN_SILU>(p, sum[b], bias, l + lane, row, rows); break;
            case LIN_GELU: rows_block_f32<LIN_GELU>(p, sum[b], bias, l + lane, row, rows); break;
            case LIN_GELU_TANH: rows_block_f32<LIN_GELU_TANH>(p, sum[b], bias, l + lane, row, rows); break;
            default: rows_block_f32<LIN_NONE>(p, sum[b], bias, l + lane, row, rows); break;
          }
        }
      } else {
        float bias[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) bias[i] = bias_at(p, it.e, l + 8 * i + (lane >> 2));
        if (!wait_full()) break;
#pragma unroll 1
        for (int c = side * 32; c < it.n && l < p.L; c += 32 * kSide) {
          const int rows = it.rows - c;
          const long long row = it.m0 + c;
          const uint32_t t = lanes() + c;
          switch (AMN ? LIN_NONE : p.act) {
            case LIN_RELU: rows_block<AMN ? LIN_NONE : LIN_RELU>(p, t, bias, l, row, rows, stage, lane); break;
            case LIN_SILU: rows_block<AMN ? LIN_NONE : LIN_SILU>(p, t, bias, l, row, rows, stage, lane); break;
            case LIN_GELU: rows_block<AMN ? LIN_NONE : LIN_GELU>(p, t, bias, l, row, rows, stage, lane); break;
            case LIN_GELU_TANH: rows_block<AMN ? LIN_NONE : LIN_GELU_TANH>(p, t, bias, l, row, rows, stage, lane); break;
            default: rows_block<LIN_NONE>(p, t, bias, l, row, rows, stage, lane); break;
          }
        }
        release();
      }
    }
    // zeros behind the last group, 16 bytes a lane
    const long long first = static_cast<long long>(table.start[p.E]) * p.L, end = static_cast<long long>(p.M) * p.L;
    const long long at = (static_cast<long long>(blockIdx.x) * C::kEpiWarps + warp - 2) * 32 + lane;
    const long long step = static_cast<long long>(gridDim.x) * C::kEpiWarps * 32;
    for (long long i = first + at * 8; i < end; i += step * 8) {   // L % 8 == 0
      const uint4 none = make_uint4(0u, 0u, 0u, 0u);
      if (F32) {
        reinterpret_cast<uint4*>(static_cast<float*>(p.out) + i)[0] = none;
        reinterpret_cast<uint4*>(static_cast<float*>(p.out) + i)[1] = none;
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + i) = none;
      }
      if (p.z) *reinterpret_cast<uint4*>(p.z + i) = none;
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();   // the leader's MMAs into both TMEMs are done
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
  if (p.beside_last) griddep_wait();   // what follows this kernel follows that one too
}

// ---------------------------------------------------------------- weight kernel
struct GroupedWeightMaps {
  CUtensorMap out;    // [E][N][K], boxes of 32 x 64
};
struct GroupedWeightParams {
  const int* starts;        // [E + 1]
  const CUtensorMap* dz;    // [E] maps of dz's rows up to the group's end, boxes 64 x 64
  const CUtensorMap* x;     // [E] of x's
  int E, N, K;
  int n_tiles, k_tiles;
  GroupedBias bias;
  int* status;
};
// 16 epilogue warps, each of which stores a block of 128-byte rows.  64 groups
// of 1024 x 2048 take 110 us with 512 rows each and 70 with one: a tile's own chain of
// loads, products and reads (58 without the stores), not the 268 MB, which a fill
// writes in 37 (7.3 TB/s).
struct GroupedWeightCfg {
  static constexpr int kStages = 5, kEpiWarps = 16, kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kOutBytes = 4096;   // an epilogue warp's 32 x 64 block in bf16
  static constexpr int kSmemBytes = 1024 + kStages * kGroupedStageBytes + kEpiWarps * kOutBytes + 256;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

// A tensor map in global memory that another kernel wrote: before its first use.
__device__ __forceinline__ void tensormap_acquire(const CUtensorMap* map) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

struct WeightItem {
  int e, n0, k0, first, end;
  __device__ __forceinline__ int nk() const { return (end - first + kLinBK - 1) / kLinBK; }
};
// Groups one after the other, k outside n inside groups of 8 n tiles.  The rows
// come from global memory: an item is looked up one ahead of its use.
__device__ __forceinline__ WeightItem weight_item(const GroupedWeightParams& p, int idx) {
  WeightItem it = {};
  const int per = p.n_tiles * p.k_tiles;
  it.e = idx / per;
  if (it.e >= p.E) return it;
  int nt, kt;
  unit_and_col(idx - it.e * per, p.n_tiles, p.k_tiles, 8, nt, kt);
  it.n0 = nt * 256;
  it.k0 = kt * 256;
  it.first = __ldg(p.starts + it.e);
  it.end = __ldg(p.starts + it.e + 1);
  return it;
}

// The bias's gradient from the parts that grouped_dz_kernel left (grouped.cu), a
// group's in order; thread `at` of `threads`.
__device__ __forceinline__ void grouped_bias_sums(const GroupedBias& b, const int* starts, int E, int N, long long at, long long threads) {
  for (long long i = at; i < static_cast<long long>(E) * N; i += threads) {
    const int e = static_cast<int>(i / N), col = static_cast<int>(i - static_cast<long long>(e) * N);
    const int r0 = __ldg(starts + e), r1 = __ldg(starts + e + 1);
    float v = 0.f;
    if (r0 < r1) {
      const float* part = b.part + (static_cast<long long>(r0 / b.chunk) + e) * N + col;
      const int n = (r1 - 1) / b.chunk - r0 / b.chunk + 1;
#pragma unroll 4
      for (int c = 0; c < n; ++c) v += part[static_cast<long long>(c) * N];
    }
    b.out[i] = v;
  }
}

// The pair kernel of linear.cuh with both operands MN-major, over the groups'
// rows; a group without rows gets zeros.
__global__ void __launch_bounds__(GroupedWeightCfg::kThreads, 1) grouped_weight_kernel(const __grid_constant__ GroupedWeightMaps maps, const GroupedWeightParams p) {
  using C = GroupedWeightCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* out_stage = smem + C::kStages * kGroupedStageBytes;
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
  int* const status = p.status;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * C::kEpiWarps);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&maps.out);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  griddep_wait();   // before the next kernel may start: see GroupedRowsParams::beside_last
  griddep_launch_dependents();
  const uint32_t tmem_base = *tmem_slot;
  if (warp == 0) {
    int stage = 0, e = -1;
    uint32_t phase = 0;
    long long fills = 0;
    bool ok = true;
    const uint32_t lead_full = cluster_addr(full, 0);
    WeightItem it, next = weight_item(p, pair);
    for (int idx = pair; ok && next.e < p.E; idx += pairs) {
      it = next;
      const int nk = it.nk();
      next = weight_item(p, idx + pairs);
      if (nk > 0 && it.e != e) {   // (every lane: any may be elected)
        e = it.e;
        tensormap_acquire(p.dz + e);
        tensormap_acquire(p.x + e);
        __syncwarp();
      }
      const int c0 = it.n0 + rank * 128, l0 = it.k0 + rank * 128;
      for (int kb = 0; kb < nk; ++kb) {
        if (!warp_wait(&empty[stage], phase ^ 1, abort_flag, status)) {
          ok = false;
          break;
        }
        uint8_t* sB = smem + stage * kGroupedStageBytes;
        uint8_t* sA = sB + kLinABytes;
        const uint32_t bar = lead_full + stage * 8;
        const int r0 = it.first + kb * kLinBK;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * kGroupedStageBytes);
          tma_load_2d_pair(sB, p.dz + e, bar, c0, r0);
          tma_load_2d_pair(sB + kLinChunk, p.dz + e, bar, c0 + 64, r0);
          tma_load_2d_pair(sA, p.x + e, bar, l0, r0);
          tma_load_2d_pair(sA + kLinChunk, p.x + e, bar, l0 + 64, r0);
        }
        __syncwarp();
        ++fills;
        if (++stage == C::kStages) stage = 0, phase ^= 1;
      }
    }
    if (!ok && rank == 0 && lane == 0) {
      const int n = fills < C::kStages ? static_cast<int>(fills) : C::kStages;
      for (int i = 0; i < n; ++i) {
        if (--stage < 0) stage = C::kStages - 1, phase ^= 1;
        mbar_drain(&full[stage], phase);
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const uint64_t bd = linear_desc<true>(smem_u32(smem)), ad = linear_desc<true>(smem_u32(smem) + kLinABytes);
      constexpr uint32_t idesc = idesc_bf16(256, 256, true, true);
      int stage = 0, buf = 0;
      uint32_t phase = 0, bphase = 0;
      bool ok = true;
      WeightItem it, next = weight_item(p, pair);
      for (int idx = pair; ok && next.e < p.E; idx += pairs) {
        it = next;
        const int nk = it.nk();
        next = weight_item(p, idx + pairs);
        if (nk == 0) continue;
        if (!warp_wait(&tempty[buf], bphase ^ 1, abort_flag, status)) break;
        tc_fence_after();
        const uint32_t acc = tmem_base + static_cast<uint32_t>(buf * 256);
        for (int kb = 0; kb < nk; ++kb) {
          if (!warp_wait(&full[stage], phase, abort_flag, status)) {
            ok = false;
            break;
          }
          const uint32_t at = stage * kGroupedStageBytes;
          if (elect_one()) {
            umma_bf16_pair(acc, desc_at(bd, at), desc_at(ad, at), idesc, kb != 0);
#pragma unroll
            for (int kk = 1; kk < kLinBK / 16; ++kk)
              umma_bf16_pair(acc, desc_at(bd, at + kk * kStep<true>), desc_at(ad, at + kk * kStep<true>), idesc, 1u);
            umma_commit_pair(&empty[stage], 0x3);
            if (kb == nk - 1) umma_commit_pair(&tfull[buf], 0x3);
          }
          __syncwarp();
          if (++stage == C::kStages) stage = 0, phase ^= 1;
        }
        buf ^= 1;
        if (buf == 0) bphase ^= 1;
      }
      if (elect_one()) {
        umma_commit_pair(done, 0x1);
        mbar_drain(done, 0);
      }
    }
  } else {
    const int q = warp & 3, col0 = ((warp - 2) >> 2) * 64;   // this warp's rows and columns of the tile
    uint8_t* stage = out_stage + (warp - 2) * C::kOutBytes;
    int buf = 0;
    uint32_t bphase = 0;
    WeightItem it, next = weight_item(p, pair);
    if (p.bias.out)   // while the first tile is made
      grouped_bias_sums(p.bias, p.starts, p.E, p.N, (blockIdx.x * C::kEpiWarps + warp - 2) * 32 + lane, gridDim.x * C::kEpiWarps * 32);
    for (int idx = pair; next.e < p.E; idx += pairs) {
      it = next;
      const int nk = it.nk();
      next = weight_item(p, idx + pairs);
      const int n = it.n0 + rank * 128 + q * 32, k = it.k0 + col0;
      const bool in = n < p.N && k < p.K;
      uint32_t w[32];
      if (nk > 0) {
        const int got = lane == 0 ? (mbar_wait(&tfull[buf], bphase, abort_flag, status) ? 1 : 0) : 0;
        const bool ok = __shfl_sync(0xffffffffu, got, 0) != 0;
        tc_fence_after();
        if (!ok) break;
        if (in) {
          const uint32_t tb = tmem_base + static_cast<uint32_t>(buf * 256 + col0) + (static_cast<uint32_t>(q * 32) << 16);
          const uint32_t at[2] = {tb, tb + 32};
          float v[64];
          tmem_ld32_multi<2>(at, v);
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = 0u;
      }
      if (nk > 0) {
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
      if (in) {
        if (lane == 0) bulk_wait_read<0>();   // the copy that last read the block is done reading
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)   // rows of 128 bytes, 16-byte pieces swizzled by the row
          reinterpret_cast<uint4*>(stage)[lane * 8 + (j ^ (lane & 7))] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&maps.out, stage, k, n, it.e);
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait<0>();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

}  // namespace mok
