// 4-bit weights with a scale (and a zero) for each group of 32, 64 or 128 along
// K: their layout, its writers and reader, and the products with few rows.
//
//   w[n][k] = (q[n][k] - zero[n][k / group]) scale[n][k / group],  q in 0..15
//
// Layout: tiles of 16 rows n x 128 columns k, 1024 bytes each, row tile by row
// tile and along K within one.  A tile is what a warp's 32 lanes load as two
// 16-byte pieces each, rows 0..7 and then 8..15: lane (g, t) = (lane / 4, lane %
// 4) holds row g, and its word j the columns 32 j + 8 t .. + 7, so that a word
// never leaves a group and the four lanes of a row hold 32 neighbouring columns.
// In a word the codes of columns 2 i and 2 i + 1 are the nibbles i and i + 4, so
// that a shift, a mask and an exponent make a pair of bf16 values 128 + q of it.
// A tile's scales are [16 rows][groups of the block], and its zeros too.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "api_util.h"
#include "experts.h"
#include "gemm.cuh"
#include "internal.h"
#include "linear.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace mok {
namespace {

// ---------------------------------------------------------------- writers and reader
// 256 threads to a tile: thread (row, p) has the columns 8 p .. 8 p + 7 of a row.
struct TilePlace {
  long long tile;
  long long row;     // of the matrices, one after the other
  int r, p, k;       // row in the tile, piece, first column
  bool in;           // the row and the columns exist
};
__device__ __forceinline__ TilePlace tile_place(const Int4Shape& s) {
  TilePlace t;
  t.tile = static_cast<long long>(blockIdx.x) + static_cast<long long>(blockIdx.y) * gridDim.x;
  t.r = threadIdx.x >> 4;
  t.p = threadIdx.x & 15;
  const int nb = s.blocks();
  const long long rt = t.tile / nb, m = rt / s.row_tiles();
  const long long n = (rt - m * s.row_tiles()) * kInt4Rows + t.r;
  t.k = static_cast<int>(t.tile - rt * nb) * kInt4Block + 8 * t.p;
  t.in = n < s.N && t.k < s.K;
  t.row = m * s.N + n;
  return t;
}
// Where thread (r, p)'s word lies in its tile.
__device__ __forceinline__ int word_at(int r, int p) { return (r >> 3) * 512 + ((r & 7) * 4 + (p & 3)) * 16 + (p >> 2) * 4; }
__device__ __forceinline__ uint32_t interleave(const int (&q)[8]) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) w |= static_cast<uint32_t>(q[2 * i]) << (4 * i) | static_cast<uint32_t>(q[2 * i + 1]) << (4 * i + 16);
  return w;
}
__device__ __forceinline__ int code_of(uint32_t w, int i) { return (w >> (4 * (i >> 1) + 16 * (i & 1))) & 15; }

__device__ __forceinline__ float bf16_round(float v) { return __bfloat162float(__float2bfloat16_rn(v)); }

// Symmetric: scale = bf16(amax / 7), q = round(w / scale) + 8; with zeros: the
// range [lo, hi] that holds 0, scale = bf16((hi - lo) / 15), zero = round(-lo /
// scale), q = round(w / scale) + zero; both clamped to 0..15.
template <bool F32, bool ZEROS>
__global__ void __launch_bounds__(256) int4_quantize_kernel(const void* __restrict__ w, const Int4Shape s, uint8_t* __restrict__ codes,
                                                            uint16_t* __restrict__ scales, uint8_t* __restrict__ zeros) {
  griddep_wait();
  griddep_launch_dependents();
  const TilePlace t = tile_place(s);
  if (t.tile >= s.tiles()) return;   // whole blocks
  float v[8] = {};
  if (t.in) load_vals<8>(w, F32, t.row * s.K + t.k, v);
  float lo = 0.f, hi = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) lo = fminf(lo, v[i]), hi = fmaxf(hi, v[i]);
  for (int o = 1; o < s.group / 8; o <<= 1) {   // the group's threads: 4, 8 or 16 neighbours
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float scale = bf16_round(ZEROS ? (hi - lo) / 15.f : fmaxf(-lo, hi) / 7.f);
  float zero = 8.f;
  if (ZEROS) zero = scale > 0.f ? fminf(fmaxf(rintf(-lo / scale), 0.f), 15.f) : 0.f;
  int q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = scale > 0.f ? static_cast<int>(fminf(fmaxf(rintf(v[i] / scale) + zero, 0.f), 15.f)) : static_cast<int>(zero);
  *reinterpret_cast<uint32_t*>(codes + t.tile * kInt4TileBytes + word_at(t.r, t.p)) = interleave(q);
  const int each = s.group / 8, gpb = kInt4Block / s.group;
  if (t.p % each == 0) {
    const long long at = t.tile * s.tile_scales() + t.r * gpb + t.p / each;
    scales[at] = __bfloat16_as_ushort(__float2bfloat16_rn(scale));
    if (ZEROS) zeros[at] = static_cast<uint8_t>(zero);
  }
}

// From row-major codes, two to a byte, the even column's in the low half.
__global__ void __launch_bounds__(256) int4_pack_kernel(const uint8_t* __restrict__ qp, const uint16_t* __restrict__ qs,
                                                        const uint8_t* __restrict__ qz, const Int4Shape s, uint8_t* __restrict__ codes,
                                                        uint16_t* __restrict__ scales, uint8_t* __restrict__ zeros) {
  griddep_wait();
  griddep_launch_dependents();
  const TilePlace t = tile_place(s);
  if (t.tile >= s.tiles()) return;
  const uint32_t four = t.in ? __ldg(reinterpret_cast<const uint32_t*>(qp + (t.row * s.K + t.k) / 2)) : 0u;
  int q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = (four >> (4 * i)) & 15;
  *reinterpret_cast<uint32_t*>(codes + t.tile * kInt4TileBytes + word_at(t.r, t.p)) = interleave(q);
  const int each = s.group / 8, gpb = kInt4Block / s.group;
  if (t.p % each == 0) {
    const long long at = t.tile * s.tile_scales() + t.r * gpb + t.p / each, from = t.row * (s.K / s.group) + t.k / s.group;
    scales[at] = t.in ? __ldg(qs + from) : static_cast<uint16_t>(0);
    if (zeros) zeros[at] = t.in ? __ldg(qz + from) & 15 : 0;
  }
}

__global__ void __launch_bounds__(256) int4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                                                              const uint8_t* __restrict__ zeros, const Int4Shape s,
                                                              uint16_t* __restrict__ out) {
  griddep_wait();
  griddep_launch_dependents();
  const TilePlace t = tile_place(s);
  if (t.tile >= s.tiles() || !t.in) return;
  const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(codes + t.tile * kInt4TileBytes + word_at(t.r, t.p)));
  const long long at = t.tile * s.tile_scales() + t.r * (kInt4Block / s.group) + t.p / (s.group / 8);
  const float scale = __uint_as_float(static_cast<uint32_t>(__ldg(scales + at)) << 16);
  const int zero = zeros ? __ldg(zeros + at) : 8;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(code_of(w, i) - zero) * scale;
  *reinterpret_cast<uint4*>(out + t.row * s.K + t.k) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

dim3 tile_grid(long long tiles) {
  const long long y = (tiles + 0x3fffffffll) / 0x40000000ll;   // up to 2^30 in x
  return dim3(static_cast<unsigned>((tiles + y - 1) / y), static_cast<unsigned>(y));
}

// ---------------------------------------------------------------- products with few rows
// The rows of x are the columns of a 16 x 8 x 16 tensor-core product whose rows
// are 16 rows of w: at this size the weights' bytes bound the kernel, and what
// counts is how few instructions a code takes.  A word of 8 codes is 3 shifts, 4
// masks and 4 subtractions (128 + q - 128 - zero: exact in bf16) and half of
// two products; the sums of a group, exact products added in fp32, then take its
// scale in fp32, so that no weight is rounded.
// Since any order of k will do where both operands agree, lane (g, t)'s word j
// meets the 16 bytes of x's columns 32 j + 8 t .. + 7 as they lie in memory.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The codes of columns 2 i, 2 i + 1 of a word less the zero, as bf16: z holds 128
// + zero twice.
__device__ __forceinline__ uint32_t pair_of(uint32_t w, int i, __nv_bfloat162 z) {
  const uint32_t u = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
  const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), z);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 load_once(const uint8_t* p) {   // codes are read once: not kept in L1
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

constexpr int kInt4Warps = 8;

// A tile's codes, scales and zeros as a lane holds them: rows g and g + 8.
template <int GPB>
struct Int4Frag {
  uint4 c[2];
  uint16_t s[2][GPB];
  uint8_t z[2][GPB];
};
template <int GPB, bool ZEROS>
__device__ __forceinline__ void load_frag(Int4Frag<GPB>& f, const Int4LinearArgs& a, long long tile, int lane) {
  const uint8_t* c = a.codes + tile * kInt4TileBytes + lane * 16;
  f.c[0] = load_once(c);
  f.c[1] = load_once(c + 512);
  const int g = lane >> 2;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint16_t* s = a.scales + tile * (kInt4Rows * GPB) + (g + 8 * h) * GPB;
    if constexpr (GPB == 4) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(s));
      f.s[h][0] = v.x, f.s[h][1] = v.x >> 16, f.s[h][2] = v.y, f.s[h][3] = v.y >> 16;
    } else if constexpr (GPB == 2) {
      const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(s));
      f.s[h][0] = v, f.s[h][1] = v >> 16;
    } else {
      f.s[h][0] = __ldg(s);
    }
    if constexpr (ZEROS) {
      const uint8_t* z = a.zeros + tile * (kInt4Rows * GPB) + (g + 8 * h) * GPB;
      if constexpr (GPB == 4) {
        const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(z));
        f.z[h][0] = v, f.z[h][1] = v >> 8, f.z[h][2] = v >> 16, f.z[h][3] = v >> 24;
      } else if constexpr (GPB == 2) {
        const uint16_t v = __ldg(reinterpret_cast<const uint16_t*>(z));
        f.z[h][0] = v, f.z[h][1] = v >> 8;
      } else {
        f.z[h][0] = __ldg(z);
      }
    }
  }
}

__device__ __forceinline__ float act_of(float z, int act) {
  switch (act) {
    case LIN_RELU: return act_value<LIN_RELU>(z);
    case LIN_SILU: return act_value<LIN_SILU>(z);
    case LIN_GELU: return act_value<LIN_GELU>(z);
    case LIN_GELU_TANH: return act_value<LIN_GELU_TANH>(z);
    default: return z;
  }
}

__device__ __forceinline__ void store_out(const Int4LinearArgs& a, long long row, int n, float v) {
  const long long at = row * a.w.N + n;
  if (a.out_f32)
    static_cast<float*>(a.y)[at] = v;
  else
    static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
}

// grid {groups of R row tiles, rows of x in steps of 8 NG; with experts: rows of
// y}.  A block makes 16 R outputs of up to 8 NG rows; its warps take the blocks of
// K in turn, each with its next codes in flight, and add their sums in order.
// With experts the block of a row whose expert no earlier row has serves all
// rows of that expert, and the others' blocks end at once: an expert's weights
// are read once.
template <int NG, int R, int GPB, bool ZEROS, bool EXPERTS>
__global__ void __launch_bounds__(32 * kInt4Warps) int4_linear_kernel(const Int4LinearArgs a) {
  constexpr int kCols = 8 * NG, kRows = 16 * R;
  __shared__ float part[kInt4Warps][kCols][kRows + 1];
  __shared__ int list[kCols];
  __shared__ int found, next;
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const long long rt0 = static_cast<long long>(blockIdx.x) * R;
  const int n0 = static_cast<int>(rt0) * kInt4Rows, nb = a.w.blocks();
  long long matrix = 0;
  if constexpr (EXPERTS) {
    const int r = blockIdx.y;
    matrix = __ldg(a.experts + r);
    if (matrix < 0 || matrix >= a.w.matrices) {   // no expert: zeros; any id but -1 is an error besides
      if (matrix != -1 && threadIdx.x == 0 && blockIdx.x == 0 && a.status) atomicCAS(a.status, 0, MOK_ERR_INDEX);
      for (int n = n0 + threadIdx.x; n < min(n0 + kRows, a.w.N); n += blockDim.x) store_out(a, r, n, 0.f);
      return;
    }
    int earlier = 0;
    for (int i = threadIdx.x; i < r; i += blockDim.x) earlier |= __ldg(a.experts + i) == matrix;
    if (__syncthreads_or(earlier)) return;
    if (threadIdx.x == 0) next = r;
  }
  const long long tile0 = (matrix * a.w.row_tiles() + rt0) * nb;
  const int tiles = static_cast<int>(min(static_cast<long long>(R), a.w.row_tiles() - rt0));
  for (;;) {
    // the rows of y that this pass makes
    int cols;
    if constexpr (EXPERTS) {
      __syncthreads();
      if (warp == 0) {
        int at = next, n = 0;
        while (at < a.rows && n < kCols) {
          const bool hit = at + lane < a.rows && __ldg(a.experts + at + lane) == matrix;
          const unsigned m = __ballot_sync(0xffffffffu, hit);
          const int mine = n + __popc(m & ((1u << lane) - 1u));
          if (hit && mine < kCols) list[mine] = at + lane;
          const int all = n + __popc(m);
          if (all > kCols) {   // the next pass begins with the first that did not fit
            const unsigned over = __ballot_sync(0xffffffffu, hit && mine == kCols);
            at += __ffs(over) - 1;
            n = kCols;
            break;
          }
          n = all;
          at += 32;
        }
        if (lane == 0) found = n, next = at;
      }
      __syncthreads();
      cols = found;
      if (cols == 0) return;
    } else {
      cols = min(kCols, a.rows - static_cast<int>(blockIdx.y) * kCols);
    }
    const uint16_t* xp[NG];
#pragma unroll
    for (int c = 0; c < NG; ++c) {
      const int col = c * 8 + g;
      xp[c] = nullptr;
      if (col < cols) {
        const int r = EXPERTS ? list[col] : static_cast<int>(blockIdx.y) * kCols + col;
        xp[c] = a.x + static_cast<long long>(r / a.x_div) * a.w.K + t * 8;
      }
    }
    float acc[R][NG][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < NG; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][c][i] = 0.f;
    Int4Frag<GPB> now[R], ahead[R];
    int kb = warp;
    if (kb < nb) {
#pragma unroll
      for (int r = 0; r < R; ++r) load_frag<GPB, ZEROS>(now[r], a, tile0 + static_cast<long long>(min(r, tiles - 1)) * nb + kb, lane);
    }
    for (; kb < nb; kb += kInt4Warps) {
      if (kb + kInt4Warps < nb) {
#pragma unroll
        for (int r = 0; r < R; ++r)
          load_frag<GPB, ZEROS>(ahead[r], a, tile0 + static_cast<long long>(min(r, tiles - 1)) * nb + kb + kInt4Warps, lane);
      }
      constexpr int kWords = 4 / GPB;   // words of a group
#pragma unroll
      for (int gr = 0; gr < GPB; ++gr) {
        float sum[R][NG][4];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int c = 0; c < NG; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[r][c][i] = 0.f;
        __nv_bfloat162 zero[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t z = 0x43004300u | (ZEROS ? now[r].z[h][gr] * 0x00010001u : 0x00080008u);
            zero[r][h] = *reinterpret_cast<const __nv_bfloat162*>(&z);
          }
#pragma unroll
        for (int jj = 0; jj < kWords; ++jj) {
          const int j = gr * kWords + jj, k = kb * kInt4Block + 32 * j;
          uint4 b[NG];
#pragma unroll
          for (int c = 0; c < NG; ++c) {
            b[c] = make_uint4(0u, 0u, 0u, 0u);
            if (xp[c] && k < a.w.K) b[c] = __ldg(reinterpret_cast<const uint4*>(xp[c] + k));   // K % 32 == 0
          }
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const uint32_t lo = j == 0 ? now[r].c[0].x : j == 1 ? now[r].c[0].y : j == 2 ? now[r].c[0].z : now[r].c[0].w;
            const uint32_t hi = j == 0 ? now[r].c[1].x : j == 1 ? now[r].c[1].y : j == 2 ? now[r].c[1].z : now[r].c[1].w;
            uint32_t wl[4], wh[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) wl[i] = pair_of(lo, i, zero[r][0]), wh[i] = pair_of(hi, i, zero[r][1]);
#pragma unroll
            for (int c = 0; c < NG; ++c) {
              mma_16816(sum[r][c], wl[0], wh[0], wl[1], wh[1], b[c].x, b[c].y);
              mma_16816(sum[r][c], wl[2], wh[2], wl[3], wh[3], b[c].z, b[c].w);
            }
          }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float sl = __uint_as_float(static_cast<uint32_t>(now[r].s[0][gr]) << 16);
          const float sh = __uint_as_float(static_cast<uint32_t>(now[r].s[1][gr]) << 16);
#pragma unroll
          for (int c = 0; c < NG; ++c) {
            acc[r][c][0] = fmaf(sl, sum[r][c][0], acc[r][c][0]);
            acc[r][c][1] = fmaf(sl, sum[r][c][1], acc[r][c][1]);
            acc[r][c][2] = fmaf(sh, sum[r][c][2], acc[r][c][2]);
            acc[r][c][3] = fmaf(sh, sum[r][c][3], acc[r][c][3]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) now[r] = ahead[r];
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < NG; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[warp][c * 8 + 2 * t + (i & 1)][r * 16 + g + 8 * (i >> 1)] = acc[r][c][i];
    __syncthreads();
    for (int i = threadIdx.x; i < cols * kRows; i += blockDim.x) {
      const int c = i / kRows, m = i % kRows, n = n0 + m;
      if (n >= a.w.N) continue;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kInt4Warps; ++w) v += part[w][c][m];
      if (a.bias) {
        const long long at = matrix * a.w.N + n;
        v += a.bias_f32 ? __ldg(static_cast<const float*>(a.bias) + at)
                        : __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(a.bias) + at)) << 16);
      }
      store_out(a, EXPERTS ? list[c] : blockIdx.y * kCols + c, n, act_of(v, a.act));
    }
    if constexpr (!EXPERTS) return;
  }
}

template <int NG, int R, int GPB, bool ZEROS>
cudaError_t int4_launch(const Int4LinearArgs& a, cudaStream_t st) {
  const unsigned x = static_cast<unsigned>((a.w.row_tiles() + R - 1) / R);
  if (a.experts)
    return launch_dependent(int4_linear_kernel<NG, R, GPB, ZEROS, true>, dim3(x, a.rows), dim3(32 * kInt4Warps), 0, st, a);
  return launch_dependent(int4_linear_kernel<NG, R, GPB, ZEROS, false>, dim3(x, (a.rows + 8 * NG - 1) / (8 * NG)),
                          dim3(32 * kInt4Warps), 0, st, a);
}

template <int NG, int R>
cudaError_t int4_group(const Int4LinearArgs& a, cudaStream_t st) {
  const bool z = a.zeros != nullptr;
  if (a.w.group == 32) return z ? int4_launch<NG, R, 4, true>(a, st) : int4_launch<NG, R, 4, false>(a, st);
  if (a.w.group == 64) return z ? int4_launch<NG, R, 2, true>(a, st) : int4_launch<NG, R, 2, false>(a, st);
  return z ? int4_launch<NG, R, 1, true>(a, st) : int4_launch<NG, R, 1, false>(a, st);
}

}  // namespace

cudaError_t launch_int4_quantize(const void* w, int f32, const Int4Shape& s, uint8_t* codes, uint16_t* scales, uint8_t* zeros,
                                 cudaStream_t st) {
  const dim3 g = tile_grid(s.tiles());
  if (f32)
    return zeros ? launch_dependent(int4_quantize_kernel<true, true>, g, dim3(256), 0, st, w, s, codes, scales, zeros)
                 : launch_dependent(int4_quantize_kernel<true, false>, g, dim3(256), 0, st, w, s, codes, scales, zeros);
  return zeros ? launch_dependent(int4_quantize_kernel<false, true>, g, dim3(256), 0, st, w, s, codes, scales, zeros)
               : launch_dependent(int4_quantize_kernel<false, false>, g, dim3(256), 0, st, w, s, codes, scales, zeros);
}

cudaError_t launch_int4_pack(const uint8_t* q, const uint16_t* qs, const uint8_t* qz, const Int4Shape& s, uint8_t* codes,
                             uint16_t* scales, uint8_t* zeros, cudaStream_t st) {
  return launch_dependent(int4_pack_kernel, tile_grid(s.tiles()), dim3(256), 0, st, q, qs, qz, s, codes, scales, zeros);
}

cudaError_t launch_int4_dequantize(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, const Int4Shape& s,
                                   uint16_t* out, cudaStream_t st) {
  return launch_dependent(int4_dequantize_kernel, tile_grid(s.tiles()), dim3(256), 0, st, codes, scales, zeros, s, out);
}

cudaError_t launch_int4_linear(const Int4LinearArgs& a, int num_sms, cudaStream_t st) {
  // columns of the product: what there are, or with experts the rows that one has on average
  const double per = a.experts ? static_cast<double>(a.rows) / static_cast<double>(a.w.matrices) : static_cast<double>(a.rows);
  // two row tiles to a warp halve its loads of x; one, where there would be few blocks
  const long long blocks = (a.w.row_tiles() + 1) / 2 * (a.experts ? a.rows : 1);
  if (per > 16) return int4_group<4, 2>(a, st);
  if (per > 8) return int4_group<2, 2>(a, st);
  return blocks >= 4ll * num_sms ? int4_group<1, 2>(a, st) : int4_group<1, 1>(a, st);
}

}  // namespace mok
