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

#include <atomic>

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
// scale), q = round(w / scale) + zero; both clamped to 0..15.  A group with a
// value that is not finite gets a NaN scale.  64 matrices of 2048 x 2048 in bf16
// take 427 to 488 us, 680 MB or so that a copy moves in 100: a tile to a block, with
// its place to find, and eight divisions to a thread.
template <bool F32, bool ZEROS>
__global__ void __launch_bounds__(256) int4_quantize_kernel(const void* __restrict__ w, const Int4Shape s, uint8_t* __restrict__ codes,
                                                            uint16_t* __restrict__ scales, uint8_t* __restrict__ zeros) {
  griddep_wait();
  griddep_launch_dependents();
  const TilePlace t = tile_place(s);
  if (t.tile >= s.tiles()) return;   // whole blocks
  float v[8] = {};
  if (t.in) load_vals<8>(w, F32, t.row * s.K + t.k, v);
  float lo = 0.f, hi = 0.f, none = 0.f;   // none: 0, or NaN where a value is not finite, which the range would not show
#pragma unroll
  for (int i = 0; i < 8; ++i) lo = fminf(lo, v[i]), hi = fmaxf(hi, v[i]), none = fmaf(v[i], 0.f, none);
  for (int o = 1; o < s.group / 8; o <<= 1) {   // the group's threads: 4, 8 or 16 neighbours
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    none += __shfl_xor_sync(0xffffffffu, none, o);
  }
  const float range = hi - lo;   // (may pass the largest number, which a fifteenth of it does not)
  const float step = !ZEROS ? fmaxf(-lo, hi) / 7.f : isinf(range) ? hi / 15.f - lo / 15.f : range / 15.f;
  const float scale = bf16_round(step) + none;
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

// From row-major codes, two to a byte, the even column's in the low half: as many
// matrices 275 to 292 us, 285 MB or so that a copy moves in 42.
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

// Up to kReadTiles neighbours along K to a block, a tile's loads not waiting for
// another's: 64 matrices of 2048 x 2048 151 us (groups of 128) to 181 (of 32, with
// zeros), 680 MB or so that a copy moves in 100; a tile to a block, with its place
// to find, took about 260.
constexpr int kReadTiles = 8;
__global__ void __launch_bounds__(256) int4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint16_t* __restrict__ scales,
                                                              const uint8_t* __restrict__ zeros, const Int4Shape s,
                                                              uint16_t* __restrict__ out) {
  griddep_wait();
  griddep_launch_dependents();
  const int nb = s.blocks(), parts = (nb + kReadTiles - 1) / kReadTiles, r = threadIdx.x >> 4, p = threadIdx.x & 15;
  const long long part = static_cast<long long>(blockIdx.x) + static_cast<long long>(blockIdx.y) * gridDim.x;
  const long long rt = part / parts, m = rt / s.row_tiles();
  const long long n = (rt - m * s.row_tiles()) * kInt4Rows + r;
  if (m >= s.matrices || n >= s.N) return;
  const int kb0 = static_cast<int>(part - rt * parts) * kReadTiles, tiles = min(kReadTiles, nb - kb0);
  const long long tile0 = rt * nb + kb0;
  const uint8_t* const code = codes + tile0 * kInt4TileBytes + word_at(r, p);
  const int each = s.tile_scales();
  const long long first = tile0 * each + r * (kInt4Block / s.group) + p * 8 / s.group;
  uint16_t* const to = out + (m * s.N + n) * s.K;
  constexpr int kAtOnce = 4;
#pragma unroll 1
  for (int i0 = 0; i0 < tiles; i0 += kAtOnce) {
    uint32_t w[kAtOnce], scale[kAtOnce], zero[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = min(i0 + u, tiles - 1);   // (behind the last tile: that one again, not stored)
      w[u] = __ldg(reinterpret_cast<const uint32_t*>(code + i * kInt4TileBytes));
      scale[u] = __ldg(scales + first + static_cast<long long>(i) * each);
      zero[u] = zeros ? __ldg(zeros + first + static_cast<long long>(i) * each) : 8u;
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int k = (kb0 + i0 + u) * kInt4Block + 8 * p;
      if (i0 + u >= tiles || k >= s.K) break;
      const float by = __uint_as_float(scale[u] << 16), less = static_cast<float>(128u + zero[u]);
      uint32_t v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {   // 128 + q, from its bits
        const float even = __uint_as_float(((w[u] << (16 - 4 * j)) & 0x000F0000u) | 0x43000000u);
        const float odd = __uint_as_float(((w[u] >> (4 * j)) & 0x000F0000u) | 0x43000000u);
        v[j] = pack_bf16((even - less) * by, (odd - less) * by);
      }
      *reinterpret_cast<uint4*>(to + k) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
}

dim3 tile_grid(long long tiles) {
  const long long y = (tiles + 0x3fffffffll) / 0x40000000ll;   // up to 2^30 in x
  return dim3(static_cast<unsigned>((tiles + y - 1) / y), static_cast<unsigned>(y));
}

// ---------------------------------------------------------------- products with few rows
// The rows of x are the columns of 16 x 8 x 16 tensor-core products whose rows
// are 16 rows of w: at this size the weights' bytes bound the kernels, and what
// counts is how few instructions a code takes.  A word of 8 codes is 3 shifts, 4
// masks and 4 additions (128 + q less 128 + zero: exact in bf16) and half of
// two products; the sums of a group, exact products added in fp32, then take its
// scale in fp32, so that no weight is rounded.
// Since any order of k will do where both operands agree, lane (g, t)'s word j
// meets the 16 bytes of x's columns 32 j + 8 t .. + 7 as they lie in memory.
// Codes, scales and x come in through shared memory by asynchronous copies some
// stages ahead: registers would hold too few bytes in flight (8 experts of 2048 x
// 7168 took 30 us so, and 19 with stages in graph replays, 20.4 in calls on other
// experts: 245 instructions a tile, issue slots 52% busy, DRAM 40%).  One row times
// 7168 x 2048: 3.6 us.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same without sums to add to.
__device__ __forceinline__ void mma_16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                                uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// The codes of columns 2 i, 2 i + 1 of a word less the zero, as bf16: z holds
// -(128 + zero) twice.
__device__ __forceinline__ uint32_t pair_of(uint32_t w, int i, uint32_t z) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(w >> (4 * i)), "r"(0x000F000Fu), "r"(0x43004300u));   // (a & b) | c
  asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(z));
  return v;
}

constexpr int kInt4Warps = 8;   // of a block, at most

// CH tiles of a row tile, neighbours along K, in shared memory: their codes, then
// their scales, then their zeros.
template <int GPB, bool ZEROS, int CH>
struct Int4Chunk {
  static constexpr int kScales = CH * kInt4TileBytes, kZeros = kScales + CH * 32 * GPB;
  static constexpr int kBytes = kZeros + (ZEROS ? CH * 16 * GPB : 0);
  static_assert(CH * 2 * GPB <= 16 && CH * GPB <= 16, "a warp copies scales and zeros at one go");
};
// What a lane copies of a row tile, chunk by chunk: two pieces of each tile's
// codes, and of the scales or zeros one or none.
template <int GPB, bool ZEROS, int CH>
struct Int4Source {
  using L = Int4Chunk<GPB, ZEROS, CH>;
  const uint8_t* codes;
  const uint8_t* extra;
  int extra_step, extra_at;   // extra_at: -1 for none
  __device__ __forceinline__ void start(const Int4LinearArgs& a, long long tile, int lane) {
    codes = a.codes + tile * kInt4TileBytes + lane * 16;
    extra = nullptr, extra_step = 0, extra_at = -1;
    if (lane < CH * 2 * GPB) {
      extra = reinterpret_cast<const uint8_t*>(a.scales) + tile * (32 * GPB) + lane * 16;
      extra_step = CH * 32 * GPB, extra_at = L::kScales + lane * 16;
    } else if (ZEROS && lane >= 16 && lane < 16 + CH * GPB) {
      extra = a.zeros + tile * (16 * GPB) + (lane - 16) * 16;
      extra_step = CH * 16 * GPB, extra_at = L::kZeros + (lane - 16) * 16;
    }
  }
  // n (1 .. CH) tiles into dst; then on by `step` chunks.
  __device__ __forceinline__ void fetch(uint8_t* dst, int n, int step, int lane) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (i < n) {
        cp_async16(dst + i * kInt4TileBytes + lane * 16, codes + i * kInt4TileBytes, 16);
        cp_async16(dst + i * kInt4TileBytes + 512 + lane * 16, codes + i * kInt4TileBytes + 512, 16);
      }
    }
    codes += step * (CH * kInt4TileBytes);
    // (a piece lies in one tile: 16 bytes are a divisor of a tile's scales, and of its zeros)
    if (extra_at >= 0 && (n == CH || (extra_at < L::kZeros ? lane < n * 2 * GPB : lane - 16 < n * GPB))) cp_async16(dst + extra_at, extra, 16);
    extra += step * extra_step;
  }
};
// A column of a chunk of x: 256 bytes for each block of K, and 64 more, so that
// the eight lanes of a shared-memory access (two columns) meet all banks.
template <int CH>
constexpr int kXColumn = CH * 256 + 64;

// A lane's rows g and g + 8 of tile i of a chunk; scales two to a word, zeros four.
template <int GPB, bool ZEROS, int CH>
struct Int4Frag {
  using L = Int4Chunk<GPB, ZEROS, CH>;
  uint4 c[2];
  uint32_t s[2][(GPB + 1) / 2], z[2];
  __device__ __forceinline__ void load(const uint8_t* chunk, int i, int lane) {
    c[0] = *reinterpret_cast<const uint4*>(chunk + i * kInt4TileBytes + lane * 16);
    c[1] = *reinterpret_cast<const uint4*>(chunk + i * kInt4TileBytes + 512 + lane * 16);
    const int g = lane >> 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t* at = chunk + L::kScales + g * (GPB * 2) + i * (32 * GPB) + h * (16 * GPB);
      if constexpr (GPB == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(at);
        s[h][0] = v.x, s[h][1] = v.y;
      } else if constexpr (GPB == 2) {
        s[h][0] = *reinterpret_cast<const uint32_t*>(at);
      } else {
        s[h][0] = *reinterpret_cast<const uint16_t*>(at);
      }
      if constexpr (ZEROS) {
        const uint8_t* zt = chunk + L::kZeros + g * GPB + i * (16 * GPB) + h * (8 * GPB);
        if constexpr (GPB == 4)
          z[h] = *reinterpret_cast<const uint32_t*>(zt);
        else if constexpr (GPB == 2)
          z[h] = *reinterpret_cast<const uint16_t*>(zt);
        else
          z[h] = *zt;
      }
    }
  }
  __device__ __forceinline__ float scale(int h, int gr) const {
    const uint32_t v = s[h][gr >> 1];
    return __uint_as_float(gr & 1 ? v & 0xFFFF0000u : v << 16);
  }
  // -(128 + zero) in bf16, twice: the bytes zero, 0xC3, zero, 0xC3.
  __device__ __forceinline__ uint32_t zero(int h, int gr) const { return ZEROS ? __byte_perm(z[h], 0xC3u, 0x4040u + 0x0101u * gr) : 0xC308C308u; }
};

// acc += tile i of R chunks (step bytes apart) times that block of x's COLS
// columns (2, or 8 NG): acc[.][c] holds rows g (0, 1) and g + 8 (2, 3) of the
// columns 8 c + 2 t + {0, 1}.  COLS = 2: the others repeat them.
template <int COLS, int NG, int R, int GPB, bool ZEROS, int CH>
__device__ __forceinline__ void block_products(float (&acc)[R][NG][4], const uint8_t* chunk, int step, const uint8_t* x, int i, int lane) {
  const int g = lane >> 2, t = lane & 3;
  constexpr int kWords = 4 / GPB;   // words of a group
  Int4Frag<GPB, ZEROS, CH> f[R];
#pragma unroll
  for (int r = 0; r < R; ++r) f[r].load(chunk + r * step, i, lane);
  x += (g & (COLS - 1)) * kXColumn<CH> + t * 16 + i * 256;
#pragma unroll
  for (int gr = 0; gr < GPB; ++gr) {
    float sum[R][NG][4];
#pragma unroll
    for (int jj = 0; jj < kWords; ++jj) {
      const int j = gr * kWords + jj;
      uint4 b[NG];
#pragma unroll
      for (int c = 0; c < NG; ++c) b[c] = *reinterpret_cast<const uint4*>(x + c * 8 * kXColumn<CH> + j * 64);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t lo = j == 0 ? f[r].c[0].x : j == 1 ? f[r].c[0].y : j == 2 ? f[r].c[0].z : f[r].c[0].w;
        const uint32_t hi = j == 0 ? f[r].c[1].x : j == 1 ? f[r].c[1].y : j == 2 ? f[r].c[1].z : f[r].c[1].w;
        uint32_t wl[4], wh[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) wl[i] = pair_of(lo, i, f[r].zero(0, gr)), wh[i] = pair_of(hi, i, f[r].zero(1, gr));
#pragma unroll
        for (int c = 0; c < NG; ++c) {
          if (jj == 0)
            mma_16816_first(sum[r][c], wl[0], wh[0], wl[1], wh[1], b[c].x, b[c].y);
          else
            mma_16816(sum[r][c], wl[0], wh[0], wl[1], wh[1], b[c].x, b[c].y);
        }
#pragma unroll
        for (int c = 0; c < NG; ++c) mma_16816(sum[r][c], wl[2], wh[2], wl[3], wh[3], b[c].z, b[c].w);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float sl = f[r].scale(0, gr), sh = f[r].scale(1, gr);
#pragma unroll
      for (int c = 0; c < NG; ++c) {
        acc[r][c][0] = fmaf(sl, sum[r][c][0], acc[r][c][0]);
        acc[r][c][1] = fmaf(sl, sum[r][c][1], acc[r][c][1]);
        acc[r][c][2] = fmaf(sh, sum[r][c][2], acc[r][c][2]);
        acc[r][c][3] = fmaf(sh, sum[r][c][3], acc[r][c][3]);
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

__device__ __forceinline__ float int4_bias(const Int4LinearArgs& a, long long at) {
  if (!a.bias) return 0.f;
  return a.bias_f32 ? __ldg(static_cast<const float*>(a.bias) + at)
                    : __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(a.bias) + at)) << 16);
}
__device__ __forceinline__ void store_out(const Int4LinearArgs& a, long long row, int n, float v) {
  const long long at = row * a.w.N + n;
  if (a.out_f32)
    static_cast<float*>(a.y)[at] = v;
  else
    static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
}

// ---- warps that share K: few rows of w to a block
// grid {groups of R row tiles, rows of x in steps of COLS; with experts: rows of
// y, or the experts where they are fewer}, 1 to 8 warps.  A block makes 16 R outputs of up to COLS rows; each warp
// takes a part of K through stages of its own, and their sums are added in order.
// With experts, the block of an expert, or of a row whose expert no earlier row
// has, serves all rows of that expert, and the others end at once: an expert's
// weights are read once for COLS of its rows.
template <int COLS, int R, int GPB, bool ZEROS>
struct Int4SplitCfg {
  static constexpr int kCols = COLS, kRows = 16 * R, kGroups = COLS < 8 ? 1 : COLS / 8;
  static constexpr int kChunk = COLS == 2 ? 2 : 1;   // blocks of K to a stage
  static constexpr int kStages = COLS == 2 || COLS == 32 ? 2 : 3;
  static constexpr int kTiles = Int4Chunk<GPB, ZEROS, kChunk>::kBytes;
  static constexpr int kStageBytes = R * kTiles + kCols * kXColumn<kChunk>;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static_assert(kCols * (kRows + 1) * 4 <= kWarpBytes, "the parts fit the stages");
  static_assert(kInt4Warps * kWarpBytes + 4096 <= 227 * 1024, "shared memory");
};

template <int COLS, int R, int GPB, bool ZEROS, bool EXPERTS>
__global__ void __launch_bounds__(32 * kInt4Warps, COLS <= 8 ? 4 : 1) int4_split_kernel(const Int4LinearArgs a) {
  using C = Int4SplitCfg<COLS, R, GPB, ZEROS>;
  constexpr int kCols = C::kCols, kRows = C::kRows, NG = C::kGroups, D = C::kStages, CH = C::kChunk;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int lists[kInt4Warps][kCols];   // each warp its own: rows of y
  __shared__ const uint16_t* x_rows[kInt4Warps][kCols];   // and of x
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  griddep_wait();
  griddep_launch_dependents();
  const long long rt0 = static_cast<long long>(blockIdx.x) * R;
  const int n0 = static_cast<int>(rt0) * kInt4Rows, nb = a.w.blocks();
  long long matrix = 0;
  unsigned same = 0;   // up to 32 rows: those of this block's expert
  const bool few = EXPERTS && a.rows <= 32;
  if constexpr (EXPERTS) {
    const int r = blockIdx.y;
    const long long id = few ? (lane < a.rows ? __ldg(a.experts + lane) : -2) : a.by_expert ? 0 : __ldg(a.experts + r);
    matrix = a.by_expert ? r : few ? __shfl_sync(0xffffffffu, id, r) : id;
    if (a.by_expert) {
      if (r == 0) {   // rows of no expert: zeros; any id but -1 is an error besides
        for (int f = warp * 32; f < a.rows; f += blockDim.x) {   // 32 of them at a time
          const long long e = f + lane < a.rows ? __ldg(a.experts + f + lane) : 0;
          const bool none = e < 0 || e >= a.w.matrices;
          if (none && e != -1 && blockIdx.x == 0 && a.status) atomicCAS(a.status, 0, MOK_ERR_INDEX);
          for (unsigned m = __ballot_sync(0xffffffffu, none); m; m &= m - 1)
            for (int n = n0 + lane; n < min(n0 + kRows, a.w.N); n += 32) store_out(a, f + __ffs(m) - 1, n, 0.f);
        }
      }
    } else if (matrix < 0 || matrix >= a.w.matrices) {
      if (matrix != -1 && threadIdx.x == 0 && blockIdx.x == 0 && a.status) atomicCAS(a.status, 0, MOK_ERR_INDEX);
      for (int n = n0 + threadIdx.x; n < min(n0 + kRows, a.w.N); n += blockDim.x) store_out(a, r, n, 0.f);
      return;
    }
    if (few) {   // each warp for itself
      same = __ballot_sync(0xffffffffu, id == matrix);
      if (!a.by_expert && (same & ((1u << r) - 1u))) return;
    } else if (!a.by_expert) {
      int earlier = 0;
      for (int i = threadIdx.x; i < r; i += blockDim.x) earlier |= __ldg(a.experts + i) == matrix;
      if (__syncthreads_or(earlier)) return;
    }
  }
  const int warps = blockDim.x >> 5;
  uint8_t* const stages = smem + warp * C::kWarpBytes;
  int* const list = lists[warp];
  const long long tile0 = (matrix * a.w.row_tiles() + rt0) * nb;
  const int tiles = static_cast<int>(min(static_cast<long long>(R), a.w.row_tiles() - rt0));
  // this warp's blocks of K
  const int each = nb / warps, more = nb - each * warps;
  const int kb0 = each * warp + min(warp, more), kb1 = kb0 + each + (warp < more ? 1 : 0);
  int next = EXPERTS && !a.by_expert ? blockIdx.y : 0;
  for (;;) {
    // the rows of y that this pass makes
    int cols;
    if constexpr (EXPERTS) {
      cols = 0;
      while (next < a.rows && cols < kCols) {
        const bool hit = next + lane < a.rows && (few ? (same >> (next + lane)) & 1u : __ldg(a.experts + next + lane) == matrix);
        const unsigned m = __ballot_sync(0xffffffffu, hit);
        const int at = cols + __popc(m & ((1u << lane) - 1u)), all = cols + __popc(m);
        if (hit && at < kCols) list[at] = next + lane;
        if (all > kCols) {   // the next pass begins with the first that did not fit
          next += __ffs(__ballot_sync(0xffffffffu, hit && at == kCols)) - 1;
          cols = kCols;
          break;
        }
        cols = all;
        next += 32;
      }
      if (cols == 0) return;
    } else {
      cols = min(kCols, a.rows - static_cast<int>(blockIdx.y) * kCols);
      for (int i = lane; i < cols; i += 32) list[i] = blockIdx.y * kCols + i;
    }
    __syncwarp();
    for (int i = lane; i < cols; i += 32) x_rows[warp][i] = a.x + static_cast<long long>(list[i] / a.x_div) * a.w.K;
    __syncwarp();
    Int4Source<GPB, ZEROS, CH> src[R];
#pragma unroll
    for (int r = 0; r < R; ++r) src[r].start(a, tile0 + (r < tiles ? r : 0) * static_cast<long long>(nb) + kb0, lane);   // (behind the last row tile: the first again)
    // a lane's piece of the columns of x: all of one column (CH = 2), or half of two
    constexpr int kLanes = CH * 16;
    const int p = lane % kLanes, odd = lane / kLanes;
    const uint16_t* const xp = odd < cols ? x_rows[warp][odd] + p * 8 : nullptr;
    int ahead = kb0, to = 0;   // the next block that is fetched, and its stage
    const auto fetch = [&]() {
      if (ahead < kb1) {
        uint8_t* st = stages + to * C::kStageBytes;
        const int n = min(CH, kb1 - ahead), k = ahead * kInt4Block;
#pragma unroll
        for (int r = 0; r < R; ++r) src[r].fetch(st + r * C::kTiles, n, 1, lane);
        const uint32_t in = k + p * 8 < a.w.K ? 16u : 0u;   // zeros behind the last column
        const int from = in ? k : -p * 8;
        if (p < 16 * n) {
#pragma unroll
          for (int c = 0; c < kCols; c += 32 / kLanes) {   // columns without a row hold anything: theirs are not stored
            if (c >= cols) break;
            if (c + odd < cols)
              cp_async16(st + R * C::kTiles + (c + odd) * kXColumn<CH> + p * 16, (c == 0 ? xp : x_rows[warp][c + odd] + p * 8) + from, in);
          }
        }
        ahead += CH;
        if (++to == D) to = 0;
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < D - 1; ++i) fetch();
    float acc[R][NG][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < NG; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][c][i] = 0.f;
    int at = 0;
#pragma unroll 1
    for (int kb = kb0; kb < kb1; kb += CH) {
      cp_async_wait<D - 2>();
      __syncwarp();   // every lane's copies are there, and the stage that is filled next has been read
      fetch();
      const uint8_t* st = stages + at * C::kStageBytes;
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (kb + i < kb1) block_products<kCols, NG, R, GPB, ZEROS, CH>(acc, st, C::kTiles, st + R * C::kTiles, i, lane);
      if (++at == D) at = 0;
    }
    cp_async_wait<0>();
    __syncthreads();   // the parts lie over the stages
    float* part = reinterpret_cast<float*>(smem);   // [warp][kCols][kRows + 1]
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < NG; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (kCols >= 8 || t == 0) part[(warp * kCols + c * 8 + 2 * t + (i & 1)) * (kRows + 1) + r * 16 + g + 8 * (i >> 1)] = acc[r][c][i];
    __syncthreads();
    for (int i = threadIdx.x; i < cols * kRows; i += blockDim.x) {
      const int c = i / kRows, m = i % kRows, n = n0 + m;
      if (n >= a.w.N) continue;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kInt4Warps; ++w)
        if (w < warps) v += part[(w * kCols + c) * (kRows + 1) + m];
      v += int4_bias(a, matrix * a.w.N + n);
      store_out(a, list[c], n, act_of(v, a.act));
    }
    if constexpr (!EXPERTS) return;
    __syncthreads();   // the parts have been read
  }
}

// ---- warps that share x: many rows of w
// grid {groups of 16 row tiles}, one matrix, up to 8 rows of x (more of them are for
// int4_tc.cu).  A warp makes 32 rows of w over all of K; the block's warps go
// through K together, so that a block of x is fetched once for 256 rows of w.
template <int GPB, bool ZEROS>
struct Int4WideCfg {
  static constexpr int kCols = 8, kRowTiles = 2 * kInt4Warps;
  static constexpr int kStages = 3;
  static constexpr int kTile = Int4Chunk<GPB, ZEROS, 1>::kBytes;
  static constexpr int kStageBytes = kRowTiles * kTile + kCols * kXColumn<1>;
  static constexpr int kSmemBytes = kStages * kStageBytes;
  static_assert(kInt4Warps * kCols * 33 * 4 <= kSmemBytes, "the outputs fit the stages");
  static_assert(kSmemBytes <= 112 * 1024, "two blocks to an SM");
};

template <int GPB, bool ZEROS>
__global__ void __launch_bounds__(32 * kInt4Warps, 2) int4_wide_kernel(const Int4LinearArgs a) {
  using C = Int4WideCfg<GPB, ZEROS>;
  constexpr int kCols = C::kCols, D = C::kStages;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  griddep_wait();
  griddep_launch_dependents();
  const int nb = a.w.blocks(), row_tiles = static_cast<int>(a.w.row_tiles());
  const int rt = static_cast<int>(blockIdx.x) * C::kRowTiles + 2 * warp;   // this warp's first row tile
  const int cols = a.rows;
  Int4Source<GPB, ZEROS, 1> src[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) src[r].start(a, static_cast<long long>(min(rt + r, row_tiles - 1)) * nb, lane);
  // this thread's piece of x: column tid / 16, where there is one
  const int p = threadIdx.x & 15, col = threadIdx.x >> 4;
  const uint16_t* const xp = col < cols ? a.x + static_cast<long long>(col) * a.w.K : nullptr;
  int ahead = 0;
  const auto fetch = [&]() {
    if (ahead < nb) {
      uint8_t* st = smem + ahead % D * C::kStageBytes;
#pragma unroll
      for (int r = 0; r < 2; ++r) src[r].fetch(st + (2 * warp + r) * C::kTile, 1, 1, lane);
      const int k = ahead * kInt4Block + p * 8, from = k < a.w.K ? k : 0;
      if (xp) cp_async16(st + C::kRowTiles * C::kTile + col * kXColumn<1> + p * 16, xp + from, k < a.w.K ? 16u : 0u);
      ++ahead;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < D - 1; ++i) fetch();
  float acc[2][1][4] = {};
#pragma unroll 1
  for (int kb = 0; kb < nb; ++kb) {
    cp_async_wait<D - 2>();
    __syncthreads();   // every thread's copies are there, and the stage that is filled next has been read
    fetch();
    const uint8_t* st = smem + kb % D * C::kStageBytes;
    block_products<kCols, 1, 2, GPB, ZEROS, 1>(acc, st + 2 * warp * C::kTile, C::kTile, st + C::kRowTiles * C::kTile, 0, lane);
  }
  cp_async_wait<0>();
  __syncthreads();
  float* out = reinterpret_cast<float*>(smem) + warp * kCols * 33;   // [kCols][33] of this warp's 32 rows of w
#pragma unroll
  for (int r = 0; r < 2; ++r)
    for (int i = 0; i < 4; ++i) out[(2 * t + (i & 1)) * 33 + r * 16 + g + 8 * (i >> 1)] = acc[r][0][i];
  __syncwarp();
  const int n = rt * kInt4Rows + lane;
  if (n >= a.w.N) return;
  const float bias = int4_bias(a, n);
#pragma unroll 4
  for (int c = 0; c < cols; ++c) store_out(a, c, n, act_of(out[c * 33 + lane] + bias, a.act));
}

// The kernels' shared memory is above the default limit, which is raised once per
// kernel and device.
struct SmemLimit {
  std::atomic<bool> done[64] = {};   // any thread may be the first
  template <class K>
  cudaError_t raise(K kern, int bytes) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess) done[dev].store(true, std::memory_order_release);
    return err;
  }
};

template <int COLS, int R, int GPB, bool ZEROS, bool EXPERTS>
cudaError_t split_launch(const Int4LinearArgs& a, int num_sms, cudaStream_t st) {
  using C = Int4SplitCfg<COLS, R, GPB, ZEROS>;
  auto kern = int4_split_kernel<COLS, R, GPB, ZEROS, EXPERTS>;
  static SmemLimit limit;
  const cudaError_t err = limit.raise(kern, kInt4Warps * C::kWarpBytes);
  if (err != cudaSuccess) return err;
  const unsigned x = static_cast<unsigned>((a.w.row_tiles() + R - 1) / R);
  const unsigned y = !EXPERTS ? (a.rows + C::kCols - 1) / C::kCols : a.by_expert ? static_cast<unsigned>(a.w.matrices) : a.rows;
  // 4 warps to a block, 8 where an SM would have fewer than ten warps and each has a block of K.  Measured (graph replays, here and below) with 2, 4 and 8: one row
  // times 7168 x 2048 4.2, 3.5 and 4.1 us, 8 experts of 2048 x 7168 20.4, 17.7 and 19.5, 12 rows times 2048 x 2048 8.4, 5.2 and
  // 4.3, 30 rows times 7504 x 512 7.4, 5.6 and 7.8.  Two or one where K is short and there are many blocks, of
  // which an SM then holds more.  Measured with 1, 2 and 4: 42 rows among 55 experts of 9712 x 384 29, 37 and 53 us, 120 rows among
  // 64 of 2048 x 512 18.5, 21.5 and 31, 256 rows among 64 of 4096 x 2048 104, 115 and 138, 64 rows among 8 of 8192 x 2048 38, 38
  // and 43; but one row times 49152 x 2048 20.3, 15.6 and 15.2, and 8 experts of 4096 x 4096 24.6, 22.6 and 20.5.
  const long long all = static_cast<long long>(x) * y;
  const int blocks = a.w.blocks();
  int warps = all * 4 < 10ll * num_sms && blocks >= 8 ? 8 : 4;
  if (blocks <= 16 && all >= 12ll * num_sms) warps = all >= 32ll * num_sms && (COLS > 2 || blocks <= 8) ? 1 : 2;
  return launch_dependent(kern, dim3(x, y), dim3(32 * warps), warps * C::kWarpBytes, st, a);
}
template <int GPB, bool ZEROS>
cudaError_t wide_launch(const Int4LinearArgs& a, cudaStream_t st) {
  using C = Int4WideCfg<GPB, ZEROS>;
  auto kern = int4_wide_kernel<GPB, ZEROS>;
  static SmemLimit limit;
  const cudaError_t err = limit.raise(kern, C::kSmemBytes);
  if (err != cudaSuccess) return err;
  const unsigned x = static_cast<unsigned>((a.w.row_tiles() + C::kRowTiles - 1) / C::kRowTiles);
  return launch_dependent(kern, dim3(x), dim3(32 * kInt4Warps), C::kSmemBytes, st, a);
}

// COLS columns of x at a time; wide: shared x.
template <int COLS, int GPB, bool ZEROS>
cudaError_t int4_kind(const Int4LinearArgs& a, bool wide, int num_sms, cudaStream_t st) {
  if constexpr (COLS <= 8)
    if (wide) return wide_launch<GPB, ZEROS>(a, st);
  constexpr int R = COLS > 8 ? 2 : 1;   // two row tiles to a block halve the bytes of x
  return a.experts ? split_launch<COLS, R, GPB, ZEROS, true>(a, num_sms, st) : split_launch<COLS, R, GPB, ZEROS, false>(a, num_sms, st);
}
template <int COLS>
cudaError_t int4_group(const Int4LinearArgs& a, bool wide, int num_sms, cudaStream_t st) {
  const bool z = a.zeros != nullptr;
  if (a.w.group == 32) return z ? int4_kind<COLS, 4, true>(a, wide, num_sms, st) : int4_kind<COLS, 4, false>(a, wide, num_sms, st);
  if (a.w.group == 64) return z ? int4_kind<COLS, 2, true>(a, wide, num_sms, st) : int4_kind<COLS, 2, false>(a, wide, num_sms, st);
  return z ? int4_kind<COLS, 1, true>(a, wide, num_sms, st) : int4_kind<COLS, 1, false>(a, wide, num_sms, st);
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
  const long long parts = (s.blocks() + kReadTiles - 1) / kReadTiles;
  return launch_dependent(int4_dequantize_kernel, tile_grid(s.matrices * s.row_tiles() * parts), dim3(256), 0, st, codes, scales, zeros, s,
                          out);
}

cudaError_t launch_int4_linear(const Int4LinearArgs& args, int num_sms, cudaStream_t st) {
  Int4LinearArgs a = args;
  a.by_expert = a.experts && a.w.matrices < a.rows;
  // columns of the product: what there are, or with experts the rows that one has on average
  const double per = a.experts ? static_cast<double>(a.rows) / static_cast<double>(a.w.matrices) : static_cast<double>(a.rows);
  const int cols = per > (a.experts ? 10 : 16) ? 32 : per > (a.experts ? 5 : 8) ? 16 : per > (a.experts ? 1.25 : 2) ? 8 : 2;
  // rows of w for two blocks of 256 to an SM.  Measured, that and the other: one row times 40960 x 4096 33 and 22 us, times 152064 x
  // 4096 64 and 66; eight rows 34 and 30, 66 and 101
  const bool wide = !a.experts && a.rows <= 8 && a.w.row_tiles() / (2 * kInt4Warps) >= 2 * num_sms;
  if (cols == 32) return int4_group<32>(a, wide, num_sms, st);
  if (cols == 16) return int4_group<16>(a, wide, num_sms, st);
  if (cols == 8) return int4_group<8>(a, wide, num_sms, st);
  return int4_group<2>(a, wide, num_sms, st);
}

}  // namespace mok
