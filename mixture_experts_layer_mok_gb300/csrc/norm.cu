// Root-mean-square norm with the residual's addition, an output in bf16 and /
// or MXFP8, and its backward; and the reader of MXFP8 tensors.
//
// Forward, per row:  h = x + residual,  r = (mean(h^2) + eps)^-1/2,
//                    y_j = w_j h_j r.
// Backward, with g_j = w_j dy_j and xhat_j = h_j r:
//                    dx_j = r (g_j - xhat_j mean(g xhat)) + dh_j,
//                    dw_j = sum over rows of dy_j xhat_j.
// Both are bound by memory: a row is read once and stays in registers between
// the sum over it and the values that need the sum.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gemm.cuh"
#include "internal.h"
#include "ops.h"

namespace mok {
namespace {

struct NoType {};
// The other of the two types that a stream has.
template <class T>
using Other = std::conditional_t<sizeof(T) == 4, uint16_t, float>;

// V consecutive values (8, or 1 where a row's length is not a multiple of 8)
// as they lie in memory.
template <class T, int V>
struct Raw {
  T v[V];
};
template <>
struct Raw<uint16_t, 8> {
  uint4 v;
};
template <>
struct Raw<float, 8> {
  float4 v[2];
};
template <int V>
struct Raw<NoType, V> {};

template <class T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T* p) {
  Raw<T, V> r;
  if constexpr (V == 8 && sizeof(T) == 2) {
    r.v = __ldcs(reinterpret_cast<const uint4*>(p));
  } else if constexpr (V == 8) {
    r.v[0] = __ldcs(reinterpret_cast<const float4*>(p));
    r.v[1] = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = p[i];
  }
  return r;
}

__device__ __forceinline__ void unpack(const Raw<uint16_t, 8>& r, float* f) {
  const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack(const Raw<float, 8>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[4 * i] = r.v[i].x;
    f[4 * i + 1] = r.v[i].y;
    f[4 * i + 2] = r.v[i].z;
    f[4 * i + 3] = r.v[i].w;
  }
}
__device__ __forceinline__ void unpack(const Raw<uint16_t, 1>& r, float* f) {
  f[0] = __uint_as_float(static_cast<uint32_t>(r.v[0]) << 16);
}
__device__ __forceinline__ void unpack(const Raw<float, 1>& r, float* f) { f[0] = r.v[0]; }

template <int V>
__device__ __forceinline__ void store_vals(uint16_t* p, const float* f) {
  if constexpr (V == 8) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                                                   pack_bf16(f[6], f[7])));
  } else {
    p[0] = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
  }
}
template <int V>
__device__ __forceinline__ void store_vals(float* p, const float* f) {
  if constexpr (V == 8) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
  } else {
    p[0] = f[0];
  }
}

// V weights at element j (bf16 or fp32), through the read-only cache: every
// row reads the same ones.
template <int V>
__device__ __forceinline__ void load_weight(const void* w, bool f32, int j, float* f) {
  if (f32) {
    const float* p = static_cast<const float*>(w) + j;
    if constexpr (V == 8) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
      f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
      f[0] = __ldg(p);
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(w) + j;
    if constexpr (V == 8) {
      Raw<uint16_t, 8> r;
      r.v = __ldg(reinterpret_cast<const uint4*>(p));
      unpack(r, f);
    } else {
      f[0] = __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
    }
  }
}

__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Sum over the threads of a row: the warp, or the block (`red`: one slot per
// warp; the caller alternates two of them, so that one barrier per row is
// enough).  Fixed order.
template <bool WARP_ROW>
__device__ __forceinline__ float row_sum(float s, float* red) {
  s = warp_sum(s);
  if constexpr (!WARP_ROW) {
    const int nw = (blockDim.x + 31) >> 5;
    if (nw > 1) {
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
      __syncthreads();
      s = 0.f;
      for (int i = 0; i < nw; ++i) s += red[i];
    }
  }
  return s;
}

constexpr int kWarpRows = 4;   // rows of a block in the one-warp-per-row kernels

// XT: x's type; RT: the residual's (NoType: none).  V values per load, ITEMS
// loads per thread; WARP_ROW: one warp per row, else one block.  Bound by
// memory where lengths are a multiple of 8: bf16 with a bf16 residual, 65536 x
// 7168, 526 us (7.1 TB/s); an fp32 residual and MXFP8 out, 16384 x 4096, 102.5 us
// (7.2 TB/s), with bf16 out too 127 us (6.9 TB/s); 2048 x 32768 87 us (6.2 TB/s);
// one row 5.6 us, a launch and two trips to memory.  Other lengths go an element
// a load, bound by instructions: 67041 x 1001 146 us (3.7 TB/s), 16388 x 4095 186,
// and above 4096, where a thread of 1024 spills up to 164 bytes, 16380 x 4097 251
// us and 2048 x 32767 299 (2.1 and 1.8 TB/s).
template <class XT, class RT, int V, int ITEMS, bool WARP_ROW, int MAXT>
__global__ void __launch_bounds__(MAXT) rms_norm_kernel(const NormArgs a) {
  constexpr bool kRes = !std::is_same_v<RT, NoType>;
  __shared__ float red[32];
  griddep_wait();
  griddep_launch_dependents();
  const int T = WARP_ROW ? 32 : blockDim.x;
  const int tid = WARP_ROW ? threadIdx.x & 31 : threadIdx.x;
  const long long row = WARP_ROW ? static_cast<long long>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP_ROW && row >= a.rows) return;   // whole warps; no block barrier in this form
  const int nv = a.H / V;
  const long long base = row * a.H;
  Raw<XT, V> rx[ITEMS];
  Raw<RT, V> rr[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = tid + i * T;
    if (c < nv) {
      rx[i] = load_raw<XT, V>(static_cast<const XT*>(a.x) + base + c * V);
      if constexpr (kRes) rr[i] = load_raw<RT, V>(static_cast<const RT*>(a.residual) + base + c * V);
    }
  }
  float v[ITEMS][V];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = tid + i * T;
    if (c < nv) {
      unpack(rx[i], v[i]);
      if constexpr (kRes) {
        float r[V];
        unpack(rr[i], r);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] += r[j];
        store_vals<V>(static_cast<RT*>(a.h) + base + c * V, v[i]);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = 0.f;
    }
  }
  ss = row_sum<WARP_ROW>(ss, red);
  const float rstd = rsqrtf(ss / static_cast<float>(a.H) + a.eps);
  if (tid == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = tid + i * T;
    if (c < nv) {
      float w[V];
      load_weight<V>(a.weight, a.weight_f32, c * V, w);
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] *= rstd * w[j];
      if (a.y) store_vals<V>(a.y + base + c * V, v[i]);
    }
    if constexpr (V == 8) {
      if (a.codes) {
        // four neighbouring lanes hold a block of 32 (H is a multiple of 32,
        // so the four are all inside the row or all outside); lanes outside
        // hold zeros and only take part in the shuffles
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[i][j]));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int s = mx_scale_exponent(amax);
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - s) << 23);
        uint32_t q[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[i][4 * k] * inv, v[i][4 * k + 1] * inv),
                                                       __NV_SATFINITE, __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[i][4 * k + 2] * inv, v[i][4 * k + 3] * inv),
                                                       __NV_SATFINITE, __NV_E4M3);
          q[k] = lo | (hi << 16);
        }
        if (c < nv) {
          __stcs(reinterpret_cast<uint2*>(a.codes + base + c * 8), make_uint2(q[0], q[1]));
          if ((c & 3) == 0) a.scales[row * (a.H / 32) + (c >> 2)] = static_cast<uint8_t>(s + 127);
        }
      }
    }
  }
}

// The sums of R values over the W warps of a row, in a fixed order.  `red`: 32
// slots of R; the caller alternates two of them, so that one barrier (of the
// row's warps alone) serves R rows.
template <int W, int R>
__device__ __forceinline__ void row_sums(float (&s)[R], float (*red)[R]) {
#pragma unroll
  for (int r = 0; r < R; ++r) s[r] = warp_sum(s[r]);
  if constexpr (W > 1) {
    const int warp = threadIdx.x >> 5, first = warp / W * W;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) red[warp][r] = s[r];
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / W), "n"(32 * W) : "memory");
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[r] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s[r] += red[first + w][r];
    }
  }
}

// The backward: a grid of fixed size, W warps to a row and ITEMS x 8 of its
// elements to a thread; each such group walks the rows, R at a time, and keeps
// its columns' share of dw in registers.  `part` gets one row of sums per block,
// which column_sum_kernel adds in order.
//   acc_j += rstd (dy_j h_j),   s = sum_j w_j dy_j h_j,   k = -((s rstd) / H) rstd,
//   dx_j = rstd (w_j dy_j + k h_j) + dh_j
// (s rstd) / H is the mean of g xhat and k h_j that times xhat_j, of order 1
// whatever the size of h; with rstd^3 in one factor dx would be lost for rows of
// a root mean square above 1e12 or below 1e-13.
template <class HT, bool BOTH, int ITEMS, int R, int W, int THREADS>
__global__ void __launch_bounds__(THREADS) rms_norm_bwd_kernel(const NormBwdArgs a) {
  constexpr int kGroups = THREADS / (32 * W), T = 32 * W;
  __shared__ float red[2][32][R];
  __shared__ float sums[kGroups > 1 ? kGroups : 1][kGroups > 1 ? T * ITEMS * 8 : 1];
  griddep_wait();
  griddep_launch_dependents();
  const int group = threadIdx.x / T, tid = threadIdx.x % T, nv = a.H / 8;
  const long long step = static_cast<long long>(gridDim.x) * kGroups * R;
  float acc[ITEMS][8];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  const float inv_h = 1.f / static_cast<float>(a.H);
  int odd = 0;
  for (long long row0 = (static_cast<long long>(blockIdx.x) * kGroups + group) * R; row0 < a.rows; row0 += step, odd ^= 1) {
    Raw<uint16_t, 8> dy[R][ITEMS];
    Raw<HT, 8> h[R][ITEMS], dh[R][ITEMS];
    float rstd[R], dot[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool in = row0 + r < a.rows;
      const long long base = (row0 + r) * a.H;
      rstd[r] = in ? __ldg(a.rstd + row0 + r) : 0.f;
      dot[r] = 0.f;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int c = tid + i * T;
        dy[r][i] = {};
        h[r][i] = {};
        dh[r][i] = {};
        if (in && c < nv) {
          dy[r][i] = load_raw<uint16_t, 8>(a.dy + base + c * 8);
          h[r][i] = load_raw<HT, 8>(static_cast<const HT*>(a.h) + base + c * 8);
          if (a.dh) dh[r][i] = load_raw<HT, 8>(static_cast<const HT*>(a.dh) + base + c * 8);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * T;
      if (c < nv) {
        float w[8];
        load_weight<8>(a.weight, a.weight_f32, c * 8, w);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float y[8], x[8];
          unpack(dy[r][i], y);
          unpack(h[r][i], x);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float t = y[j] * x[j];
            acc[i][j] = fmaf(t, rstd[r], acc[i][j]);
            dot[r] = fmaf(t, w[j], dot[r]);
          }
        }
      }
    }
    row_sums<W, R>(dot, red[odd]);
#pragma unroll
    for (int r = 0; r < R; ++r) dot[r] = dot[r] * rstd[r] * -inv_h * rstd[r];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * T;
      if (c < nv) {
        float w[8];
        load_weight<8>(a.weight, a.weight_f32, c * 8, w);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if (row0 + r < a.rows) {
            const long long at = (row0 + r) * a.H + c * 8;
            float y[8], x[8], d[8];
            unpack(dy[r][i], y);
            unpack(h[r][i], x);
            unpack(dh[r][i], d);
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = fmaf(fmaf(x[j], dot[r], y[j] * w[j]), rstd[r], d[j]);
            store_vals<8>(static_cast<HT*>(a.dx) + at, d);
            if (BOTH && a.dx_other) store_vals<8>(static_cast<Other<HT>*>(a.dx_other) + at, d);
          }
        }
      }
    }
  }
  float* part = a.part + static_cast<long long>(blockIdx.x) * a.H;
  if constexpr (kGroups > 1) {   // the block's groups in order
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) sums[group][(tid + i * T) * 8 + j] = acc[i][j];
    __syncthreads();
    for (int c = threadIdx.x; c < a.H; c += THREADS) {
      float v = 0.f;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) v += sums[g][c];
      part[c] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * T;
      if (c < nv) {
#pragma unroll
        for (int j = 0; j < 8; ++j) part[c * 8 + j] = acc[i][j];
      }
    }
  }
}

// The same with a block to a row, the next row's values in registers: for middle
// lengths, whose rows one block's threads hold in 8 elements each, bound by
// memory, between 5.4 TB/s (512 columns) and 6.2 (8192): a row's sum is a barrier,
// with one row more in flight behind it.  Rings of asynchronous copies and
// several rows a block were slower.  And for the lengths that nothing was made
// for.  Not a multiple of 8: an element a load, bound by instructions, 67041 x
// 1001 152 us (3.5 TB/s), 16388 x 4095 171; above 4096 besides by the 1.3 to 2.5 KB
// that a thread of 1024 spills, 16380 x 4097 1.78 ms (0.3 TB/s), 8193 x 8191 1.51,
// 2048 x 32767 1.37; above 16384 likewise, 2048 x 32768 373 us in bf16 and 880 in
// fp32 (1.4 and 1.1 TB/s).
template <class HT, bool BOTH, int V, int ITEMS, int MAXT>
__global__ void __launch_bounds__(MAXT) rms_norm_bwd_block_kernel(const NormBwdArgs a) {
  __shared__ float red[2][32];
  griddep_wait();
  griddep_launch_dependents();
  const int T = blockDim.x, tid = threadIdx.x;
  const long long walkers = gridDim.x, walker = blockIdx.x;
  const int nv = a.H / V;
  float acc[ITEMS][V], w[ITEMS][V];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = tid + i * T;
#pragma unroll
    for (int j = 0; j < V; ++j) acc[i][j] = w[i][j] = 0.f;
    if (c < nv) load_weight<V>(a.weight, a.weight_f32, c * V, w[i]);
  }
  const float inv_h = 1.f / static_cast<float>(a.H);
  // one row ahead: the next row's loads are in flight while this one is summed
  Raw<uint16_t, V> ndy[ITEMS];
  Raw<HT, V> nh[ITEMS], ndh[ITEMS];
  float nr = 0.f;
  const auto fetch = [&](long long row) {
    if (row >= a.rows) return;
    const long long base = row * a.H;
    nr = __ldg(a.rstd + row);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * T;
      if (c < nv) {
        ndy[i] = load_raw<uint16_t, V>(a.dy + base + c * V);
        nh[i] = load_raw<HT, V>(static_cast<const HT*>(a.h) + base + c * V);
        if (a.dh) ndh[i] = load_raw<HT, V>(static_cast<const HT*>(a.dh) + base + c * V);
      }
    }
  };
  fetch(walker);
  int odd = 0;
  for (long long row = walker; row < a.rows; row += walkers, odd ^= 1) {
    const long long base = row * a.H;
    const float rstd = nr;
    Raw<uint16_t, V> rdy[ITEMS];
    Raw<HT, V> rh[ITEMS], rdh[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) rdy[i] = ndy[i], rh[i] = nh[i], rdh[i] = ndh[i];
    fetch(row + walkers);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (tid + i * T < nv) {
        float dy[V], h[V];
        unpack(rdy[i], dy);
        unpack(rh[i], h);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float t = dy[j] * h[j];
          acc[i][j] = fmaf(t, rstd, acc[i][j]);
          dot = fmaf(t, w[i][j], dot);
        }
      }
    }
    const float k = row_sum<false>(dot, red[odd]) * rstd * -inv_h * rstd;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * T;
      if (c < nv) {
        float dy[V], h[V], d[V] = {};
        unpack(rdy[i], dy);
        unpack(rh[i], h);
        if (a.dh) unpack(rdh[i], d);
#pragma unroll
        for (int j = 0; j < V; ++j) d[j] = fmaf(fmaf(h[j], k, dy[j] * w[i][j]), rstd, d[j]);
        store_vals<V>(static_cast<HT*>(a.dx) + base + c * V, d);
        if (BOTH && a.dx_other) store_vals<V>(static_cast<Other<HT>*>(a.dx_other) + base + c * V, d);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = tid + i * T;
    if (c < nv) {
#pragma unroll
      for (int j = 0; j < V; ++j) a.part[walker * a.H + c * V + j] = acc[i][j];
    }
  }
}

// Column sums of [n][H] fp32 partial rows, in a fixed order: 32 columns per
// block, 32 rows in step, then the 32 running sums.  LATE: the kernel launched
// before this one does not write `part` and waited itself for the one that
// does, so that the sums may run beside it (it lets its dependents start only
// after that wait); this kernel still ends after it, for what follows on the
// stream.  4 us after 608 rows of partial sums, one trip to L2 and two barriers.
template <bool LATE>
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* __restrict__ part, int n, int H,
                                                          float* __restrict__ out) {
  __shared__ float s[32][33];
  if (!LATE) griddep_wait();
  griddep_launch_dependents();
  const int col = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (col < H) {
#pragma unroll 8
    for (int r = threadIdx.y; r < n; r += 32) v += part[static_cast<long long>(r) * H + col];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && col < H) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += s[i][threadIdx.x];
    out[col] = v;
  }
  if (LATE) griddep_wait();
}

// E4M3 codes and E8M0 scales -> bf16: 16 codes per thread, half a block.  Bound
// by memory: 402.7M codes 189 us, 6.5 TB/s (8 codes per thread: 216 us).
__global__ void __launch_bounds__(256) mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, long long n,
                                                            uint16_t* __restrict__ out) {
  griddep_wait();
  griddep_launch_dependents();
  const long long c = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x, at = c * 16;
  if (at >= n) return;
  if (at + 16 <= n) {
    const uint4 q = __ldcs(reinterpret_cast<const uint4*>(codes) + c);
    const float s = e8m0_value(__ldg(scales + (c >> 1)));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    float f[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) e4m3x4_values(w[i], f + 4 * i);
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] *= s;
    store_vals<8>(out + at, f);
    store_vals<8>(out + at + 8, f + 8);
  } else {
    const float s = e8m0_value(scales[c >> 1]);
    for (long long i = at; i < n; ++i) {
      float f[4];
      e4m3x4_values(codes[i], f);
      f[0] *= s;
      store_vals<1>(out + i, f);
    }
  }
}

int ceil32(int n) { return (n + 31) / 32 * 32; }

template <class XT, class RT>
cudaError_t norm_launch(const NormArgs& a, cudaStream_t st) {
  const unsigned rows = static_cast<unsigned>(a.rows);
  const unsigned wgrid = static_cast<unsigned>((a.rows + kWarpRows - 1) / kWarpRows);
  if (a.H % 8) {
    if (a.H <= 4096)
      return launch_dependent(rms_norm_kernel<XT, RT, 1, 4, false, 1024>, dim3(rows), dim3(ceil32((a.H + 3) / 4)), 0, st, a);
    return launch_dependent(rms_norm_kernel<XT, RT, 1, 32, false, 1024>, dim3(rows), dim3(ceil32((a.H + 31) / 32)), 0, st, a);
  }
  const int nv = a.H / 8;
  if (nv <= 32) return launch_dependent(rms_norm_kernel<XT, RT, 8, 1, true, 128>, dim3(wgrid), dim3(128), 0, st, a);
  if (nv <= 64) return launch_dependent(rms_norm_kernel<XT, RT, 8, 2, true, 128>, dim3(wgrid), dim3(128), 0, st, a);
  if (nv <= 128) return launch_dependent(rms_norm_kernel<XT, RT, 8, 4, true, 128>, dim3(wgrid), dim3(128), 0, st, a);
  if (nv <= 256)
    return launch_dependent(rms_norm_kernel<XT, RT, 8, 1, false, 256>, dim3(rows), dim3(ceil32(nv)), 0, st, a);
  if (nv <= 512)
    return launch_dependent(rms_norm_kernel<XT, RT, 8, 2, false, 256>, dim3(rows), dim3(ceil32((nv + 1) / 2)), 0, st, a);
  if (nv <= 1024)
    return launch_dependent(rms_norm_kernel<XT, RT, 8, 4, false, 256>, dim3(rows), dim3(ceil32((nv + 3) / 4)), 0, st, a);
  return launch_dependent(rms_norm_kernel<XT, RT, 8, 4, false, 1024>, dim3(rows), dim3(ceil32((nv + 3) / 4)), 0, st, a);
}

// The backward's kernel for a row length.  Measured (us; groups of warps, block
// per row): 65536 x 512 bf16 45 and 47, 16384 x 2048 65 and 49, 16384 x 7168 162
// and 173, in fp32 305 and 265, 1000 x 16384 bf16 40 and 108.
bool bwd_groups(int H, bool f32) { return H % 8 == 0 && H <= 16384 && (H <= 512 || H > (f32 ? 8192 : 4096)); }

// BOTH: dx in the other type too, where the pointer says so.  For an fp32 h always
// built in; a bf16 one has a form without: there the test alone takes the odd
// lengths up to 4096 from 152 to 172 us (67041 x 1001) and those above 16384 from
// 329 to 560 (4094 x 16392, whose registers spill).
template <class HT, bool BOTH>
cudaError_t norm_bwd_launch(const NormBwdArgs& a, int blocks, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(blocks));
  const int H = a.H, nv = H / 8;
  if (bwd_groups(H, sizeof(HT) == 4)) {
    if (H <= 256) return launch_dependent(rms_norm_bwd_kernel<HT, BOTH, 1, 4, 1, 128>, grid, dim3(128), 0, st, a);
    if (H <= 512) return launch_dependent(rms_norm_bwd_kernel<HT, BOTH, 2, 2, 1, 128>, grid, dim3(128), 0, st, a);
    if constexpr (sizeof(HT) == 2)
      if (H <= 8192) return launch_dependent(rms_norm_bwd_kernel<HT, BOTH, 4, 1, 8, 256>, grid, dim3(256), 0, st, a);
    return launch_dependent(rms_norm_bwd_kernel<HT, BOTH, 4, 1, 16, 512>, grid, dim3(512), 0, st, a);
  }
  if (H % 8) {
    if (H <= 4096) return launch_dependent(rms_norm_bwd_block_kernel<HT, BOTH, 1, 4, 1024>, grid, dim3(ceil32((H + 3) / 4)), 0, st, a);
    return launch_dependent(rms_norm_bwd_block_kernel<HT, BOTH, 1, 32, 1024>, grid, dim3(ceil32((H + 31) / 32)), 0, st, a);
  }
  if (H <= 4096) return launch_dependent(rms_norm_bwd_block_kernel<HT, BOTH, 8, 1, 512>, grid, dim3(ceil32(nv)), 0, st, a);
  if (H <= 8192) return launch_dependent(rms_norm_bwd_block_kernel<HT, BOTH, 8, 2, 512>, grid, dim3(ceil32((nv + 1) / 2)), 0, st, a);
  return launch_dependent(rms_norm_bwd_block_kernel<HT, BOTH, 8, 4, 1024>, grid, dim3(ceil32((nv + 3) / 4)), 0, st, a);
}

}  // namespace

int norm_bwd_walkers(long long rows, int H, bool f32) {
  long long each = 1, most = H % 8 == 0 && H <= 1024 ? 1216 : 608;   // rows that a block works on at a time; blocks
  if (bwd_groups(H, f32)) {
    each = H <= 256 ? 16 : H <= 512 ? 8 : 1;
    most = H <= 512 ? 608 : H <= 8192 ? 304 : 152;
  }
  const long long groups = (rows + each - 1) / each;
  if (groups == 0) return 0;
  const long long turns = (groups + most - 1) / most;   // every block as many, but for the last
  return static_cast<int>((groups + turns - 1) / turns);
}

cudaError_t launch_rms_norm(const NormArgs& a, int x_f32, int residual, cudaStream_t st) {
  if (a.rows == 0) return cudaSuccess;
  if (x_f32) {
    if (residual == 0) return norm_launch<float, NoType>(a, st);
    return residual == 1 ? norm_launch<float, uint16_t>(a, st) : norm_launch<float, float>(a, st);
  }
  if (residual == 0) return norm_launch<uint16_t, NoType>(a, st);
  return residual == 1 ? norm_launch<uint16_t, uint16_t>(a, st) : norm_launch<uint16_t, float>(a, st);
}

cudaError_t launch_column_sum(const float* part, int n, int H, float* out, bool late, cudaStream_t st) {
  return launch_dependent(late ? column_sum_kernel<true> : column_sum_kernel<false>, dim3((H + 31) / 32), dim3(32, 32), 0, st,
                          part, n, H, out);
}

cudaError_t launch_rms_norm_bwd(const NormBwdArgs& a, int h_f32, float* d_weight, cudaStream_t st) {
  const int walkers = norm_bwd_walkers(a.rows, a.H, h_f32 != 0);
  if (walkers > 0) {
    const cudaError_t err = h_f32        ? norm_bwd_launch<float, true>(a, walkers, st)
                            : a.dx_other ? norm_bwd_launch<uint16_t, true>(a, walkers, st)
                                         : norm_bwd_launch<uint16_t, false>(a, walkers, st);
    if (err != cudaSuccess) return err;
  }
  return launch_column_sum(a.part, walkers, a.H, d_weight, false, st);
}

cudaError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, long long n, uint16_t* out,
                                 cudaStream_t st) {
  const long long grid = (n + 16 * 256 - 1) / (16 * 256);
  return launch_dependent(mx_dequantize_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, st, codes, scales, n, out);
}

}  // namespace mok
