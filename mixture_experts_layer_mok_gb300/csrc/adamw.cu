// The AdamW step over many tensors in one launch, with 32-bit or MXFP8 states.
//
//   g' = grad_scale g
//   m  = b1 m + (1 - b1) g',   v = b2 v + (1 - b2) g'^2
//   p  = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
//
// MXFP8 states keep m and r = sqrt(v) as E4M3 codes with one E8M0 scale per
// 32 consecutive elements: 2 + 1/16 bytes per element instead of 8.  r rather
// than v, because E4M3 spans 2^17.8 between its largest and smallest value,
// which is 2^35.6 in v.  Both are rounded stochastically (up with probability
// equal to the distance from the lower neighbour): b2 = 0.999 changes r by
// 0.05% a step, far less than half of E4M3's 6 to 12% spacing, so rounding to
// nearest would never move it.  A positive r is never rounded to zero: m's
// step is bounded by about 3.2 r, so with the smallest code kept |m| / r stays
// bounded whatever both were rounded to.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "gemm.cuh"
#include "internal.h"
#include "ops.h"

namespace mok {
namespace {

constexpr int kAdamwPerSm = 4;   // resident blocks on each of 152 SMs

template <int CAP>
struct AdamwList {
  AdamwTensor t[CAP];
  int n;
};

__device__ __forceinline__ uint32_t mix_bits(uint32_t i, uint32_t key) {
  uint32_t h = (i + key) * 0x9E3779B1u;   // multipliers from the fractions of phi and sqrt 2
  h ^= h >> 15;
  h *= 0xB504F333u;
  return h ^ (h >> 16);
}

// Eight elements as they lie in memory.
template <class T>
struct Raw8 {
  uint32_t w[2 * sizeof(T)];
};

// `left`: elements that exist (8: all, loaded as vectors; fewer: the end of a tensor).
template <class T>
__device__ __forceinline__ Raw8<T> load8(const T* p, int left) {
  Raw8<T> r;
  if (left == 8) {
    if constexpr (sizeof(T) == 1) {
      const uint2 a = __ldcs(reinterpret_cast<const uint2*>(p));
      r.w[0] = a.x, r.w[1] = a.y;
    } else {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
        const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p) + i);
        r.w[4 * i] = a.x, r.w[4 * i + 1] = a.y, r.w[4 * i + 2] = a.z, r.w[4 * i + 3] = a.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2 * static_cast<int>(sizeof(T)); ++i) r.w[i] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < left) {
        if constexpr (sizeof(T) == 4)
          r.w[i] = __float_as_uint(p[i]);
        else if constexpr (sizeof(T) == 2)
          r.w[i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
        else
          r.w[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
      }
    }
  }
  return r;
}
__device__ __forceinline__ void values(const Raw8<float>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r.w[i]);
}
__device__ __forceinline__ void values(const Raw8<uint16_t>& r, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(r.w[i] << 16);
    f[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void values(const Raw8<uint8_t>& r, float* f) {
  e4m3x4_values(r.w[0], f);
  e4m3x4_values(r.w[1], f + 4);
}

template <class T>
__device__ __forceinline__ void store8(T* p, bool whole, int left, const float* f) {
  if (whole) {
    if constexpr (sizeof(T) == 2) {
      __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                     pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])));
    } else {
      __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
      __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) {
        if constexpr (sizeof(T) == 2)
          p[i] = __bfloat16_as_ushort(__float2bfloat16_rn(f[i]));
        else
          p[i] = f[i];
      }
  }
}

// |y| <= 448 (not NaN) onto the E4M3 grid, rounded up or down by 16 random bits: the
// bits are added below the last kept place of the fp32 form and the rest is
// cut off.  Below 2^-6 the grid is uniform (2^-9), as it is in [2^-6, 2^-5):
// such a value is moved there and back.
// `below`: the 16 random bits in places 4 to 19, zeros elsewhere.
__device__ __forceinline__ float e4m3_stochastic(float y, uint32_t below) {
  const float off = fabsf(y) < 0.015625f ? 0.015625f : 0.f;
  return __uint_as_float((__float_as_uint(fabsf(y) + off) + below) & 0xFFF00000u) - off;   // sign dropped
}

// The larger of two values; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// Writes 8 values as codes with the scale of their block of 32 (four
// neighbouring lanes); `v` are values before rounding, none of them infinite,
// `rand` their bits (m: the high half, r: the low one).  A NaN has no say in
// the scale and stays NaN.
template <bool R>
__device__ __forceinline__ void store_codes8(uint8_t* codes, uint8_t* scales, long long block, bool whole, int left,
                                             const float* v, const uint32_t* rand) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const int s = mx_scale_exponent(amax);
  const float inv = __uint_as_float(static_cast<uint32_t>(127 - s) << 23);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = v[i] * inv;
    q[i] = e4m3_stochastic(y, R ? (rand[i] << 4) & 0xFFFF0u : (rand[i] >> 12) & 0xFFFF0u);
    if (R)
      q[i] = max_nan(q[i], y > 0.f ? 0.001953125f : y);   // 2^-9, the smallest code
    else
      q[i] = fmaf(y, 0.f, copysignf(q[i], y));            // (the rounding loses a NaN)
  }
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * k], q[4 * k + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * k + 2], q[4 * k + 3]), __NV_SATFINITE, __NV_E4M3);
    w[k] = lo | (hi << 16);
  }
  if (whole) {
    __stcs(reinterpret_cast<uint2*>(codes), make_uint2(w[0], w[1]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) codes[i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
  }
  if ((threadIdx.x & 3) == 0 && left > 0) scales[block] = static_cast<uint8_t>(s + 127);
}

// What a thread reads of its eight elements.
template <class PT, class GT, bool MASTER, bool MX>
struct AdamwIn {
  using P = std::conditional_t<MASTER, float, PT>;
  using S = std::conditional_t<MX, uint8_t, float>;
  Raw8<GT> g;
  Raw8<P> p;
  Raw8<S> m, v;
  uint32_t ms, rs;   // MXFP8: the scales of the thread's block
  long long i0;
  int left, tensor;

  // Chunk `c` of the launch, of the tensor that holds it (searched from `from` on).
  template <class L>
  __device__ __forceinline__ void load(const L& list, int c, int from) {
    tensor = from;
    while (tensor + 1 < list.n && list.t[tensor + 1].first <= c) ++tensor;
    const AdamwTensor& t = list.t[tensor];
    i0 = static_cast<long long>(c - t.first) * kAdamwBlock + threadIdx.x * 8;
    const long long rest = t.n - i0;
    left = rest >= 8 ? 8 : rest > 0 ? static_cast<int>(rest) : 0;
    g = load8(static_cast<const GT*>(t.g) + i0, left);
    p = load8(static_cast<const P*>(MASTER ? static_cast<const void*>(t.master) : t.p) + i0, left);
    m = load8(static_cast<const S*>(t.m) + i0, left);
    v = load8(static_cast<const S*>(t.v) + i0, left);
    ms = rs = 0;
    if (MX && left > 0) {
      ms = t.m_scale[i0 >> 5];
      rs = t.r_scale[i0 >> 5];
    }
  }
};

// Persistent blocks of 256 threads over chunks of kAdamwBlock elements, 8 per
// thread, each chunk within one tensor; a block's next chunk is in flight
// while it works on this one.  32-bit states: a chunk to a block, bound by
// memory; bf16 parameters with master copies, 402.7M elements, 1604 us (7.0
// TB/s).  MXFP8 states: 98 instructions an element keep the issue slots busy
// 84% of the time beside 62 to 69% of the memory's peak; the same tensors 1187
// us (5.5 TB/s).  16 elements a thread took fewer instructions but left fewer
// warps, and were slower.
// COUNTED: what depends on the step count comes from device memory.
template <class PT, class GT, bool MASTER, bool MX, int CAP, bool COUNTED>
__global__ void __launch_bounds__(256, MX ? kAdamwPerSm : 6)
    adamw_kernel(const __grid_constant__ AdamwList<CAP> list, const int chunks, const AdamwScalars s,
                 const AdamwCounter* counter) {
  using In = AdamwIn<PT, GT, MASTER, MX>;
  griddep_wait();
  griddep_launch_dependents();
  const float gs = s.grad_scale ? __ldg(s.grad_scale) : 1.f;
  const float decay = COUNTED ? counter->decay : s.decay, step_size = COUNTED ? counter->step_size : s.step_size;
  const float inv_sqrt_bc2 = COUNTED ? counter->inv_sqrt_bc2 : s.inv_sqrt_bc2;
  const uint32_t step_key = COUNTED ? counter->key : 0u;
  In next;
  next.load(list, blockIdx.x, 0);
  for (int c = blockIdx.x; c < chunks;) {
    const In in = next;
    c += gridDim.x;
    if (MX && c < chunks) next.load(list, c, in.tensor);
    const AdamwTensor& t = list.t[in.tensor];
    const int left = in.left;
    if (!MX && left == 0) continue;
    const bool whole = left == 8;
    float g[8], p[8], m[8], v[8], r[8];
    values(in.g, g);
    values(in.p, p);
    values(in.m, m);
    values(in.v, v);
    if (MX) {
      const float ms = e8m0_value(in.ms), rs = e8m0_value(in.rs);
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] *= ms, v[i] *= rs, v[i] *= v[i];
    }
    // What the states keep is formed by single roundings, no fused ones, and the
    // root rounded correctly: a last-bit difference would put one element in
    // 10^6 on the other side of its random bits, a whole code away from a
    // restatement in 32 bits.  With fused operations and an approximate root
    // 402.7M elements took 1144 us, this way 1158.
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float gi = g[i] * gs;
      m[i] = __fadd_rn(__fmul_rn(s.beta1, m[i]), __fmul_rn(s.one_minus_beta1, gi));
      v[i] = __fadd_rn(__fmul_rn(s.beta2, v[i]), __fmul_rn(__fmul_rn(s.one_minus_beta2, gi), gi));
      r[i] = __fsqrt_rn(v[i]);
      p[i] = fmaf(-step_size, m[i] * fast_rcp(fmaf(r[i], inv_sqrt_bc2, s.eps)), p[i] * decay);
    }
    if (MASTER) store8(t.master + in.i0, whole, left, p);
    store8(static_cast<PT*>(t.p) + in.i0, whole, left, p);
    if (MX) {
      const long long block = in.i0 >> 5;
      // An infinity becomes NaN, which E4M3 has: as the block's scale it would
      // make each neighbour's smallest code 2^111.  These and the NaNs' way
      // through the rounding cost 2% (402.7M elements 1160 us, so 1187).
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = fmaf(m[i], 0.f, m[i]), r[i] = fmaf(r[i], 0.f, r[i]);
      uint32_t rand[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) rand[i] = mix_bits(static_cast<uint32_t>(in.i0) + i, t.key + step_key);
      store_codes8<false>(static_cast<uint8_t*>(t.m) + in.i0, t.m_scale, block, whole, left, m, rand);
      store_codes8<true>(static_cast<uint8_t*>(t.v) + in.i0, t.r_scale, block, whole, left, r, rand);
    } else {
      store8(static_cast<float*>(t.m) + in.i0, whole, left, m);
      store8(static_cast<float*>(t.v) + in.i0, whole, left, v);
    }
  }
}

// The list is handed over by address: through the launch templates, which take
// arguments by value, its 30 KB would be copied twice more.
template <class PT, class GT, bool MASTER, bool MX, int CAP, bool COUNTED>
cudaError_t launch_cap(const AdamwTensor* t, int n, int chunks, const AdamwScalars& s, const AdamwCounter* counter,
                       cudaStream_t st) {
  AdamwList<CAP> list;
  memcpy(list.t, t, sizeof(AdamwTensor) * n);
  list.n = n;
  constexpr int kResident = 152 * kAdamwPerSm;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(MX && chunks > kResident ? kResident : chunks);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  AdamwScalars scalars = s;
  void* args[] = {&list, &chunks, &scalars, &counter};
  return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(adamw_kernel<PT, GT, MASTER, MX, CAP, COUNTED>), args);
}

template <class PT, class GT, bool MASTER, bool MX>
cudaError_t launch_typed(const AdamwTensor* t, int n, int chunks, const AdamwScalars& s, const AdamwCounter* counter,
                         cudaStream_t st) {
  // a counted step's list is copied at its capture only: one size will do
  if (counter) return launch_cap<PT, GT, MASTER, MX, kAdamwMaxTensors, true>(t, n, chunks, s, counter, st);
  if (n <= 16) return launch_cap<PT, GT, MASTER, MX, 16, false>(t, n, chunks, s, nullptr, st);
  if (n <= 128) return launch_cap<PT, GT, MASTER, MX, 128, false>(t, n, chunks, s, nullptr, st);
  return launch_cap<PT, GT, MASTER, MX, kAdamwMaxTensors, false>(t, n, chunks, s, nullptr, st);
}

template <class PT, class GT, bool MASTER>
cudaError_t launch_state(const AdamwTensor* t, int n, int chunks, const AdamwScalars& s, const AdamwCounter* counter, int mx,
                         cudaStream_t st) {
  return mx ? launch_typed<PT, GT, MASTER, true>(t, n, chunks, s, counter, st)
            : launch_typed<PT, GT, MASTER, false>(t, n, chunks, s, counter, st);
}

// One step more, and what depends on its number, in 64 bits as on the host.
__global__ void adamw_advance_kernel(const AdamwAdvance a, AdamwCounter* c) {
  griddep_wait();   // the step before this one has read what is written here
  griddep_launch_dependents();
  const long long count = ++c->count, step = a.step + count;
  const double lr = a.fixed_lr || isnan(c->lr) ? a.lr : c->lr;
  c->decay = static_cast<float>(1.0 - lr * a.weight_decay);
  c->step_size = static_cast<float>(lr / (1.0 - pow(a.beta1, static_cast<double>(step))));
  c->inv_sqrt_bc2 = static_cast<float>(1.0 / sqrt(1.0 - pow(a.beta2, static_cast<double>(step))));
  c->key = adamw_step_key(a.seed ^ c->seed_change, step);
}

}  // namespace

cudaError_t launch_adamw_advance(const AdamwAdvance& a, AdamwCounter* counter, cudaStream_t st) {
  return launch_dependent(adamw_advance_kernel, dim3(1), dim3(1), 0, st, a, counter);
}

cudaError_t launch_adamw(const AdamwTensor* t, int n, int chunks, const AdamwScalars& s, const AdamwCounter* counter, int p_f32,
                         int g_f32, int master, int mx, cudaStream_t st) {
  if (p_f32)
    return g_f32 ? launch_state<float, float, false>(t, n, chunks, s, counter, mx, st)
                 : launch_state<float, uint16_t, false>(t, n, chunks, s, counter, mx, st);
  if (master)
    return g_f32 ? launch_state<uint16_t, float, true>(t, n, chunks, s, counter, mx, st)
                 : launch_state<uint16_t, uint16_t, true>(t, n, chunks, s, counter, mx, st);
  return g_f32 ? launch_state<uint16_t, float, false>(t, n, chunks, s, counter, mx, st)
               : launch_state<uint16_t, uint16_t, false>(t, n, chunks, s, counter, mx, st);
}

}  // namespace mok
