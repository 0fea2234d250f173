// The router: each token's k experts and their weights from its logits, what
// the balance and z losses need, and the gradient of the logits.
//
// A warp to a token; lane l holds the V consecutive logits from l V on, so that
// the lowest lane of several with the same largest value holds the lowest
// index.  The k largest are taken one after the other: each lane keeps the
// largest of what is left of its own, one warp reduction finds the largest of
// those, and only the lane that held it looks for its next.
#include <cuda_runtime.h>
#include <stdint.h>

#include "api_util.h"
#include "experts.h"
#include "gemm.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace mok {
namespace {

constexpr int kRouteWarps = 8;
constexpr unsigned kAll = 0xffffffffu;

// Unsigned integers in the order of the values: -0 as 0, NaN above all, and
// above 0, which stands for nothing.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if (x != x) return 0xffffffffu;
  return u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
}

// Lane l's V logits; -inf behind the last.
template <class LT, int V>
__device__ __forceinline__ void load_logits(const LT* row, int E, int lane, float (&x)[V]) {
  constexpr int kVec = sizeof(LT) == 4 ? (V < 4 ? V : 4) : (V < 8 ? V : 8);
  const int at = lane * V;
  if (kVec > 1 && E % kVec == 0) {   // rows begin on whole vectors, and a vector is inside or behind
#pragma unroll
    for (int i = 0; i < V; i += kVec) {
      if (at + i < E) {
        if constexpr (sizeof(LT) == 4) {
          if constexpr (kVec == 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(row + at + i));
            x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
          } else if constexpr (kVec == 2) {
            const float2 v = __ldg(reinterpret_cast<const float2*>(row + at + i));
            x[i] = v.x, x[i + 1] = v.y;
          }
        } else {
          uint32_t w[(kVec + 1) / 2];
          if constexpr (kVec == 8) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + at + i));
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
          } else if constexpr (kVec == 4) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + at + i));
            w[0] = v.x, w[1] = v.y;
          } else {
            w[0] = __ldg(reinterpret_cast<const uint32_t*>(row + at + i));
          }
#pragma unroll
          for (int j = 0; j < kVec / 2; ++j) {
            x[i + 2 * j] = __uint_as_float(w[j] << 16);
            x[i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) x[i + j] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (at + i >= E)
        x[i] = -INFINITY;
      else if constexpr (sizeof(LT) == 4)
        x[i] = __ldg(row + at + i);
      else
        x[i] = __uint_as_float(static_cast<uint32_t>(__ldg(row + at + i)) << 16);
    }
  }
}

template <class LT>
__device__ __forceinline__ float logit_at(const LT* row, long long i) {
  if constexpr (sizeof(LT) == 4) return __ldg(row + i);
  return __uint_as_float(static_cast<uint32_t>(__ldg(row + i)) << 16);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

// The row's largest logit (0 where it is -inf: exp(x - 0) is then 0 for all)
// and e[i] = exp(x[i] - it); returns the sum of e.
template <int V>
__device__ __forceinline__ float exps(const float (&x)[V], float (&e)[V], float& top) {
  float m = x[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = fmaxf(m, x[i]);
  m = warp_max(m);
  top = m == -INFINITY ? 0.f : m;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) sum += e[i] = expf(x[i] - top);
  return warp_sum(sum);
}

template <class LT, int V>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteArgs a) {
  extern __shared__ float shared[];   // with counts: [E] counts, then [kRouteWarps][E] sums of scores
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool balance = a.counts != nullptr;
  int* cnt = reinterpret_cast<int*>(shared);
  if (balance) {
    for (int i = threadIdx.x; i < a.E; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
  }
  float mean[V];
#pragma unroll
  for (int i = 0; i < V; ++i) mean[i] = 0.f;
  const long long step = static_cast<long long>(gridDim.x) * kRouteWarps;
  for (long long t = static_cast<long long>(blockIdx.x) * kRouteWarps + warp; t < a.T; t += step) {
    float x[V], s[V], top;
    load_logits<LT, V>(static_cast<const LT*>(a.logits) + t * a.E, a.E, lane, x);
    const float total = exps<V>(x, s, top);
    if (lane == 0) a.lse[t] = top == INFINITY ? top : top + logf(total);
    const float inv = total > 0.f || total != total ? 1.f / total : 0.f;
    if (a.sigmoid) {
      if (balance || a.bias) {
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = sigmoid(x[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] *= inv;
    }
    if (balance) {
#pragma unroll
      for (int i = 0; i < V; ++i) mean[i] += s[i];
    }
    // the choice: by the logits, in whose order the scores are, or by score + bias
    uint32_t key[V], most = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      float by = x[i];
      if (a.bias && e < a.E && x[i] != -INFINITY) by = s[i] + __ldg(a.bias + e);
      key[i] = e < a.E ? order_key(by) : 0u;
      most = max(most, key[i]);
    }
    int id[2] = {0, 0};
    float picked[2] = {-INFINITY, -INFINITY};   // the logits of the picked, lane j's j-th and (j + 32)-th
    for (int j = 0; j < a.k; ++j) {
      const uint32_t best = __reduce_max_sync(kAll, most);
      const int src = __ffs(__ballot_sync(kAll, most == best)) - 1;
      int at = 0;
      float val = 0.f;
      if (lane == src) {
        most = 0;
        bool found = false;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const bool it = !found && key[i] == best;
          if (it) at = lane * V + i, val = x[i], key[i] = 0;
          found = found || it;
          most = max(most, key[i]);
        }
      }
      at = __shfl_sync(kAll, at, src);
      val = __shfl_sync(kAll, val, src);
      if (lane == (j & 31)) {
        if (j < 32)
          id[0] = at, picked[0] = val;
        else
          id[1] = at, picked[1] = val;
      }
    }
    float w[2], sum = 0.f, first = -INFINITY;
    if (!a.sigmoid && a.normalize) {   // from the largest of the picked, whatever the others sum to
      first = warp_max(fmaxf(picked[0], picked[1]));
      if (first == -INFINITY) first = 0.f;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool have = lane + 32 * h < a.k;
      if (a.sigmoid)
        w[h] = have ? sigmoid(picked[h]) : 0.f;
      else
        w[h] = have ? (a.normalize ? expf(picked[h] - first) : expf(picked[h] - top) * inv) : 0.f;
      sum += w[h];
    }
    if (a.normalize) {
      sum = warp_sum(sum);
      const float by = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
      w[0] *= by, w[1] *= by;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = lane + 32 * h;
      if (j < a.k) {
        a.experts[t * a.k + j] = id[h];
        a.weights[t * a.k + j] = w[h] * a.scale;
        if (balance) atomicAdd(cnt + id[h], 1);   // whole numbers: any order
      }
    }
  }
  if (!balance) return;
  float* sums = shared + a.E;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (lane * V + i < a.E) sums[warp * a.E + lane * V + i] = mean[i];
  __syncthreads();
  int* part_cnt = reinterpret_cast<int*>(a.part + static_cast<long long>(gridDim.x) * a.E);
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kRouteWarps; ++w) v += sums[w * a.E + e];
    a.part[static_cast<long long>(blockIdx.x) * a.E + e] = v;
    part_cnt[static_cast<long long>(blockIdx.x) * a.E + e] = cnt[e];
  }
}

// The blocks' parts joined in order: 32 experts a block, 32 parts in step.
__global__ void __launch_bounds__(1024) route_join_kernel(const float* __restrict__ part, int n, int E, float inv_t,
                                                          int* __restrict__ counts, float* __restrict__ mean_score) {
  __shared__ float s[32][33];
  __shared__ int c[32][33];
  griddep_wait();
  griddep_launch_dependents();
  const int e = blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  int m = 0;
  if (e < E) {
    const int* part_cnt = reinterpret_cast<const int*>(part + static_cast<long long>(n) * E);
#pragma unroll 4
    for (int b = threadIdx.y; b < n; b += 32) {
      v += part[static_cast<long long>(b) * E + e];
      m += part_cnt[static_cast<long long>(b) * E + e];
    }
  }
  s[threadIdx.y][threadIdx.x] = v;
  c[threadIdx.y][threadIdx.x] = m;
  __syncthreads();
  if (threadIdx.y == 0 && e < E) {
    v = 0.f, m = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += s[i][threadIdx.x], m += c[i][threadIdx.x];
    counts[e] = m;
    mean_score[e] = v * inv_t;
  }
}

// With s the scores, p = softmax, u_j = s_j / sum of the picked, g_j = dL/dw_j:
//   normalize:     dl at pick j  += scale u_j (g_j - sum_m u_m g_m) [sigmoid: x (1 - s_j)]
//   else softmax:  dl_i          += s_i (a_i - sum s a), a = scale g at the picks
//   else sigmoid:  dl at pick j  += scale g_j s_j (1 - s_j)
//   mean score b / T, softmax:  s_i (b_i - sum s b) / T;   sigmoid: b_i s_i (1 - s_i) / T
//   lse:           p_i dlse
// u comes from the picked logits alone, so that it holds where s underflows.
template <class LT, int V>
__global__ void __launch_bounds__(32 * kRouteWarps) route_bwd_kernel(const RouteBwdArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long step = static_cast<long long>(gridDim.x) * kRouteWarps;
  const bool dense_softmax = !a.sigmoid && (!a.normalize || a.d_mean_score);
  const float inv_t = 1.f / static_cast<float>(a.T);
  for (long long t = static_cast<long long>(blockIdx.x) * kRouteWarps + warp; t < a.T; t += step) {
    const LT* row = static_cast<const LT*>(a.logits) + t * a.E;
    float d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = 0.f;
    // the picks: lane j's j-th and (j + 32)-th
    int id[2];
    float l[2], g[2], c[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = lane + 32 * h;
      const long long e = j < a.k ? __ldg(a.experts + t * a.k + j) : -1;
      const bool in = e >= 0 && e < a.E;   // an id outside is no expert's
      id[h] = in ? static_cast<int>(e) : -1;
      l[h] = in ? logit_at(row, e) : -INFINITY;
      g[h] = in ? __ldg(a.d_weights + t * a.k + j) * a.scale : 0.f;
    }
    float x[V], p[V], top = 0.f, inv = 0.f;
    if (dense_softmax || a.d_lse || (a.sigmoid && a.d_mean_score)) load_logits<LT, V>(row, a.E, lane, x);
    if (dense_softmax || a.d_lse) {
      const float total = exps<V>(x, p, top);
      inv = total > 0.f || total != total ? 1.f / total : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] *= inv;
    }
    float q = 0.f;   // sum of s x (the gradients that reach the scores)
    if (a.normalize) {
      float u[2], first = 0.f;
      if (!a.sigmoid) {
        first = warp_max(fmaxf(l[0], l[1]));
        if (first == -INFINITY) first = 0.f;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) u[h] = id[h] < 0 ? 0.f : a.sigmoid ? sigmoid(l[h]) : expf(l[h] - first);
      const float sum = warp_sum(u[0] + u[1]);
      const float by = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
      u[0] *= by, u[1] *= by;
      const float mean = warp_sum(u[0] * g[0] + u[1] * g[1]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        c[h] = u[h] * (g[h] - mean);
        if (a.sigmoid) c[h] *= sigmoid(-l[h]);
      }
    } else if (a.sigmoid) {
#pragma unroll
      for (int h = 0; h < 2; ++h) c[h] = id[h] < 0 ? 0.f : g[h] * sigmoid(l[h]) * sigmoid(-l[h]);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) c[h] = id[h] < 0 ? 0.f : g[h] * (expf(l[h] - top) * inv);
      q = warp_sum(c[0] + c[1]);
    }
    // to the lanes that hold the picks' logits, one after the other
    for (int j = 0; j < a.k; ++j) {
      const int e = __shfl_sync(kAll, j < 32 ? id[0] : id[1], j & 31);
      const float v = __shfl_sync(kAll, j < 32 ? c[0] : c[1], j & 31);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e == lane * V + i) d[i] += v;
    }
    float b[V];
    if (a.d_mean_score) {
#pragma unroll
      for (int i = 0; i < V; ++i) b[i] = lane * V + i < a.E ? __ldg(a.d_mean_score + lane * V + i) * inv_t : 0.f;
      if (!a.sigmoid) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) m += p[i] * b[i];
        q += warp_sum(m);
      }
    }
    const float dl = a.d_lse ? __ldg(a.d_lse + t) : 0.f;
    if (dense_softmax) {
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] += p[i] * ((a.d_mean_score ? b[i] : 0.f) - q);
    }
    if (a.sigmoid && a.d_mean_score) {
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] += b[i] * sigmoid(x[i]) * sigmoid(-x[i]);
    }
    if (a.d_lse) {
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] += p[i] * dl;
    }
    LT* out = static_cast<LT*>(a.d_logits) + t * a.E + lane * V;
    constexpr int kVec = sizeof(LT) == 4 ? (V < 4 ? V : 4) : (V < 8 ? V : 8);
    const int left = a.E - lane * V;
    if (kVec > 1 && a.E % kVec == 0) {
#pragma unroll
      for (int i = 0; i < V; i += kVec) {
        if (i >= left) continue;
        if constexpr (sizeof(LT) == 4) {
          if constexpr (kVec == 4)
            *reinterpret_cast<float4*>(out + i) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
          else if constexpr (kVec == 2)
            *reinterpret_cast<float2*>(out + i) = make_float2(d[i], d[i + 1]);
        } else if constexpr (kVec == 8) {
          *reinterpret_cast<uint4*>(out + i) = make_uint4(pack_bf16(d[i], d[i + 1]), pack_bf16(d[i + 2], d[i + 3]),
                                                          pack_bf16(d[i + 4], d[i + 5]), pack_bf16(d[i + 6], d[i + 7]));
        } else if constexpr (kVec == 4) {
          *reinterpret_cast<uint2*>(out + i) = make_uint2(pack_bf16(d[i], d[i + 1]), pack_bf16(d[i + 2], d[i + 3]));
        } else if constexpr (kVec == 2) {
          *reinterpret_cast<uint32_t*>(out + i) = pack_bf16(d[i], d[i + 1]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (i >= left) continue;
        if constexpr (sizeof(LT) == 4)
          out[i] = d[i];
        else
          out[i] = static_cast<uint16_t>(pack_bf16(d[i], 0.f) & 0xffffu);
      }
    }
  }
}

int route_grid(long long T) {
  const long long want = (T + kRouteWarps - 1) / kRouteWarps;
  return static_cast<int>(want < 608 ? want : 608);
}

template <class LT>
cudaError_t route_typed(const RouteArgs& a, int grid, size_t smem, cudaStream_t st) {
  const dim3 g(grid), b(32 * kRouteWarps);
  if (a.E <= 32) return launch_dependent(route_kernel<LT, 1>, g, b, smem, st, a);
  if (a.E <= 64) return launch_dependent(route_kernel<LT, 2>, g, b, smem, st, a);
  if (a.E <= 128) return launch_dependent(route_kernel<LT, 4>, g, b, smem, st, a);
  if (a.E <= 256) return launch_dependent(route_kernel<LT, 8>, g, b, smem, st, a);
  if (a.E <= 512) return launch_dependent(route_kernel<LT, 16>, g, b, smem, st, a);
  return launch_dependent(route_kernel<LT, 32>, g, b, smem, st, a);
}

template <class LT>
cudaError_t route_bwd_typed(const RouteBwdArgs& a, cudaStream_t st) {
  const dim3 g(route_grid(a.T) < 608 ? route_grid(a.T) : 1216), b(32 * kRouteWarps);
  if (a.E <= 32) return launch_dependent(route_bwd_kernel<LT, 1>, g, b, 0, st, a);
  if (a.E <= 64) return launch_dependent(route_bwd_kernel<LT, 2>, g, b, 0, st, a);
  if (a.E <= 128) return launch_dependent(route_bwd_kernel<LT, 4>, g, b, 0, st, a);
  if (a.E <= 256) return launch_dependent(route_bwd_kernel<LT, 8>, g, b, 0, st, a);
  if (a.E <= 512) return launch_dependent(route_bwd_kernel<LT, 16>, g, b, 0, st, a);
  return launch_dependent(route_bwd_kernel<LT, 32>, g, b, 0, st, a);
}

}  // namespace

int route_blocks(long long T) { return route_grid(T); }

cudaError_t launch_route(const RouteArgs& a, int f32, cudaStream_t st) {
  const int grid = route_grid(a.T);
  const size_t smem = a.counts ? static_cast<size_t>(1 + kRouteWarps) * a.E * sizeof(float) : 0;   // at most 36 KB
  const cudaError_t err = grid == 0 ? cudaSuccess : f32 ? route_typed<float>(a, grid, smem, st) : route_typed<uint16_t>(a, grid, smem, st);
  if (err != cudaSuccess || !a.counts) return err;
  return launch_dependent(route_join_kernel, dim3((a.E + 31) / 32), dim3(32, 32), 0, st, static_cast<const float*>(a.part), grid,
                          a.E, a.T > 0 ? 1.f / static_cast<float>(a.T) : 0.f, a.counts, a.mean_score);
}

cudaError_t launch_route_bwd(const RouteBwdArgs& a, int f32, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  return f32 ? route_bwd_typed<float>(a, st) : route_bwd_typed<uint16_t>(a, st);
}

}  // namespace mok
