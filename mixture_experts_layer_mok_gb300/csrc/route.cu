// The router: each token's k experts and their weights from its logits, what
// the balance and z losses need, and the gradient of the logits.
//
// G lanes to a token, 32 / G tokens to a warp at a time; lane l of a token holds
// the V consecutive logits from l V on, so that the lowest lane of several with the
// same largest value holds the lowest index.  Fewer lanes to a token of up to 64
// experts, because a token's cost is in its reductions.
//
// The choice.  A whole warp to a token: the k-th largest of the lanes' largest
// bounds the choice from below; the few logits that reach it (about k + 4 of 256
// for k = 8) are put side by side, one to a lane, and ranked by comparing each
// with all.  Where more than 32 reach it (ties, or k above 32), and for part of a
// warp, the largest are taken one after the other: each lane keeps the largest of
// what is left of its own, and only the lane that held the last one looks for its
// next.
//
// Per token of 256 experts a warp issues 476 instructions (355 of them for k = 1
// without loads), most of which wait for the ones before: issue slots 64% busy, DRAM
// 22%, 48% of the warps that fit.  65536 tokens with loads and mean scores take 36 us:
// 41 with tokens handed out round by round, whose last round was a third full, with
// a logit to an instruction in the sums, and without the next token's logits on
// their way during a choice.  With a bias, by exact scores: 53.
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

// Warps of a block, at most: fewer where a lane holds more.
template <int V>
constexpr int kRouteWarps = V > 8 ? 8 : 16;
constexpr int kSumRows = 4;   // warps' sums of scores that a block keeps at a time
constexpr unsigned kAll = 0xffffffffu;

// Unsigned integers in the order of the values: -0 as 0, NaN (which the addition
// makes 0x7fffffff) above all, and above 0, which stands for nothing.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ (static_cast<uint32_t>(static_cast<int>(~k) >> 31) | 0x80000000u));
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

// Over a token's G lanes.
template <int G>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = G / 2; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if constexpr (G == 32) return __reduce_max_sync(kAll, v);
#pragma unroll
  for (int o = G / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int G>
__device__ __forceinline__ float lanes_max(float v) {
  return key_value(lanes_max<G>(order_key(v)));
}

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

// Two sums, or two products, in one instruction.
__device__ __forceinline__ void add_pair(float& a0, float& a1, float b0, float b1) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}
__device__ __forceinline__ void mul_pair(float& a0, float& a1, float b) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(b));
}

// e[i] = exp(x[i] - top), good to 2^-21 or so; returns the sum of e over the token.
template <int G, int V>
__device__ __forceinline__ float exps(const float (&x)[V], float (&e)[V], float top) {
  float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    float d0 = x[i], d1 = x[i + 1];
    add_pair(d0, d1, -top, -top);
    mul_pair(d0, d1, kLog2e);
    e[i] = fast_exp2(d0), e[i + 1] = fast_exp2(d1);
    add_pair(sum0, sum1, e[i], e[i + 1]);
  }
  return lanes_sum<G>(sum0 + sum1);
}
// s[i] = 1 / (1 + exp(-x[i])), good to 2^-21 or so.
template <int V>
__device__ __forceinline__ void logistics(const float (&x)[V], float (&s)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    float d0 = x[i], d1 = x[i + 1];
    mul_pair(d0, d1, -kLog2e);
    d0 = fast_exp2(d0), d1 = fast_exp2(d1);
    add_pair(d0, d1, 1.f, 1.f);
    s[i] = fast_rcp(d0), s[i + 1] = fast_rcp(d1);
  }
}
template <int V>
__device__ __forceinline__ uint32_t largest(const uint32_t (&key)[V]) {
  uint32_t m = key[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = max(m, key[i]);
  return m;
}

// Picks that each of a token's P lanes holds (the j-th is slot j / P of lane j %
// P): one where there are no more than lanes, which keeps the code short, else as
// many as there can be.
template <int P, int G, int V, bool MANY>
constexpr int kSlots = MANY ? (G * V < MOK_ROUTE_MAX_K ? G * V : MOK_ROUTE_MAX_K) / P : 1;

struct Pick {
  int id;
  uint32_t key;
};
// A warp's scratch in shared memory, for a round of 32 / P tokens.
template <int P, int V, int G>
struct RouteScratch {
  static constexpr int kTokens = 32 / P;
  Pick picks[kTokens][G * V < MOK_ROUTE_MAX_K ? G * V : MOK_ROUTE_MAX_K];
  float top[kTokens], total[kTokens];
  uint4 keys[G == 32 ? 9 : 1];   // of what reaches the bound, if no more than 32 do, with zeros behind
  int index[G == 32 ? 32 : 1];
  int found;
};

// The order of logit i of a row; 0, below all others, behind the last.
template <class LT>
__device__ __forceinline__ uint32_t logit_key(const LT* row, int E, int i) {
  return i < E ? order_key(logit_at(row, i)) : 0u;
}

// The k largest keys of a token, largest first, into its picks; most: the lane's
// largest, first: the token's.  BIAS: of equal keys the one of the largest logit
// comes first (scores that 32 bits do not tell apart, beside equal biases: as
// without a bias); then, and without BIAS at once, the one of the lowest index.
template <int G, int V, bool BIAS, class LT, class Scratch>
__device__ __forceinline__ void choose(uint32_t (&key)[V], uint32_t most, uint32_t first, int k, int lane, Scratch& scratch, Pick* picks,
                                       const LT* row, int E) {
  const int l = lane % G;
  if (G == 32 && k <= 32) {
    uint32_t* const keys = reinterpret_cast<uint32_t*>(scratch.keys);
    if (lane == 0) scratch.found = 0;
    uint32_t left = most == first ? 0 : most, least = first;
#pragma unroll 2
    for (int j = 1; j < k; ++j) {   // (equal ones go at one time: the bound is then lower than it need be)
      least = lanes_max<G>(left);
      if (left == least) left = 0;
    }
    uint32_t in = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) in |= key[i] >= least ? 1u << i : 0u;
    __syncwarp();
    int at = 0;
    if (in) at = atomicAdd(&scratch.found, __popc(in));   // in any order: the ranks below do not depend on it
    __syncwarp();
    const int all = scratch.found;
    if (all <= 32) {
      if (in) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if ((in >> i) & 1u) keys[at] = key[i], scratch.index[at] = lane * V + i, ++at;
      }
      if (lane < 4) keys[all + lane] = 0;
      __syncwarp();
      const uint32_t me = keys[lane];
      int rank = 0;
      for (int j = 0; j < all; j += 4) {
        const uint4 v = scratch.keys[j / 4];
        rank += (v.x > me ? 1 : 0) + (v.y > me ? 1 : 0) + (v.z > me ? 1 : 0) + (v.w > me ? 1 : 0);
      }
      if (lane >= all) rank = 0;
      const int index = lane < all ? scratch.index[lane] : 0;
      const bool equal = __reduce_add_sync(kAll, rank) != all * (all - 1) / 2;
      if constexpr (BIAS) {
        if (equal) {
          const uint32_t mine = lane < all ? logit_key(row, E, index) : 0u;
          for (int j = 0; j < all; ++j) {
            const uint32_t its = __shfl_sync(kAll, mine, j);
            if (lane < all && keys[j] == me) rank += its > mine || (its == mine && scratch.index[j] < index) ? 1 : 0;
          }
        }
      } else if (equal && lane < all) {
        for (int j = 0; j < all; ++j) rank += keys[j] == me && scratch.index[j] < index ? 1 : 0;
      }
      if (lane < all && rank < k) picks[rank] = Pick{index, me};
      __syncwarp();
      return;
    }
  }
  bool ties = false;
  for (int j = 0; j < k; ++j) {
    const uint32_t best = lanes_max<G>(most);
    const unsigned hit = (__ballot_sync(kAll, most == best) >> (lane - l)) & (kAll >> (32 - G));
    if (BIAS) ties |= (hit & (hit - 1)) != 0;
    if (l == __ffs(hit) - 1) {
      most = 0;
      bool found = false;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool it = !found && key[i] == best;
        if (it) picks[j] = Pick{l * V + i, best}, key[i] = 0;
        found = found || it;
        most = max(most, key[i]);
      }
      if (BIAS) ties |= most == best;
    }
  }
  __syncwarp();
  if (!BIAS || !__any_sync(kAll, ties)) return;
  // equal keys: once more, by logit among them
  for (int j = 0; j < k; ++j) {
    const Pick pick = picks[j];
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (l * V + i == pick.id) key[i] = pick.key;
  }
  __syncwarp();
  for (int j = 0; j < k; ++j) {
    most = largest(key);
    const uint32_t best = lanes_max<G>(most);
    uint32_t top = 0;
    int slot = -1;
    if (most == best) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t its = key[i] == best ? logit_key(row, E, l * V + i) : 0u;
        if (its > top) top = its, slot = i;
      }
    }
    const uint32_t over = lanes_max<G>(top);
    const unsigned hit = (__ballot_sync(kAll, slot >= 0 && top == over) >> (lane - l)) & (kAll >> (32 - G));
    if (l == __ffs(hit) - 1) {
      picks[j] = Pick{l * V + slot, best};
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == slot) key[i] = 0;
    }
  }
  __syncwarp();
}

// A round of a warp is 32 / P tokens: first G lanes to each in G / P passes, which
// leave the picks and the sums in shared memory, then P lanes to each, which make
// the weights of all of them at a time.  BIAS: the choice is by score + bias, in
// kernels of their own, as exact scores take registers.
template <class LT, int G, int V, int P, bool MANY, bool BIAS>
__global__ void __launch_bounds__(32 * kRouteWarps<V>, V <= 8 ? 2 : 0) route_kernel(const RouteArgs a) {
  constexpr int S = kSlots<P, G, V, MANY>;
  using Scratch = RouteScratch<P, V, G>;
  extern __shared__ float shared[];   // with counts: [E] counts, then [kSumRows][E] sums of scores
  __shared__ __align__(16) Scratch scratches[kRouteWarps<V>];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, lane = threadIdx.x & 31, l = lane % G;
  Scratch& scratch = scratches[warp];
  const bool balance = a.counts != nullptr;
  int* cnt = reinterpret_cast<int*>(shared);
  if (balance) {
    for (int i = threadIdx.x; i < a.E; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
  }
  float mean[V];
#pragma unroll
  for (int i = 0; i < V; ++i) mean[i] = 0.f;
  // this warp's tokens, one after the other: as many passes' as any other warp's, or one pass's more
  const unsigned passes = static_cast<unsigned>((a.T + 32 / G - 1) / (32 / G)), all_warps = gridDim.x * warps,
                 mine = blockIdx.x * warps + warp, each = passes / all_warps, more = passes - each * all_warps;
  const long long begin = static_cast<long long>(each * mine + min(mine, more)) * (32 / G);
  const long long end = min(a.T, begin + static_cast<long long>(each + (mine < more ? 1 : 0)) * (32 / G));
  const LT* const logits = static_cast<const LT*>(a.logits);
  float x[V];   // the next token's are on their way while the choice of the last one is made
  if (begin < end) load_logits<LT, V>(logits + min(begin + lane / G, end - 1) * a.E, a.E, l, x);   // (behind the last token: that one again)
  for (long long t0 = begin; t0 < end; t0 += 32 / P) {
#pragma unroll 1
    for (int pass = 0; pass < G / P && t0 + pass * (32 / G) < end; ++pass) {
      const int at = pass * (32 / G) + lane / G;   // the token's place in the round
      const bool live = t0 + at < end;
      float s[V];
      // the choice: by the logits, in whose order the scores are, or by score + bias; what lies behind the last expert is -inf
      // and behind everything
      uint32_t key[V];
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = order_key(x[i]);
      uint32_t most = largest(key), first = lanes_max<G>(most);
      float top = key_value(first);
      if (top == -INFINITY) top = 0.f;   // exp(x - 0) is 0 for all
      float total;
      if (BIAS && !a.sigmoid) {   // a choice is by the exact scores
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = expf(x[i] - top), sum += s[i];
        total = lanes_sum<G>(sum);
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = total == 0.f ? 0.f : s[i] / total;
      } else {
        total = exps<G, V>(x, s, top);
      }
      if (l == 0) scratch.top[at] = top, scratch.total[at] = total;
      if (a.sigmoid) {
        if (BIAS) {   // likewise
#pragma unroll
          for (int i = 0; i < V; ++i) s[i] = sigmoid(x[i]);
        } else if (balance) {
          logistics(x, s);
        }
      } else if (balance && !BIAS) {
        const float inv = total > 0.f || total != total ? 1.f / total : 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] *= inv;
      }
      if (balance && live) {
#pragma unroll
        for (int i = 0; i < V; i += 2) add_pair(mean[i], mean[i + 1], s[i], s[i + 1]);
      }
      if (BIAS) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = l * V + i;
          if (e < a.E && x[i] != -INFINITY) key[i] = order_key(s[i] + __ldg(a.bias + e));
        }
        most = largest(key), first = lanes_max<G>(most);
      }
      load_logits<LT, V>(logits + min(t0 + at + 32 / G, end - 1) * a.E, a.E, l, x);
      choose<G, V, BIAS>(key, most, first, a.k, lane, scratch, scratch.picks[at], logits + min(t0 + at, end - 1) * a.E, a.E);
    }
    __syncwarp();
    const int p = lane % P, at = lane / P;
    const long long t = t0 + at;
    const bool live = t < end;
    const float top = live ? scratch.top[at] : 0.f, total = live ? scratch.total[at] : 1.f;
    if (p == 0 && live) a.lse[t] = top == INFINITY ? top : top + logf(total);
    const float inv = total > 0.f || total != total ? 1.f / total : 0.f;
    int id[S];
    float w[S], logit[S], sum = 0.f, first = -INFINITY;
#pragma unroll
    for (int h = 0; h < S; ++h) {
      id[h] = -1, logit[h] = -INFINITY;
      if (P * h >= a.k) continue;
      if (p + P * h < a.k && live) {
        const Pick pick = scratch.picks[at][p + P * h];
        id[h] = pick.id;
        logit[h] = BIAS ? logit_at(static_cast<const LT*>(a.logits) + t * a.E, pick.id) : key_value(pick.key);
        first = fmaxf(first, logit[h]);
      }
    }
    __syncwarp();   // the scratch has been read
    if (!a.sigmoid && a.normalize) {   // from the largest of the picked, whatever the others sum to
      first = lanes_max<P>(first);
      if (first == -INFINITY) first = 0.f;
    }
#pragma unroll
    for (int h = 0; h < S; ++h) {
      w[h] = 0.f;
      if (P * h >= a.k) continue;
      if (a.sigmoid)
        w[h] = sigmoid(logit[h]);   // (0 where there is no pick)
      else
        w[h] = a.normalize ? expf(logit[h] - first) : expf(logit[h] - top) * inv;
      sum += w[h];
    }
    float by = 1.f;
    if (a.normalize) {
      sum = lanes_sum<P>(sum);
      by = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
    }
#pragma unroll
    for (int h = 0; h < S; ++h) {
      const int j = p + P * h;
      if (P * h >= a.k) continue;
      if (j < a.k && live) {
        a.experts[t * a.k + j] = id[h];
        a.weights[t * a.k + j] = w[h] * by * a.scale;
        if (balance) atomicAdd(cnt + id[h], 1);   // whole numbers: any order
      }
    }
  }
  if (!balance) return;
#pragma unroll
  for (int o = G; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < V; ++i) mean[i] += __shfl_xor_sync(kAll, mean[i], o);
  float* sums = shared + a.E;
#pragma unroll
  for (int w0 = kRouteWarps<V> - kSumRows; w0 >= 0; w0 -= kSumRows) {   // the last warps' first
    if (warp >= w0 && warp < w0 + kSumRows && lane < G) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = l * V + i;
        if (e < a.E) sums[(warp - w0) * a.E + e] = mean[i] + (warp + kSumRows < warps ? sums[(warp - w0) * a.E + e] : 0.f);
      }
    }
    __syncthreads();
  }
  int* part_cnt = reinterpret_cast<int*>(a.part + static_cast<long long>(gridDim.x) * a.E);
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    float v = 0.f;
    for (int w = 0; w < min(warps, kSumRows); ++w) v += sums[w * a.E + e];
    a.part[static_cast<long long>(blockIdx.x) * a.E + e] = v;
    part_cnt[static_cast<long long>(blockIdx.x) * a.E + e] = cnt[e];
  }
}

// The blocks' parts joined in a fixed order: 8 experts a block, 64 parts in step,
// so that few loads of a thread follow one another.
constexpr int kJoinThreads = 512;
__global__ void __launch_bounds__(kJoinThreads) route_join_kernel(const float* __restrict__ part, int n, int E, float inv_t,
                                                                  int* __restrict__ counts, float* __restrict__ mean_score) {
  constexpr int kWarps = kJoinThreads / 32;
  __shared__ float s[kWarps][8];
  __shared__ int c[kWarps][8];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, e = blockIdx.x * 8 + (lane & 7);
  float v = 0.f;
  int m = 0;
  if (e < E) {
    const int* part_cnt = reinterpret_cast<const int*>(part + static_cast<long long>(n) * E);
#pragma unroll 5
    for (int b = threadIdx.x >> 3; b < n; b += kJoinThreads / 8) {
      v += part[static_cast<long long>(b) * E + e];
      m += part_cnt[static_cast<long long>(b) * E + e];
    }
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) v += __shfl_xor_sync(kAll, v, o), m += __shfl_xor_sync(kAll, m, o);
  if (lane < 8) s[threadIdx.x >> 5][lane] = v, c[threadIdx.x >> 5][lane] = m;
  __syncthreads();
  if (threadIdx.x < 8 && e < E) {
    v = 0.f, m = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += s[i][threadIdx.x], m += c[i][threadIdx.x];
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
template <class LT, int G, int V, bool MANY>
__global__ void __launch_bounds__(32 * kRouteWarps<V>) route_bwd_kernel(const RouteBwdArgs a) {
  constexpr int S = kSlots<G, G, V, MANY>;
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, lane = threadIdx.x & 31, l = lane % G;
  const long long step = static_cast<long long>(gridDim.x) * warps * (32 / G);
  const bool dense_softmax = !a.sigmoid && (!a.normalize || a.d_mean_score);
  const float inv_t = 1.f / static_cast<float>(a.T);
  for (long long t0 = (static_cast<long long>(blockIdx.x) * warps + warp) * (32 / G); t0 < a.T; t0 += step) {
    const long long t = min(t0 + lane / G, a.T - 1);   // (behind the last token: that one again, not stored)
    const LT* row = static_cast<const LT*>(a.logits) + t * a.E;
    float d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = 0.f;
    int id[S];
    float lg[S], g[S], c[S];
#pragma unroll
    for (int h = 0; h < S; ++h) {
      const int j = l + G * h;
      const long long e = j < a.k ? __ldg(a.experts + t * a.k + j) : -1;
      const bool in = e >= 0 && e < a.E;   // an id outside is no expert's
      id[h] = in ? static_cast<int>(e) : -1;
      lg[h] = in ? logit_at(row, e) : -INFINITY;
      g[h] = in ? __ldg(a.d_weights + t * a.k + j) * a.scale : 0.f;
      c[h] = 0.f;
    }
    float x[V], p[V], top = 0.f, inv = 0.f;
    if (dense_softmax || a.d_lse || (a.sigmoid && a.d_mean_score)) load_logits<LT, V>(row, a.E, l, x);
    if (dense_softmax || a.d_lse) {
      float m = x[0];
#pragma unroll
      for (int i = 1; i < V; ++i) m = fmaxf(m, x[i]);
      m = lanes_max<G>(m);
      top = m == -INFINITY ? 0.f : m;
      const float total = exps<G, V>(x, p, top);
      inv = total > 0.f || total != total ? 1.f / total : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] *= inv;
    }
    float q = 0.f;   // sum of s x (the gradients that reach the scores)
    if (a.normalize) {
      float first = 0.f, sum = 0.f, mean = 0.f;
      if (!a.sigmoid) {
        first = -INFINITY;
#pragma unroll
        for (int h = 0; h < S; ++h) first = fmaxf(first, lg[h]);
        first = lanes_max<G>(first);
        if (first == -INFINITY) first = 0.f;
      }
#pragma unroll
      for (int h = 0; h < S; ++h) {
        if (G * h >= a.k) break;
        c[h] = id[h] < 0 ? 0.f : a.sigmoid ? sigmoid(lg[h]) : expf(lg[h] - first);
        sum += c[h];
      }
      sum = lanes_sum<G>(sum);
      const float by = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
#pragma unroll
      for (int h = 0; h < S; ++h) c[h] *= by, mean += c[h] * g[h];
      mean = lanes_sum<G>(mean);
#pragma unroll
      for (int h = 0; h < S; ++h) {
        if (G * h >= a.k) break;
        c[h] *= g[h] - mean;
        if (a.sigmoid) c[h] *= sigmoid(-lg[h]);
      }
    } else {
#pragma unroll
      for (int h = 0; h < S; ++h) {
        if (G * h >= a.k) break;
        if (id[h] < 0) continue;
        c[h] = a.sigmoid ? g[h] * sigmoid(lg[h]) * sigmoid(-lg[h]) : g[h] * (expf(lg[h] - top) * inv);
        q += c[h];
      }
      q = a.sigmoid ? 0.f : lanes_sum<G>(q);
    }
    // to the lanes that hold the picks' logits, one after the other
#pragma unroll
    for (int h = 0; h < S; ++h) {
#pragma unroll 4
      for (int j = 0; j < G && G * h + j < a.k; ++j) {
        const int e = __shfl_sync(kAll, id[h], j, G) - l * V;
        const float v = __shfl_sync(kAll, c[h], j, G);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (e == i) d[i] += v;
      }
    }
    float b[V];
    if (a.d_mean_score) {
#pragma unroll
      for (int i = 0; i < V; ++i) b[i] = l * V + i < a.E ? __ldg(a.d_mean_score + l * V + i) * inv_t : 0.f;
      if (!a.sigmoid) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) m += p[i] * b[i];
        q += lanes_sum<G>(m);
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
    if (t0 + lane / G >= a.T) continue;
    LT* out = static_cast<LT*>(a.d_logits) + t * a.E + l * V;
    constexpr int kVec = sizeof(LT) == 4 ? (V < 4 ? V : 4) : (V < 8 ? V : 8);
    const int left = a.E - l * V;
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

// Lanes that make a token's weights, warps to a block, and blocks.  A token to a
// round where that gives no SM more than 16 warps (1024 tokens among 256 experts
// 6.0 us with four), fewer warps to a block where that spreads few rounds over
// more SMs; at most 32 warps to each of 152 SMs.
struct RouteGrid {
  bool alone;   // a token to a round (of more than 64 experts)
  int warps, blocks;
};
RouteGrid route_grid(long long T, int E) {
  const bool alone = E > 64 && T <= 16 * 152;
  const int each = alone ? 1 : E <= 32 ? 8 : 4;   // tokens of a round
  const long long all = (T + each - 1) / each;
  const int warps = all <= 4 * 152 ? 1 : all <= 16 * 152 ? 4 : E <= 256 ? kRouteWarps<8> : kRouteWarps<16>;
  const long long want = (all + warps - 1) / warps;
  const long long most = 32 / warps * 152;
  return {alone, warps, static_cast<int>(want < most ? want : most)};
}

template <class LT, int G, int V, int P>
cudaError_t route_picks(const RouteArgs& a, RouteGrid r, size_t smem, cudaStream_t st) {
  const dim3 g(r.blocks), b(32 * r.warps);
  const auto launch = [&](auto kern) { return launch_dependent(kern, g, b, smem, st, a); };
  if (a.bias) return a.k <= P ? launch(route_kernel<LT, G, V, P, false, true>) : launch(route_kernel<LT, G, V, P, true, true>);
  return a.k <= P ? launch(route_kernel<LT, G, V, P, false, false>) : launch(route_kernel<LT, G, V, P, true, false>);
}
template <class LT, int G, int V>
cudaError_t route_lanes(const RouteArgs& a, RouteGrid r, size_t smem, cudaStream_t st) {
  if constexpr (G == 32)
    if (r.alone) return route_picks<LT, G, V, 32>(a, r, smem, st);
  return route_picks<LT, G, V, (G < 8 ? G : 8)>(a, r, smem, st);
}
template <class LT>
cudaError_t route_typed(const RouteArgs& a, RouteGrid r, size_t smem, cudaStream_t st) {
  if (a.E <= 32) return route_lanes<LT, 4, 8>(a, r, smem, st);
  if (a.E <= 64) return route_lanes<LT, 8, 8>(a, r, smem, st);
  if (a.E <= 128) return route_lanes<LT, 32, 4>(a, r, smem, st);   // (16 lanes and 8 logits each, largest by largest, took 14 us for 16384 tokens)
  if (a.E <= 256) return route_lanes<LT, 32, 8>(a, r, smem, st);
  if (a.E <= 512) return route_lanes<LT, 32, 16>(a, r, smem, st);
  return route_lanes<LT, 32, 32>(a, r, smem, st);
}

template <class LT, int G, int V>
cudaError_t route_bwd_lanes(const RouteBwdArgs& a, cudaStream_t st) {
  // four warps to a block: a warp has few tokens, and small blocks spread and end evenly
  const long long warps = (a.T + 32 / G - 1) / (32 / G), blocks = (warps + 3) / 4;
  const dim3 g(static_cast<unsigned>(blocks < 8 * 152 ? blocks : 8 * 152)), b(128);
  return a.k <= G ? launch_dependent(route_bwd_kernel<LT, G, V, false>, g, b, 0, st, a)
                  : launch_dependent(route_bwd_kernel<LT, G, V, true>, g, b, 0, st, a);
}
template <class LT>
cudaError_t route_bwd_typed(const RouteBwdArgs& a, cudaStream_t st) {
  if (a.E <= 32) return route_bwd_lanes<LT, 4, 8>(a, st);
  if (a.E <= 64) return route_bwd_lanes<LT, 8, 8>(a, st);
  if (a.E <= 128) return route_bwd_lanes<LT, 16, 8>(a, st);
  if (a.E <= 256) return route_bwd_lanes<LT, 32, 8>(a, st);
  if (a.E <= 512) return route_bwd_lanes<LT, 32, 16>(a, st);
  return route_bwd_lanes<LT, 32, 32>(a, st);
}

}  // namespace

int route_blocks(long long T, int E) { return route_grid(T, E).blocks; }

cudaError_t launch_route(const RouteArgs& a, int f32, cudaStream_t st) {
  const RouteGrid r = route_grid(a.T, a.E);
  const size_t smem = a.counts ? static_cast<size_t>(1 + kSumRows) * a.E * sizeof(float) : 0;   // at most 20 KB
  const cudaError_t err = r.blocks == 0 ? cudaSuccess : f32 ? route_typed<float>(a, r, smem, st) : route_typed<uint16_t>(a, r, smem, st);
  if (err != cudaSuccess || !a.counts) return err;
  return launch_dependent(route_join_kernel, dim3((a.E + 7) / 8), dim3(kJoinThreads), 0, st, static_cast<const float*>(a.part), r.blocks,
                          a.E, a.T > 0 ? 1.f / static_cast<float>(a.T) : 0.f, a.counts, a.mean_score);
}

cudaError_t launch_route_bwd(const RouteBwdArgs& a, int f32, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  return f32 ? route_bwd_typed<float>(a, st) : route_bwd_typed<uint16_t>(a, st);
}

}  // namespace mok
