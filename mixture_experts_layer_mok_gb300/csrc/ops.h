// Internal launch interface of the operators around the layer: the norm, the
// dense projection and the optimiser step.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mok.h"

namespace mok {

// One special-function instruction each (subnormals flushed): 2^x and 1/x,
// good to about 2^-22.
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The value 2^(s - 127) of an E8M0 scale (255: NaN).
__device__ __forceinline__ float e8m0_value(uint32_t s) {
  return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7FC00000u : s << 23);
}

// The values of the four E4M3 codes in a word, lowest byte first.
__device__ __forceinline__ void e4m3x4_values(uint32_t w, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * i)), __NV_E4M3);
    const float2 v = __half22float2(__half2(h));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

// ---------------------------------------------------------------- norm
struct NormArgs {
  const void* x;
  const void* residual;
  const void* weight;
  void* h;          // x + residual in the residual's type (with a residual)
  uint16_t* y;      // bf16 output or NULL
  uint8_t* codes;   // MXFP8 output or NULL
  uint8_t* scales;
  float* rstd;
  long long rows;
  int H;
  int weight_f32;
  float eps;
};
struct NormBwdArgs {
  const uint16_t* dy;
  const void* h;
  const void* weight;
  const float* rstd;
  const void* dh;     // gradient of h from its other uses, or NULL
  void* dx;           // in h's type
  void* dx_other;     // the same unrounded values in the other type, or NULL
  float* part;        // [norm_bwd_walkers][H]
  long long rows;
  int H;
  int weight_f32;
};
// Partial rows of the weight gradient (part of the workspace's size).
int norm_bwd_walkers(long long rows, int H, bool f32);
// residual: 0 none, 1 bf16, 2 fp32.
cudaError_t launch_rms_norm(const NormArgs& a, int x_f32, int residual, cudaStream_t st);
cudaError_t launch_rms_norm_bwd(const NormBwdArgs& a, int h_f32, float* d_weight, cudaStream_t st);
// out[j] = sum over n rows of part[.][j], in a fixed order (n = 0: zeros).
// late: the last kernel launched on the stream neither writes part nor started
// before part was complete.
cudaError_t launch_column_sum(const float* part, int n, int H, float* out, bool late, cudaStream_t st);
cudaError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, long long n, uint16_t* out, cudaStream_t st);

// ---------------------------------------------------------------- dense projection
enum LinAct : int { LIN_NONE = 0, LIN_RELU = 1, LIN_SILU = 2, LIN_GELU = 3, LIN_GELU_TANH = 4 };

struct LinearParams {
  long long L;      // the output's contiguous length
  int C;            // the output's rows
  int nk;           // K-blocks of 64
  int split;        // split kernel: CTAs of a cluster along K
  int l_tiles;      // pair kernel: 256-wide tiles, and the order's group
  int c_tiles;
  int group;
  int act;          // forward epilogue
  int out_f32;
  int bias_f32;
  int residual_f32;
  const void* bias;      // [L] or NULL
  const void* residual;  // [C][L] or NULL
  void* out;             // [C][L]
  uint16_t* z;           // [C][L] bf16 pre-activations, or NULL
  int* status;           // device word: MOK_ERR_TIMEOUT once a bounded wait gave up
};
// One of the products described in linear.cuh.  a: [L][K], or [K][L] with
// a_mn; b: [C][K], or [K][C] with b_mn; bf16, contiguous.
struct LinearOperands {
  const uint16_t* a;
  const uint16_t* b;
  long long K;
};
// The device word that a bounded wait which gave up sets (current device).
cudaError_t linear_status_word(int** word);
// The last three name kernels only: dx and dW together, the forward over few
// K-blocks, and the forward over many of them into fp32.
enum LinKind : int { LIN_FWD = 0, LIN_DX = 1, LIN_DW = 2, LIN_GRADS = 3, LIN_FWD_SHORT = 4, LIN_FWD_F32 = 5 };
mok_status_t run_linear(LinKind kind, const LinearOperands& o, const LinearParams& p, int num_sms, cudaStream_t st);
// dx and dW of one projection, in one launch where both are large enough.
mok_status_t run_linear_grads(const LinearOperands& ox, const LinearParams& px, const LinearOperands& ow, const LinearParams& pw,
                              int num_sms, cudaStream_t st);

// dz = dy act'(z) in bf16 (dz may be NULL) and the partial column sums of its
// fp32 values ([dz_partials][N], part may be NULL).
int dz_partials(long long M, int N);
cudaError_t launch_linear_dz(const void* dy, int dy_f32, const uint16_t* z, int act, long long M, int N, uint16_t* dz,
                             float* part, cudaStream_t st);

// ---------------------------------------------------------------- AdamW
struct AdamwTensor {
  void* p;
  float* master;
  const void* g;
  void* m;
  void* v;
  uint8_t* m_scale;
  uint8_t* r_scale;
  long long n;
  uint32_t key;     // seeds the tensor's rounding bits
  int first;        // its first chunk of the launch
};
struct AdamwScalars {
  float beta1, one_minus_beta1, beta2, one_minus_beta2;
  float decay;         // 1 - lr weight_decay
  float step_size;     // lr / (1 - beta1^t)
  float inv_sqrt_bc2;  // (1 - beta2^t)^-1/2
  float eps;
  const float* grad_scale;  // device scalar or NULL
};
// What a counted step reads in place of the scalars above: in device memory,
// so that a replayed graph takes the step that is due.
struct AdamwCounter {
  long long count;       // steps counted
  double lr;             // NaN: the call's
  uint64_t seed_change;  // the seed is the call's, exclusive-or this
  float decay, step_size, inv_sqrt_bc2;   // written by launch_adamw_advance
  uint32_t key;                           // the step's and the seed's share of the tensors' keys
};
static_assert(sizeof(AdamwCounter) <= MOK_ADAMW_COUNTER_BYTES, "the documented size");
struct AdamwAdvance {
  double lr, weight_decay, beta1, beta2;
  long long step;   // added to the count
  uint64_t seed;
  int fixed_lr;     // lr as it is here, whatever the counter says
};
cudaError_t launch_adamw_advance(const AdamwAdvance& a, AdamwCounter* counter, cudaStream_t st);
// The step's and the seed's share of a tensor's key, and the tensor's.
__host__ __device__ constexpr uint32_t adamw_step_key(uint64_t seed, long long step) {
  return static_cast<uint32_t>(seed * 0x9E3779B1ull + static_cast<uint64_t>(step) * 0xB504F333ull);
}
constexpr int kAdamwBlock = 2048;   // elements per chunk, the work of one block at a time
// Tensors one launch takes at most, and the launch itself; t[i].first is set.
// counter: NULL, or of a counted step (t[i].key is the tensor's share alone).
constexpr int kAdamwMaxTensors = 400;
cudaError_t launch_adamw(const AdamwTensor* t, int n, int chunks, const AdamwScalars& s, const AdamwCounter* counter, int p_f32,
                         int g_f32, int master, int mx, cudaStream_t st);

}  // namespace mok
