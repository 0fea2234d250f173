// C ABI of the operators around the layer (declared in include/mok.h): the
// norm, the MXFP8 reader, the dense projection and the optimiser step.
// Argument checks and launch sequences; no allocation happens here.
#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cmath>

#include "api_util.h"
#include "internal.h"
#include "ops.h"

using namespace mok;

namespace {

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

bool is_dtype(int d) { return d == MOK_DTYPE_BF16 || d == MOK_DTYPE_F32; }


// Tile coordinates are 32-bit; a tile may begin up to 256 rows past the end.
constexpr int64_t kMaxM = 0x7fffffffll - 512;

mok_status_t check_linear(int64_t M, int N, int K, int activation) {
  if (M < 0 || M > kMaxM || N < 8 || K < 8 || N % 8 || K % 8 || N > 0x7fffffff - 512 || K > 0x7fffffff - 512)
    return fail(MOK_ERR_INVALID_ARG, "need 0 <= M < 2^31 - 512 and N, K positive multiples of 8");
  if (activation < MOK_ACT_NONE || activation > MOK_ACT_GELU_TANH) return fail(MOK_ERR_INVALID_ARG, "unknown activation");
  return MOK_OK;
}

// The workspace's dz part, padded so that what follows is aligned.
size_t dz_bytes(bool dz, int64_t M, int N) {
  return dz ? (static_cast<size_t>(M) * N * sizeof(uint16_t) + 255) / 256 * 256 : 0;
}

}  // namespace

extern "C" {

mok_status_t mok_mxfp8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, uint16_t* out,
                                  void* stream) {
  NvtxRange nvtx("mok_mxfp8_dequantize");
  if (rows < 0 || K < 0 || (rows > 1 && K % 32))
    return fail(MOK_ERR_INVALID_ARG, "need rows, K >= 0, and K %% 32 == 0 for more than one row");
  if (rows == 0 || K == 0) return MOK_OK;
  if (rows > (1ll << 42) / K) return fail(MOK_ERR_INVALID_ARG, "rows * K too large");
  if (!codes || !scales || !out) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  if (!aligned16(codes) || !aligned16(out)) return fail(MOK_ERR_INVALID_ARG, "misaligned pointer");
  int sms = 0;
  mok_status_t st = device_info(&sms);
  if (st) return st;
  MOK_CUDA(launch_mx_dequantize(codes, scales, rows * K, out, static_cast<cudaStream_t>(stream)));
  return MOK_OK;
}

// ---------------------------------------------------------------- norm
mok_status_t mok_rms_norm(const void* x, int x_dtype, const void* residual, int residual_dtype, const void* weight,
                          int weight_dtype, int64_t rows, int H, float eps, void* h, uint16_t* y, uint8_t* codes,
                          uint8_t* scales, float* rstd, void* stream) {
  NvtxRange nvtx("mok_rms_norm");
  if (rows < 0 || rows > 0x7fffffffll || H < 1 || H > MOK_NORM_MAX_H)
    return fail(MOK_ERR_INVALID_ARG, "need 0 <= rows < 2^31 and 1 <= H <= %d", MOK_NORM_MAX_H);
  if (!is_dtype(x_dtype) || !is_dtype(weight_dtype) || (residual && !is_dtype(residual_dtype)))
    return fail(MOK_ERR_INVALID_ARG, "unknown dtype");
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(MOK_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (rows == 0) return MOK_OK;
  if (!y && !codes) return fail(MOK_ERR_INVALID_ARG, "no output: y and codes are both NULL");
  if ((codes == nullptr) != (scales == nullptr)) return fail(MOK_ERR_INVALID_ARG, "codes and scales go together");
  if (codes && H % 32) return fail(MOK_ERR_INVALID_ARG, "the MXFP8 output needs H %% 32 == 0");
  if (!x || !weight || !rstd || (residual && !h)) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(h) || !aligned16(y) ||
      !aligned16(codes) || !aligned16(rstd))
    return fail(MOK_ERR_INVALID_ARG, "misaligned pointer");
  int sms = 0;
  mok_status_t st = device_info(&sms);
  if (st) return st;
  NormArgs a = {};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.h = h;
  a.y = y;
  a.codes = codes;
  a.scales = scales;
  a.rstd = rstd;
  a.rows = rows;
  a.H = H;
  a.weight_f32 = weight_dtype == MOK_DTYPE_F32;
  a.eps = eps;
  MOK_CUDA(launch_rms_norm(a, x_dtype == MOK_DTYPE_F32, !residual ? 0 : residual_dtype == MOK_DTYPE_F32 ? 2 : 1,
                           static_cast<cudaStream_t>(stream)));
  return MOK_OK;
}

size_t mok_rms_norm_bwd_workspace_bytes(int64_t rows, int H) {
  if (rows < 0 || rows > 0x7fffffffll || H < 1 || H > MOK_NORM_MAX_H) return 0;
  const int n = norm_bwd_walkers(rows, H, false), m = norm_bwd_walkers(rows, H, true);   // for either type of h
  return static_cast<size_t>(n > m ? n : m) * H * sizeof(float) + 256;
}

mok_status_t mok_rms_norm_bwd(const uint16_t* dy, const void* h, int h_dtype, const void* weight, int weight_dtype,
                              const float* rstd, const void* dh, int64_t rows, int H, void* dx, uint16_t* dx_bf16,
                              float* d_weight, void* ws, size_t ws_bytes, void* stream) {
  if (dx_bf16 && h_dtype != MOK_DTYPE_F32) return fail(MOK_ERR_INVALID_ARG, "dx_bf16 goes with an fp32 h");
  return mok_rms_norm_bwd_both(dy, h, h_dtype, weight, weight_dtype, rstd, dh, rows, H, dx, dx_bf16, d_weight, ws, ws_bytes,
                               stream);
}

mok_status_t mok_rms_norm_bwd_both(const uint16_t* dy, const void* h, int h_dtype, const void* weight, int weight_dtype,
                                   const float* rstd, const void* dh, int64_t rows, int H, void* dx, void* dx_other,
                                   float* d_weight, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx("mok_rms_norm_bwd");
  if (rows < 0 || rows > 0x7fffffffll || H < 1 || H > MOK_NORM_MAX_H)
    return fail(MOK_ERR_INVALID_ARG, "need 0 <= rows < 2^31 and 1 <= H <= %d", MOK_NORM_MAX_H);
  if (!is_dtype(h_dtype) || !is_dtype(weight_dtype)) return fail(MOK_ERR_INVALID_ARG, "unknown dtype");
  if (!d_weight || !ws || !weight) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  if (rows > 0 && (!dy || !h || !rstd || !dx)) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  if (!aligned16(dy) || !aligned16(h) || !aligned16(weight) || !aligned16(rstd) || !aligned16(dh) || !aligned16(dx) ||
      !aligned16(dx_other) || !aligned16(d_weight) || !aligned16(ws))
    return fail(MOK_ERR_INVALID_ARG, "misaligned pointer");
  if (ws_bytes < mok_rms_norm_bwd_workspace_bytes(rows, H))
    return fail(MOK_ERR_INVALID_ARG, "workspace too small: %zu < %zu", ws_bytes,
                mok_rms_norm_bwd_workspace_bytes(rows, H));
  int sms = 0;
  mok_status_t st = device_info(&sms);
  if (st) return st;
  NormBwdArgs a = {};
  a.dy = dy;
  a.h = h;
  a.weight = weight;
  a.rstd = rstd;
  a.dh = dh;
  a.dx = dx;
  a.dx_other = dx_other;
  a.part = static_cast<float*>(ws);
  a.rows = rows;
  a.H = H;
  a.weight_f32 = weight_dtype == MOK_DTYPE_F32;
  MOK_CUDA(launch_rms_norm_bwd(a, h_dtype == MOK_DTYPE_F32, d_weight, static_cast<cudaStream_t>(stream)));
  return MOK_OK;
}

// ---------------------------------------------------------------- dense projection
mok_status_t mok_linear(const uint16_t* x, const uint16_t* w, const void* bias, int bias_dtype, const void* residual,
                        int residual_dtype, int activation, int64_t M, int N, int K, void* y, int y_dtype, uint16_t* z,
                        void* stream) {
  NvtxRange nvtx("mok_linear");
  mok_status_t st = check_linear(M, N, K, activation);
  if (st) return st;
  if (!is_dtype(y_dtype) || (bias && !is_dtype(bias_dtype)) || (residual && !is_dtype(residual_dtype)))
    return fail(MOK_ERR_INVALID_ARG, "unknown dtype");
  if (M == 0) return MOK_OK;
  if (!x || !w || !y) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  if (!aligned16(x) || !aligned16(w) || !aligned16(bias) || !aligned16(residual) || !aligned16(y) || !aligned16(z))
    return fail(MOK_ERR_INVALID_ARG, "misaligned pointer");
  int sms = 0;
  st = device_info(&sms);
  if (st) return st;
  LinearParams p = {};
  MOK_CUDA(linear_status_word(&p.status));
  p.L = N;
  p.C = static_cast<int>(M);
  p.act = activation;
  p.out = y;
  p.out_f32 = y_dtype == MOK_DTYPE_F32;
  p.bias = bias;
  p.bias_f32 = bias_dtype == MOK_DTYPE_F32;
  p.residual = residual;
  p.residual_f32 = residual_dtype == MOK_DTYPE_F32;
  p.z = z;
  return run_linear(LIN_FWD, {w, x, K}, p, sms, static_cast<cudaStream_t>(stream));
}

size_t mok_linear_bwd_workspace_bytes(int64_t M, int N, int activation, int dy_dtype, int with_bias) {
  if (M < 0 || M > kMaxM || N < 8 || N % 8 || activation < 0 || activation > MOK_ACT_GELU_TANH || !is_dtype(dy_dtype))
    return 0;
  const bool dz = activation != MOK_ACT_NONE || dy_dtype == MOK_DTYPE_F32;
  return dz_bytes(dz, M, N) + (with_bias ? static_cast<size_t>(dz_partials(M, N)) * N * sizeof(float) : 0) + 256;
}

mok_status_t mok_linear_bwd(const void* dy, int dy_dtype, const uint16_t* x, const uint16_t* w, const uint16_t* z,
                            int activation, int64_t M, int N, int K, uint16_t* dx, uint16_t* d_weight, float* d_bias,
                            void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx("mok_linear_bwd");
  mok_status_t st = check_linear(M, N, K, activation);
  if (st) return st;
  if (!is_dtype(dy_dtype)) return fail(MOK_ERR_INVALID_ARG, "unknown dtype");
  const bool act = activation != MOK_ACT_NONE, make_dz = act || dy_dtype == MOK_DTYPE_F32;
  if (M > 0 && (!dy || (act && !z) || (d_weight && !x) || (dx && !w))) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  if (!aligned16(dy) || !aligned16(x) || !aligned16(w) || !aligned16(z) || !aligned16(dx) || !aligned16(d_weight) ||
      !aligned16(d_bias) || !aligned16(ws))
    return fail(MOK_ERR_INVALID_ARG, "misaligned pointer");
  const size_t need = mok_linear_bwd_workspace_bytes(M, N, activation, dy_dtype, d_bias != nullptr);
  if (!ws || ws_bytes < need) return fail(MOK_ERR_INVALID_ARG, "workspace too small: %zu < %zu", ws ? ws_bytes : 0, need);
  int sms = 0;
  st = device_info(&sms);
  if (st) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {   // sums over no rows
    if (d_weight) MOK_CUDA(cudaMemsetAsync(d_weight, 0, static_cast<size_t>(N) * K * sizeof(uint16_t), s));
    if (d_bias) MOK_CUDA(cudaMemsetAsync(d_bias, 0, static_cast<size_t>(N) * sizeof(float), s));
    return MOK_OK;
  }
  uint16_t* dz = make_dz ? static_cast<uint16_t*>(ws) : nullptr;
  float* part = d_bias ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + dz_bytes(make_dz, M, N)) : nullptr;
  if (dz || part)
    MOK_CUDA(launch_linear_dz(dy, dy_dtype == MOK_DTYPE_F32, z, activation, M, N, dz, part, s));
  const uint16_t* g = make_dz ? dz : static_cast<const uint16_t*>(dy);
  LinearParams px = {};
  MOK_CUDA(linear_status_word(&px.status));
  px.L = K;
  LinearParams pw = px;
  px.C = static_cast<int>(M);
  px.out = dx;
  pw.C = N;
  pw.out = d_weight;
  const LinearOperands ox = {w, g, N}, ow = {x, g, M};
  if (dx && d_weight)
    st = run_linear_grads(ox, px, ow, pw, sms, s);
  else if (d_weight)
    st = run_linear(LIN_DW, ow, pw, sms, s);
  else if (dx)
    st = run_linear(LIN_DX, ox, px, sms, s);
  // the bias's sums run in the products' last wave
  if (!st && d_bias) MOK_CUDA(launch_column_sum(part, dz_partials(M, N), N, d_bias, dx || d_weight, s));
  return st;
}

mok_status_t mok_linear_status(int* status) {
  if (!status) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  int sms = 0;
  mok_status_t st = device_info(&sms);
  if (st) return st;
  int* word = nullptr;
  MOK_CUDA(linear_status_word(&word));
  MOK_CUDA(cudaDeviceSynchronize());
  MOK_CUDA(cudaMemcpy(status, word, sizeof(int), cudaMemcpyDeviceToHost));
  if (*status) MOK_CUDA(cudaMemset(word, 0, sizeof(int)));
  return MOK_OK;
}

}  // extern "C"

// ---------------------------------------------------------------- AdamW
namespace {

// counted: cfg->step is what is added to a count of at least 1.
mok_status_t check_adamw_config(const mok_adamw_config_t* cfg, bool counted) {
  if (!cfg) return fail(MOK_ERR_INVALID_ARG, "NULL config");
  if (!is_dtype(cfg->param_dtype) || !is_dtype(cfg->grad_dtype)) return fail(MOK_ERR_INVALID_ARG, "unknown dtype");
  if (cfg->state != MOK_ADAMW_STATE_F32 && cfg->state != MOK_ADAMW_STATE_MXFP8)
    return fail(MOK_ERR_INVALID_ARG, "unknown state kind");
  if (!std::isfinite(cfg->lr) || !(cfg->beta1 >= 0.0 && cfg->beta1 < 1.0) || !(cfg->beta2 >= 0.0 && cfg->beta2 < 1.0) ||
      !(cfg->eps >= 0.0) || !std::isfinite(cfg->eps) || !std::isfinite(cfg->weight_decay))
    return fail(MOK_ERR_INVALID_ARG, "need finite lr, eps >= 0 and weight_decay, and betas in [0, 1)");
  if (cfg->step < (counted ? 0 : 1)) return fail(MOK_ERR_INVALID_ARG, "step counts from %d", counted ? 0 : 1);
  return MOK_OK;
}

mok_status_t check_adamw(const mok_adamw_config_t* cfg, const mok_adamw_tensor_t* tensors, int num_tensors, bool counted) {
  mok_status_t st = check_adamw_config(cfg, counted);
  if (st) return st;
  if (num_tensors < 0 || (num_tensors > 0 && !tensors)) return fail(MOK_ERR_INVALID_ARG, "bad tensor list");
  const bool mx = cfg->state == MOK_ADAMW_STATE_MXFP8, p_f32 = cfg->param_dtype == MOK_DTYPE_F32;
  const bool master = num_tensors > 0 && tensors[0].master != nullptr;
  if (master && p_f32) return fail(MOK_ERR_INVALID_ARG, "master copies go with bf16 parameters");
  for (int i = 0; i < num_tensors; ++i) {
    const mok_adamw_tensor_t& t = tensors[i];
    if (t.n < 0 || t.n > (1ll << 40)) return fail(MOK_ERR_INVALID_ARG, "tensor %d: bad length", i);
    if ((t.master != nullptr) != master)
      return fail(MOK_ERR_INVALID_ARG, "tensor %d: master copies for all tensors or for none", i);
    if (t.n == 0) continue;
    if (!t.p || !t.g || !t.m || !t.v || (mx && (!t.m_scale || !t.v_scale)))
      return fail(MOK_ERR_INVALID_ARG, "tensor %d: NULL pointer", i);
    if (!aligned16(t.p) || !aligned16(t.master) || !aligned16(t.g) || !aligned16(t.m) || !aligned16(t.v))
      return fail(MOK_ERR_INVALID_ARG, "tensor %d: misaligned pointer", i);
  }
  return MOK_OK;
}

mok_status_t adamw_step(const mok_adamw_config_t* cfg, const mok_adamw_tensor_t* tensors, int num_tensors,
                        const float* grad_scale, const AdamwCounter* counter, void* stream) {
  mok_status_t st = check_adamw(cfg, tensors, num_tensors, counter != nullptr);
  if (st) return st;
  int sms = 0;
  st = device_info(&sms);
  if (st) return st;
  const bool mx = cfg->state == MOK_ADAMW_STATE_MXFP8, p_f32 = cfg->param_dtype == MOK_DTYPE_F32;
  const bool master = num_tensors > 0 && tensors[0].master != nullptr;
  AdamwScalars s = {};
  s.beta1 = static_cast<float>(cfg->beta1);
  s.one_minus_beta1 = static_cast<float>(1.0 - cfg->beta1);
  s.beta2 = static_cast<float>(cfg->beta2);
  s.one_minus_beta2 = static_cast<float>(1.0 - cfg->beta2);
  s.eps = static_cast<float>(cfg->eps);
  s.grad_scale = grad_scale;
  uint32_t key0 = 0;
  if (!counter) {
    const double bc1 = 1.0 - std::pow(cfg->beta1, static_cast<double>(cfg->step));
    const double bc2 = 1.0 - std::pow(cfg->beta2, static_cast<double>(cfg->step));
    s.decay = static_cast<float>(1.0 - cfg->lr * cfg->weight_decay);
    s.step_size = static_cast<float>(cfg->lr / bc1);
    s.inv_sqrt_bc2 = static_cast<float>(1.0 / std::sqrt(bc2));
    key0 = adamw_step_key(cfg->seed, cfg->step);
  }
  AdamwTensor list[kAdamwMaxTensors];
  int n = 0;
  long long blocks = 0;
  const auto flush = [&]() {
    const cudaError_t err = n == 0 ? cudaSuccess
                                   : launch_adamw(list, n, static_cast<int>(blocks), s, counter, p_f32,
                                                  cfg->grad_dtype == MOK_DTYPE_F32, master, mx,
                                                  static_cast<cudaStream_t>(stream));
    n = 0;
    blocks = 0;
    return err;
  };
  for (int i = 0; i < num_tensors; ++i) {
    const mok_adamw_tensor_t& t = tensors[i];
    if (t.n == 0) continue;
    const long long b = (t.n + kAdamwBlock - 1) / kAdamwBlock;
    if (n == kAdamwMaxTensors || blocks + b > 0x7fffffffll) MOK_CUDA(flush());
    AdamwTensor& d = list[n++];
    d.p = t.p;
    d.master = t.master;
    d.g = t.g;
    d.m = t.m;
    d.v = t.v;
    d.m_scale = t.m_scale;
    d.r_scale = t.v_scale;
    d.n = t.n;
    d.key = key0 + static_cast<uint32_t>(t.index) * 0xBB67AE85u;
    d.first = static_cast<int>(blocks);
    blocks += b;
  }
  MOK_CUDA(flush());
  return MOK_OK;
}

}  // namespace

extern "C" {

mok_status_t mok_adamw_step(const mok_adamw_config_t* cfg, const mok_adamw_tensor_t* tensors, int num_tensors,
                            const float* grad_scale, void* stream) {
  NvtxRange nvtx("mok_adamw_step");
  return adamw_step(cfg, tensors, num_tensors, grad_scale, nullptr, stream);
}

mok_status_t mok_adamw_check(const mok_adamw_config_t* cfg, const mok_adamw_tensor_t* tensors, int num_tensors) {
  return check_adamw(cfg, tensors, num_tensors, true);
}

mok_status_t mok_adamw_step_counted(const mok_adamw_config_t* cfg, const mok_adamw_tensor_t* tensors, int num_tensors,
                                    const float* grad_scale, const void* counter, void* stream) {
  NvtxRange nvtx("mok_adamw_step_counted");
  if (!counter || !aligned16(counter)) return fail(MOK_ERR_INVALID_ARG, "counter: NULL or misaligned pointer");
  return adamw_step(cfg, tensors, num_tensors, grad_scale, static_cast<const AdamwCounter*>(counter), stream);
}

mok_status_t mok_adamw_advance(const mok_adamw_config_t* cfg, int fixed_lr, void* counter, void* stream) {
  NvtxRange nvtx("mok_adamw_advance");
  mok_status_t st = check_adamw_config(cfg, true);
  if (st) return st;
  if (!counter || !aligned16(counter)) return fail(MOK_ERR_INVALID_ARG, "counter: NULL or misaligned pointer");
  int sms = 0;
  st = device_info(&sms);
  if (st) return st;
  AdamwAdvance a = {};
  a.lr = cfg->lr;
  a.weight_decay = cfg->weight_decay;
  a.beta1 = cfg->beta1;
  a.beta2 = cfg->beta2;
  a.step = cfg->step;
  a.seed = cfg->seed;
  a.fixed_lr = fixed_lr;
  MOK_CUDA(launch_adamw_advance(a, static_cast<AdamwCounter*>(counter), static_cast<cudaStream_t>(stream)));
  return MOK_OK;
}

}  // extern "C"
