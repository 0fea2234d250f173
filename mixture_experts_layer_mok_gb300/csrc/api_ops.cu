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


}  // namespace

extern "C" {

mok_status_t mok_mxfp8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K, uint16_t* out,
                                  void* stream) {
  NvtxRange nvtx("mok_mxfp8_dequantize");
  if (rows < 0 || K < 0 || (rows > 1 && K % 32))
    return fail(MOK_ERR_INVALID_ARG, "need rows, K >= 0, and K %% 32 == 0 for more than one row");
  if (rows == 0 || K == 0) return MOK_OK;
  if (rows > (1ll << 46) / K) return fail(MOK_ERR_INVALID_ARG, "rows * K too large");
  if (!codes || !scales || !out) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  if (!aligned16(codes) || !aligned16(out)) return fail(MOK_ERR_INVALID_ARG, "misaligned pointer");
  int sms = 0;
  mok_status_t st = device_info(&sms);
  if (st) return st;
  MOK_CUDA(launch_mx_dequantize(codes, scales, rows * K, out, sms, static_cast<cudaStream_t>(stream)));
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
  return static_cast<size_t>(norm_bwd_walkers(rows, H)) * H * sizeof(float) + 256;
}

mok_status_t mok_rms_norm_bwd(const uint16_t* dy, const void* h, int h_dtype, const void* weight, int weight_dtype,
                              const float* rstd, const void* dh, int64_t rows, int H, void* dx, uint16_t* dx_bf16,
                              float* d_weight, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx("mok_rms_norm_bwd");
  if (rows < 0 || rows > 0x7fffffffll || H < 1 || H > MOK_NORM_MAX_H)
    return fail(MOK_ERR_INVALID_ARG, "need 0 <= rows < 2^31 and 1 <= H <= %d", MOK_NORM_MAX_H);
  if (!is_dtype(h_dtype) || !is_dtype(weight_dtype)) return fail(MOK_ERR_INVALID_ARG, "unknown dtype");
  if (dx_bf16 && h_dtype != MOK_DTYPE_F32) return fail(MOK_ERR_INVALID_ARG, "dx_bf16 goes with an fp32 h");
  if (!d_weight || !ws || !weight) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  if (rows > 0 && (!dy || !h || !rstd || !dx)) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  if (!aligned16(dy) || !aligned16(h) || !aligned16(weight) || !aligned16(rstd) || !aligned16(dh) || !aligned16(dx) ||
      !aligned16(dx_bf16) || !aligned16(d_weight) || !aligned16(ws))
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
  a.dx16 = dx_bf16;
  a.part = static_cast<float*>(ws);
  a.rows = rows;
  a.H = H;
  a.weight_f32 = weight_dtype == MOK_DTYPE_F32;
  MOK_CUDA(launch_rms_norm_bwd(a, h_dtype == MOK_DTYPE_F32, d_weight, static_cast<cudaStream_t>(stream)));
  return MOK_OK;
}

// ---------------------------------------------------------------- AdamW
mok_status_t mok_adamw_step(const mok_adamw_config_t* cfg, const mok_adamw_tensor_t* tensors, int num_tensors,
                            const float* grad_scale, void* stream) {
  NvtxRange nvtx("mok_adamw_step");
  if (!cfg) return fail(MOK_ERR_INVALID_ARG, "NULL config");
  if (num_tensors < 0 || (num_tensors > 0 && !tensors)) return fail(MOK_ERR_INVALID_ARG, "bad tensor list");
  if (!is_dtype(cfg->param_dtype) || !is_dtype(cfg->grad_dtype)) return fail(MOK_ERR_INVALID_ARG, "unknown dtype");
  if (cfg->state != MOK_ADAMW_STATE_F32 && cfg->state != MOK_ADAMW_STATE_MXFP8)
    return fail(MOK_ERR_INVALID_ARG, "unknown state kind");
  if (!std::isfinite(cfg->lr) || !(cfg->beta1 >= 0.0 && cfg->beta1 < 1.0) || !(cfg->beta2 >= 0.0 && cfg->beta2 < 1.0) ||
      !(cfg->eps >= 0.0) || !std::isfinite(cfg->eps) || !std::isfinite(cfg->weight_decay))
    return fail(MOK_ERR_INVALID_ARG, "need finite lr, eps >= 0 and weight_decay, and betas in [0, 1)");
  if (cfg->step < 1) return fail(MOK_ERR_INVALID_ARG, "step counts from 1");
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
  int sms = 0;
  mok_status_t st = device_info(&sms);
  if (st) return st;
  const double bc1 = 1.0 - std::pow(cfg->beta1, static_cast<double>(cfg->step));
  const double bc2 = 1.0 - std::pow(cfg->beta2, static_cast<double>(cfg->step));
  AdamwScalars s = {};
  s.beta1 = static_cast<float>(cfg->beta1);
  s.one_minus_beta1 = static_cast<float>(1.0 - cfg->beta1);
  s.beta2 = static_cast<float>(cfg->beta2);
  s.one_minus_beta2 = static_cast<float>(1.0 - cfg->beta2);
  s.decay = static_cast<float>(1.0 - cfg->lr * cfg->weight_decay);
  s.step_size = static_cast<float>(cfg->lr / bc1);
  s.inv_sqrt_bc2 = static_cast<float>(1.0 / std::sqrt(bc2));
  s.eps = static_cast<float>(cfg->eps);
  s.grad_scale = grad_scale;
  const uint32_t key0 = static_cast<uint32_t>(cfg->seed * 0x9E3779B1ull + static_cast<uint64_t>(cfg->step) * 0xB504F333ull);
  AdamwTensor list[kAdamwMaxTensors];
  int n = 0;
  long long blocks = 0;
  const auto flush = [&]() {
    const cudaError_t err = n == 0 ? cudaSuccess
                                   : launch_adamw(list, n, static_cast<int>(blocks), s, p_f32,
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

}  // extern "C"
