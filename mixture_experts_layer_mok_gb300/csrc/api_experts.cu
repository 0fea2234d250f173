// C ABI of routed experts as operators of their own (declared in include/mok.h):
// the router, the products grouped by expert, and the products with 4-bit
// weights.  Argument checks and launch sequences; no allocation happens here.
#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cmath>

#include "api_util.h"
#include "experts.h"
#include "internal.h"
#include "ops.h"

using namespace mok;

namespace {

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

bool is_dtype(int d) { return d == MOK_DTYPE_BF16 || d == MOK_DTYPE_F32; }

// ---------------------------------------------------------------- router
mok_status_t check_route(int logits_dtype, int64_t T, int E, int k, int score, float scale) {
  if (T < 0 || T > 0x7fffffffll || E < 1 || E > MOK_ROUTE_MAX_E || k < 1 || k > MOK_ROUTE_MAX_K || k > E)
    return fail(MOK_ERR_INVALID_ARG, "need 0 <= T < 2^31, 1 <= E <= %d and 1 <= k <= min(E, %d)", MOK_ROUTE_MAX_E, MOK_ROUTE_MAX_K);
  if (!is_dtype(logits_dtype)) return fail(MOK_ERR_INVALID_ARG, "unknown dtype");
  if (score != MOK_SCORE_SOFTMAX && score != MOK_SCORE_SIGMOID) return fail(MOK_ERR_INVALID_ARG, "unknown score");
  if (!std::isfinite(scale)) return fail(MOK_ERR_INVALID_ARG, "scale must be finite");
  return MOK_OK;
}

}  // namespace

extern "C" {

size_t mok_route_workspace_bytes(int64_t T, int E) {
  if (T < 0 || T > 0x7fffffffll || E < 1 || E > MOK_ROUTE_MAX_E) return 0;
  return 2 * static_cast<size_t>(route_blocks(T, E)) * E * sizeof(float) + 256;
}

mok_status_t mok_route(const void* logits, int logits_dtype, const float* bias, int64_t T, int E, int k, int score, int normalize,
                       float scale, int64_t* experts, float* weights, float* lse, int32_t* counts, float* mean_score, void* ws,
                       size_t ws_bytes, void* stream) {
  NvtxRange nvtx("mok_route");
  mok_status_t st = check_route(logits_dtype, T, E, k, score, scale);
  if (st) return st;
  if ((counts == nullptr) != (mean_score == nullptr)) return fail(MOK_ERR_INVALID_ARG, "counts and mean_score go together");
  if (T > 0 && (!logits || !experts || !weights || !lse)) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  if (!aligned16(logits) || !aligned16(bias) || !aligned16(experts) || !aligned16(weights) || !aligned16(lse) || !aligned16(counts) ||
      !aligned16(mean_score) || !aligned16(ws))
    return fail(MOK_ERR_INVALID_ARG, "misaligned pointer");
  if (counts && (!ws || ws_bytes < mok_route_workspace_bytes(T, E)))
    return fail(MOK_ERR_INVALID_ARG, "workspace too small: %zu < %zu", ws ? ws_bytes : 0, mok_route_workspace_bytes(T, E));
  if (T == 0 && !counts) return MOK_OK;
  int sms = 0;
  st = device_info(&sms);
  if (st) return st;
  RouteArgs a = {};
  a.logits = logits;
  a.bias = bias;
  a.T = T;
  a.E = E;
  a.k = k;
  a.sigmoid = score == MOK_SCORE_SIGMOID;
  a.normalize = normalize != 0;
  a.scale = scale;
  a.experts = experts;
  a.weights = weights;
  a.lse = lse;
  a.counts = counts;
  a.mean_score = mean_score;
  a.part = static_cast<float*>(ws);
  MOK_CUDA(launch_route(a, logits_dtype == MOK_DTYPE_F32, static_cast<cudaStream_t>(stream)));
  return MOK_OK;
}

mok_status_t mok_route_bwd(const float* d_weights, const void* logits, int logits_dtype, const int64_t* experts, const float* d_lse,
                           const float* d_mean_score, int64_t T, int E, int k, int score, int normalize, float scale, void* d_logits,
                           void* stream) {
  NvtxRange nvtx("mok_route_bwd");
  mok_status_t st = check_route(logits_dtype, T, E, k, score, scale);
  if (st) return st;
  if (T == 0) return MOK_OK;
  if (!d_weights || !logits || !experts || !d_logits) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  if (!aligned16(d_weights) || !aligned16(logits) || !aligned16(experts) || !aligned16(d_lse) || !aligned16(d_mean_score) ||
      !aligned16(d_logits))
    return fail(MOK_ERR_INVALID_ARG, "misaligned pointer");
  int sms = 0;
  st = device_info(&sms);
  if (st) return st;
  RouteBwdArgs a = {};
  a.d_weights = d_weights;
  a.logits = logits;
  a.experts = experts;
  a.d_lse = d_lse;
  a.d_mean_score = d_mean_score;
  a.d_logits = d_logits;
  a.T = T;
  a.E = E;
  a.k = k;
  a.sigmoid = score == MOK_SCORE_SIGMOID;
  a.normalize = normalize != 0;
  a.scale = scale;
  MOK_CUDA(launch_route_bwd(a, logits_dtype == MOK_DTYPE_F32, static_cast<cudaStream_t>(stream)));
  return MOK_OK;
}

}  // extern "C"

// ---------------------------------------------------------------- products grouped by expert
namespace {

constexpr int64_t kMaxRows = 0x7fffffffll - 512;   // tile coordinates are 32-bit

mok_status_t check_grouped(int64_t M, int E, int N, int K, int activation) {
  if (M < 0 || M > kMaxRows || E < 1 || E > MOK_GROUPED_MAX_E || N < 8 || K < 8 || N % 8 || K % 8 || N > kMaxRows || K > kMaxRows)
    return fail(MOK_ERR_INVALID_ARG, "need 0 <= M < 2^31 - 512, 1 <= E <= %d and N, K positive multiples of 8", MOK_GROUPED_MAX_E);
  if (static_cast<int64_t>(N) * K >= 1ll << 38) return fail(MOK_ERR_INVALID_ARG, "N * K too large");
  if (activation < MOK_ACT_NONE || activation > MOK_ACT_GELU_TANH) return fail(MOK_ERR_INVALID_ARG, "unknown activation");
  return MOK_OK;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// The backward's workspace: the groups' plan, dz, and the bias's partial sums,
// each on a multiple of 256 (tensor maps want 128) from the first in it.
struct GroupedWs {
  size_t dz, part, bytes;
};
GroupedWs grouped_ws(int64_t M, int E, int N, bool dz, bool bias) {
  GroupedWs w;
  w.dz = up256(grouped_plan_bytes(E));
  w.part = w.dz + (dz ? up256(static_cast<size_t>(M) * N * sizeof(uint16_t)) : 0);
  w.bytes = w.part + (bias && M > 0 ? up256(static_cast<size_t>(grouped_dz_parts(static_cast<int>(M), N, E)) * N * sizeof(float)) : 0) + 256;
  return w;
}

}  // namespace

extern "C" {

mok_status_t mok_grouped_linear(const uint16_t* x, const uint16_t* w, const int32_t* counts, const void* bias, int bias_dtype,
                                int activation, int64_t M, int E, int N, int K, void* y, int y_dtype, uint16_t* z, void* stream) {
  NvtxRange nvtx("mok_grouped_linear");
  mok_status_t st = check_grouped(M, E, N, K, activation);
  if (st) return st;
  if (!is_dtype(y_dtype) || (bias && !is_dtype(bias_dtype))) return fail(MOK_ERR_INVALID_ARG, "unknown dtype");
  if (M == 0) return MOK_OK;
  if (!x || !w || !counts || !y) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  if (!aligned16(x) || !aligned16(w) || !aligned16(counts) || !aligned16(bias) || !aligned16(y) || !aligned16(z))
    return fail(MOK_ERR_INVALID_ARG, "misaligned pointer");
  int sms = 0;
  st = device_info(&sms);
  if (st) return st;
  GroupedRowsParams p = {};
  MOK_CUDA(linear_status_word(&p.status));
  p.counts = counts;
  p.E = E;
  p.L = N;
  p.M = static_cast<int>(M);
  p.act = activation;
  p.bias = bias;
  p.bias_f32 = bias_dtype == MOK_DTYPE_F32;
  p.out = y;
  p.z = z;
  GroupedRowsCall c = {};
  c.w = w;
  c.x = x;
  c.K = K;
  c.w_mn = false;
  c.out_f32 = y_dtype == MOK_DTYPE_F32;
  return run_grouped_rows(c, p, static_cast<cudaStream_t>(stream));
}

size_t mok_grouped_linear_bwd_workspace_bytes(int64_t M, int E, int N, int activation, int dy_dtype, int with_bias) {
  if (check_grouped(M, E, N, 8, activation) || !is_dtype(dy_dtype)) return 0;
  return grouped_ws(M, E, N, activation != MOK_ACT_NONE || dy_dtype == MOK_DTYPE_F32, with_bias != 0).bytes;
}

mok_status_t mok_grouped_linear_bwd(const void* dy, int dy_dtype, const uint16_t* x, const uint16_t* w, const int32_t* counts,
                                    const uint16_t* z, int activation, int64_t M, int E, int N, int K, uint16_t* dx,
                                    uint16_t* d_weight, float* d_bias, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx("mok_grouped_linear_bwd");
  mok_status_t st = check_grouped(M, E, N, K, activation);
  if (st) return st;
  if (!is_dtype(dy_dtype)) return fail(MOK_ERR_INVALID_ARG, "unknown dtype");
  const bool act = activation != MOK_ACT_NONE, make_dz = act || dy_dtype == MOK_DTYPE_F32;
  if (M > 0 && (!dy || !counts || (act && !z) || (d_weight && !x) || (dx && !w))) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  if (!aligned16(dy) || !aligned16(x) || !aligned16(w) || !aligned16(counts) || !aligned16(z) || !aligned16(dx) || !aligned16(d_weight) ||
      !aligned16(d_bias) || !aligned16(ws))
    return fail(MOK_ERR_INVALID_ARG, "misaligned pointer");
  const GroupedWs at = grouped_ws(M, E, N, make_dz, d_bias != nullptr);
  if (!ws || ws_bytes < at.bytes) return fail(MOK_ERR_INVALID_ARG, "workspace too small: %zu < %zu", ws ? ws_bytes : 0, at.bytes);
  int sms = 0;
  st = device_info(&sms);
  if (st) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {   // sums over no rows
    if (d_weight) MOK_CUDA(cudaMemsetAsync(d_weight, 0, static_cast<size_t>(E) * N * K * sizeof(uint16_t), s));
    if (d_bias) MOK_CUDA(cudaMemsetAsync(d_bias, 0, static_cast<size_t>(E) * N * sizeof(float), s));
    return MOK_OK;
  }
  if (!dx && !d_weight && !d_bias) return MOK_OK;
  int* status = nullptr;
  MOK_CUDA(linear_status_word(&status));
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ws) + 255) & ~static_cast<uintptr_t>(255));
  uint16_t* dz = make_dz ? reinterpret_cast<uint16_t*>(base + at.dz) : nullptr;
  float* part = d_bias ? reinterpret_cast<float*>(base + at.part) : nullptr;
  const GroupedBias bias = {part, d_bias, grouped_dz_chunk(static_cast<int>(M), N)};
  GroupedWeightCall c = {};
  c.dz = make_dz ? dz : static_cast<const uint16_t*>(dy);
  c.x = x;
  c.counts = counts;
  c.E = E;
  c.M = static_cast<int>(M);
  c.N = N;
  c.K = K;
  c.out = d_weight;
  c.status = status;
  st = run_grouped_dz(c, {dy, dy_dtype == MOK_DTYPE_F32, z, activation, dz, part}, d_weight != nullptr, base, s);
  if (st) return st;
  if (d_weight) {   // and the bias's sums
    st = run_grouped_weights(c, base, bias, s);
    if (st) return st;
  }
  if (dx) {
    GroupedRowsParams p = {};
    p.status = status;
    p.counts = counts;
    p.E = E;
    p.L = K;
    p.M = c.M;
    p.act = MOK_ACT_NONE;
    p.out = dx;
    p.beside_last = d_weight != nullptr;
    GroupedRowsCall r = {};
    r.w = w;
    r.x = c.dz;
    r.K = N;
    r.w_mn = true;
    r.out_f32 = false;
    st = run_grouped_rows(r, p, s);
    if (st) return st;
  }
  if (d_bias && !d_weight) MOK_CUDA(launch_grouped_bias(bias, base, E, N, s));
  return MOK_OK;
}

}  // extern "C"

// ---------------------------------------------------------------- 4-bit weights
namespace {

mok_status_t int4_shape(int64_t matrices, int N, int K, int group, Int4Shape* s) {
  if (matrices < 1 || N < 1 || K < 32 || (group != 32 && group != 64 && group != 128) || K % group)
    return fail(MOK_ERR_INVALID_ARG, "need matrices, N >= 1, a group of 32, 64 or 128, and K a positive multiple of it");
  if (N > 0x7fffffff - 64 || K > 0x7fffffff - 4096 || matrices > 0x7fffffffll) return fail(MOK_ERR_INVALID_ARG, "N, K or matrices too large");
  *s = {matrices, N, K, group};
  // the launches' grids: 2^30 x 2^15 tiles
  if (static_cast<double>(matrices) * static_cast<double>(s->row_tiles()) * s->blocks() > 1e12) return fail(MOK_ERR_INVALID_ARG, "weight too large");
  return MOK_OK;
}

}  // namespace

extern "C" {

mok_status_t mok_int4_bytes(int64_t matrices, int N, int K, int group, size_t* codes, size_t* scales, size_t* zeros) {
  Int4Shape s = {};
  const mok_status_t st = int4_shape(matrices, N, K, group, &s);
  if (st) return st;
  const size_t tiles = static_cast<size_t>(s.tiles()), each = static_cast<size_t>(s.tile_scales());
  if (codes) *codes = tiles * kInt4TileBytes;
  if (scales) *scales = tiles * each * sizeof(uint16_t);
  if (zeros) *zeros = tiles * each;
  return MOK_OK;
}

mok_status_t mok_int4_quantize(const void* w, int w_dtype, int64_t matrices, int N, int K, int group, uint8_t* codes, uint16_t* scales,
                               uint8_t* zeros, void* stream) {
  NvtxRange nvtx("mok_int4_quantize");
  Int4Shape s = {};
  mok_status_t st = int4_shape(matrices, N, K, group, &s);
  if (st) return st;
  if (!is_dtype(w_dtype)) return fail(MOK_ERR_INVALID_ARG, "unknown dtype");
  if (!w || !codes || !scales) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  if (!aligned16(w) || !aligned16(codes) || !aligned16(scales) || !aligned16(zeros)) return fail(MOK_ERR_INVALID_ARG, "misaligned pointer");
  int sms = 0;
  st = device_info(&sms);
  if (st) return st;
  MOK_CUDA(launch_int4_quantize(w, w_dtype == MOK_DTYPE_F32, s, codes, scales, zeros, static_cast<cudaStream_t>(stream)));
  return MOK_OK;
}

mok_status_t mok_int4_pack(const uint8_t* q, const uint16_t* q_scales, const uint8_t* q_zeros, int64_t matrices, int N, int K, int group,
                           uint8_t* codes, uint16_t* scales, uint8_t* zeros, void* stream) {
  NvtxRange nvtx("mok_int4_pack");
  Int4Shape s = {};
  mok_status_t st = int4_shape(matrices, N, K, group, &s);
  if (st) return st;
  if (!q || !q_scales || !codes || !scales) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  if ((q_zeros == nullptr) != (zeros == nullptr)) return fail(MOK_ERR_INVALID_ARG, "zeros: both or neither");
  if (!aligned16(q) || !aligned16(q_scales) || !aligned16(q_zeros) || !aligned16(codes) || !aligned16(scales) || !aligned16(zeros))
    return fail(MOK_ERR_INVALID_ARG, "misaligned pointer");
  int sms = 0;
  st = device_info(&sms);
  if (st) return st;
  MOK_CUDA(launch_int4_pack(q, q_scales, q_zeros, s, codes, scales, zeros, static_cast<cudaStream_t>(stream)));
  return MOK_OK;
}

mok_status_t mok_int4_dequantize(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t matrices, int N, int K,
                                 int group, uint16_t* out, void* stream) {
  NvtxRange nvtx("mok_int4_dequantize");
  Int4Shape s = {};
  mok_status_t st = int4_shape(matrices, N, K, group, &s);
  if (st) return st;
  if (!codes || !scales || !out) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(zeros) || !aligned16(out)) return fail(MOK_ERR_INVALID_ARG, "misaligned pointer");
  int sms = 0;
  st = device_info(&sms);
  if (st) return st;
  MOK_CUDA(launch_int4_dequantize(codes, scales, zeros, s, out, static_cast<cudaStream_t>(stream)));
  return MOK_OK;
}

mok_status_t mok_int4_linear(const uint16_t* x, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t matrices,
                             int N, int K, int group, const int64_t* experts, int64_t rows, int rows_per_x, const void* bias,
                             int bias_dtype, int activation, void* y, int y_dtype, void* stream) {
  NvtxRange nvtx("mok_int4_linear");
  Int4LinearArgs a = {};
  mok_status_t st = int4_shape(matrices, N, K, group, &a.w);
  if (st) return st;
  if (rows < 0 || rows > MOK_INT4_MAX_ROWS || rows_per_x < 1)
    return fail(MOK_ERR_INVALID_ARG, "need 0 <= rows <= %d and rows_per_x >= 1", MOK_INT4_MAX_ROWS);
  if (!experts && (matrices != 1 || rows_per_x != 1)) return fail(MOK_ERR_INVALID_ARG, "several matrices go with experts");
  if (activation < MOK_ACT_NONE || activation > MOK_ACT_GELU_TANH) return fail(MOK_ERR_INVALID_ARG, "unknown activation");
  if (!is_dtype(y_dtype) || (bias && !is_dtype(bias_dtype))) return fail(MOK_ERR_INVALID_ARG, "unknown dtype");
  if (rows == 0) return MOK_OK;
  if (!x || !codes || !scales || !y) return fail(MOK_ERR_INVALID_ARG, "NULL argument");
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales) || !aligned16(zeros) || !aligned16(experts) || !aligned16(bias) || !aligned16(y))
    return fail(MOK_ERR_INVALID_ARG, "misaligned pointer");
  int sms = 0;
  st = device_info(&sms);
  if (st) return st;
  MOK_CUDA(linear_status_word(&a.status));
  a.codes = codes;
  a.scales = scales;
  a.zeros = zeros;
  a.x = x;
  a.experts = experts;
  a.bias = bias;
  a.y = y;
  a.rows = static_cast<int>(rows);
  a.x_div = rows_per_x;
  a.act = activation;
  a.out_f32 = y_dtype == MOK_DTYPE_F32;
  a.bias_f32 = bias_dtype == MOK_DTYPE_F32;
  // more than 8 rows of x and a matrix of some size: the tensor core with codes in TMEM.  Measured, that and mma.sync: 12 rows times
  // 2048 x 2048 5.0 and 4.2 us, 7168 x 2048 7.4 and 7.5, 16384 x 8192 27 and 35; 64 rows 8.9 and 6.5, 12.7 and 18.6, 39 and 108
  if (!experts && rows > 8 && static_cast<int64_t>(N) * K > 1ll << 23) return run_int4_tc(a, static_cast<cudaStream_t>(stream));
  MOK_CUDA(launch_int4_linear(a, sms, static_cast<cudaStream_t>(stream)));
  return MOK_OK;
}

}  // extern "C"
