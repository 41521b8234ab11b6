// The extern "C" entry points of the operators around the expert layer's
// products (declared in include/fo.h): argument checks and dispatch.
#include <cuda_runtime.h>

#include <cmath>

#include "api_checks.h"
#include "block_internal.h"
#include "fo_internal.h"

using fo::aligned_type;
using fo::device_ok;
using fo::fits_int32;
using fo::type_ok;

namespace {

constexpr int64_t kMaxBytes = int64_t(1) << 62;

// Tokens and columns that the kernels walk over with 32-bit steps.
bool walkable(int64_t tokens, int64_t columns) {
  return tokens <= (int64_t(1) << 31) - (int64_t(1) << 20) && columns <= int64_t(1) << 30;
}

bool act_ok(fo_activation act) { return act >= FO_ACT_NONE && act <= FO_ACT_SILU; }

bool norm_desc_ok(const fo_norm_desc* d) {
  if (!d || d->tokens < 0 || d->hidden < 0) return false;
  if (!type_ok(fo_type(d->type)) || !type_ok(fo_type(d->stream_type)) ||
      !type_ok(fo_type(d->param_type)))
    return false;
  // (fp32 activations beside a bf16 stream have no kernel)
  if (d->type == FO_TYPE_F32 && d->stream_type != FO_TYPE_F32) return false;
  if (d->gates < 1 || (d->tokens > 0 && d->tokens % d->gates)) return false;
  return std::isfinite(d->scale) && d->eps >= 0.0f;
}

// The arguments that the norm and its gradient share.
bool norm_inputs_ok(const fo_norm_desc& d, const void* x, int64_t x_stride, const void* residual,
                    int64_t residual_stride, const void* post_gain, const void* gate,
                    int64_t gate_stride, const void* pre_gain, const float* post_rstd,
                    const float* pre_rstd) {
  const fo_type t = fo_type(d.type), s = fo_type(d.stream_type), p = fo_type(d.param_type);
  if (!x || x_stride < d.hidden || !aligned_type(x, t)) return false;
  if (residual && (residual_stride < d.hidden || !aligned_type(residual, s))) return false;
  if (gate && (gate_stride < d.hidden || !aligned_type(gate, p))) return false;
  if (!aligned_type(post_gain, p) || !aligned_type(pre_gain, p)) return false;
  if ((post_gain && !post_rstd) || (pre_gain && !pre_rstd)) return false;
  return fo::aligned4(post_rstd) && fo::aligned4(pre_rstd);
}

fo::NormArgs norm_args(const fo_norm_desc& d, const void* x, int64_t x_stride,
                       const void* residual, int64_t residual_stride, const void* post_gain,
                       const void* gate, int64_t gate_stride, const void* pre_gain,
                       const float* post_rstd, const float* pre_rstd) {
  fo::NormArgs a{};
  a.x = x, a.x_stride = x_stride;
  a.residual = residual, a.residual_stride = residual ? residual_stride : 0;
  a.post = post_gain, a.gate = gate, a.pre = pre_gain;
  a.gate_rows = int32_t(d.tokens / d.gates);
  // (a gate with one row has no stride)
  a.gate_stride = gate && d.gates > 1 ? gate_stride : 0;
  a.post_rstd = const_cast<float*>(post_rstd);
  a.pre_rstd = const_cast<float*>(pre_rstd);
  a.tokens = int32_t(d.tokens), a.hidden = int32_t(d.hidden);
  a.params_f32 = d.param_type == FO_TYPE_F32;
  a.scale = d.scale, a.eps = d.eps;
  return a;
}

}  // namespace

extern "C" {

fo_status fo_moe_combine(const void* rows, fo_type type, int64_t table_rows, int64_t hidden,
                         int64_t row_stride, const int32_t* token_row, const float* weights,
                         int64_t tokens, int32_t top_k, void* y, fo_type y_type,
                         int64_t y_stride, int32_t* dev_status, void* stream) {
  if (!type_ok(type) || !type_ok(y_type) || tokens < 0 || hidden < 0 || table_rows < 0)
    return FO_ERR_ARG;
  if (top_k < 1 || top_k > fo::kCombineSlots) return FO_ERR_ARG;
  if (row_stride < hidden || y_stride < hidden) return FO_ERR_ARG;
  if (!dev_status || !fo::aligned4(dev_status)) return FO_ERR_ARG;
  if (tokens == 0 || hidden == 0) return FO_OK;
  if (!token_row || !y || (table_rows > 0 && !rows)) return FO_ERR_ARG;
  if (!aligned_type(rows, type) || !aligned_type(y, y_type) || !fo::aligned4(token_row) ||
      !fo::aligned4(weights))
    return FO_ERR_ARG;
  if (!walkable(tokens, hidden) || !fits_int32(table_rows)) return FO_ERR_UNSUPPORTED;
  fo_status st;
  if (!device_ok(&st)) return st;
  return fo::launch_combine(rows, type, table_rows, hidden, row_stride, token_row, weights,
                            tokens, top_k, y, y_type, y_stride, dev_status, stream);
}

fo_status fo_moe_combine_backward(const void* dy, fo_type dy_type, int64_t dy_stride,
                                  const void* rows, fo_type type, int64_t table_rows,
                                  int64_t hidden, int64_t row_stride, const int32_t* token_row,
                                  const int32_t* row_token, const float* weights,
                                  int64_t tokens, int32_t top_k, void* drows,
                                  int64_t drows_stride, float* dweights, int32_t* dev_status,
                                  void* stream) {
  if (!type_ok(type) || !type_ok(dy_type) || tokens < 0 || hidden < 0 || table_rows < 0)
    return FO_ERR_ARG;
  if (top_k < 1 || top_k > fo::kCombineSlots) return FO_ERR_ARG;
  if (dy_stride < hidden || drows_stride < hidden || (dweights && row_stride < hidden))
    return FO_ERR_ARG;
  if (!dev_status || !fo::aligned4(dev_status)) return FO_ERR_ARG;
  if (tokens > 0 && (!token_row || (hidden > 0 && !dy))) return FO_ERR_ARG;
  if (table_rows > 0 && (!row_token || (hidden > 0 && (!drows || (dweights && !rows)))))
    return FO_ERR_ARG;
  if (!aligned_type(dy, dy_type) || !aligned_type(rows, type) || !aligned_type(drows, type) ||
      !fo::aligned4(token_row) || !fo::aligned4(row_token) || !fo::aligned4(weights) ||
      !fo::aligned4(dweights))
    return FO_ERR_ARG;
  if (!walkable(tokens, hidden) || !fits_int32(table_rows)) return FO_ERR_UNSUPPORTED;
  fo_status st;
  if (!device_ok(&st)) return st;
  return fo::launch_combine_backward(dy, dy_type, dy_stride, rows, type, table_rows, hidden,
                                     row_stride, token_row, row_token, weights, tokens, top_k,
                                     drows, drows_stride, dweights, dev_status, stream);
}

fo_status fo_checkpoint_sizes(int64_t rows, int64_t inter, int64_t* code_bytes,
                              int64_t* scale_bytes) {
  if (rows < 0 || inter < 0 || inter > kMaxBytes / 2 - 32) return FO_ERR_ARG;
  const int64_t padded = (inter + 31) / 32 * 32;
  int64_t n;
  if (__builtin_mul_overflow(rows, 2 * padded, &n) || n >= kMaxBytes) return FO_ERR_ARG;
  if (code_bytes) *code_bytes = n;
  if (scale_bytes) *scale_bytes = n / 32;
  return FO_OK;
}

fo_status fo_gated_act(const void* u, fo_type type, int64_t rows, int64_t inter,
                       int64_t u_stride, fo_activation act, void* h, int64_t h_stride,
                       void* codes, void* scales, void* stream) {
  if (!type_ok(type) || !act_ok(act)) return FO_ERR_ARG;
  if (fo_checkpoint_sizes(rows, inter, nullptr, nullptr) != FO_OK) return FO_ERR_ARG;
  if (u_stride < 2 * inter || h_stride < inter) return FO_ERR_ARG;
  if ((codes != nullptr) != (scales != nullptr) || !fo::aligned16(codes)) return FO_ERR_ARG;
  if (rows == 0 || inter == 0) return FO_OK;
  if (!u || !h || !aligned_type(u, type) || !aligned_type(h, type)) return FO_ERR_ARG;
  if (!fits_int32(rows) || !fits_int32(2 * inter)) return FO_ERR_UNSUPPORTED;
  fo_status st;
  if (!device_ok(&st)) return st;
  return fo::launch_gated_act(u, type, rows, inter, u_stride, act, h, h_stride, codes, scales,
                              stream);
}

fo_status fo_gated_act_backward(const void* dh, fo_type type, int64_t rows, int64_t inter,
                                int64_t dh_stride, fo_activation act, const void* codes,
                                const void* scales, void* du, int64_t du_stride, void* stream) {
  if (!type_ok(type) || !act_ok(act)) return FO_ERR_ARG;
  if (fo_checkpoint_sizes(rows, inter, nullptr, nullptr) != FO_OK) return FO_ERR_ARG;
  if (dh_stride < inter || du_stride < 2 * inter) return FO_ERR_ARG;
  if (rows == 0 || inter == 0) return FO_OK;
  if (!codes || !scales || !fo::aligned16(codes)) return FO_ERR_ARG;
  if (!dh || !du || !aligned_type(dh, type) || !aligned_type(du, type)) return FO_ERR_ARG;
  if (!fits_int32(rows) || !fits_int32(2 * inter)) return FO_ERR_UNSUPPORTED;
  fo_status st;
  if (!device_ok(&st)) return st;
  return fo::launch_gated_act_backward(dh, type, rows, inter, dh_stride, act, codes, scales, du,
                                       du_stride, stream);
}

fo_status fo_block_norm(const fo_norm_desc* d, const void* x, int64_t x_stride,
                        const void* residual, int64_t residual_stride, const void* post_gain,
                        const void* gate, int64_t gate_stride, const void* pre_gain, void* sum,
                        int64_t sum_stride, void* y, int64_t y_stride, float* post_rstd,
                        float* pre_rstd, void* stream) {
  if (!norm_desc_ok(d)) return FO_ERR_ARG;
  if (d->tokens == 0 || d->hidden == 0) return FO_OK;
  if (!norm_inputs_ok(*d, x, x_stride, residual, residual_stride, post_gain, gate, gate_stride,
                      pre_gain, post_rstd, pre_rstd))
    return FO_ERR_ARG;
  if (sum && (sum_stride < d->hidden || !aligned_type(sum, fo_type(d->stream_type))))
    return FO_ERR_ARG;
  if (pre_gain && (!y || y_stride < d->hidden || !aligned_type(y, fo_type(d->type))))
    return FO_ERR_ARG;
  if (!walkable(d->tokens, d->hidden)) return FO_ERR_UNSUPPORTED;
  fo_status st;
  if (!device_ok(&st)) return st;
  fo::NormArgs a = norm_args(*d, x, x_stride, residual, residual_stride, post_gain, gate,
                             gate_stride, pre_gain, post_rstd, pre_rstd);
  a.sum = sum, a.sum_stride = sum ? sum_stride : 0;
  a.y = pre_gain ? y : nullptr, a.y_stride = pre_gain ? y_stride : 0;
  return fo::launch_block_norm(a, fo_type(d->type), fo_type(d->stream_type), stream);
}

fo_status fo_block_norm_workspace(const fo_norm_desc* d, int64_t* bytes) {
  if (!norm_desc_ok(d) || !bytes) return FO_ERR_ARG;
  if (!walkable(d->tokens, d->hidden)) return FO_ERR_UNSUPPORTED;
  *bytes = fo::block_norm_workspace_bytes(d->tokens, d->hidden, d->gates);
  return FO_OK;
}

fo_status fo_block_norm_backward(const fo_norm_desc* d, const void* x, int64_t x_stride,
                                 const void* residual, int64_t residual_stride,
                                 const void* post_gain, const void* gate, int64_t gate_stride,
                                 const void* pre_gain, const float* post_rstd,
                                 const float* pre_rstd, const void* dsum, int64_t dsum_stride,
                                 const void* dy, int64_t dy_stride, void* dx, int64_t dx_stride,
                                 void* dresidual, int64_t dresidual_stride, void* dpost,
                                 void* dgate, void* dpre, void* workspace, void* stream) {
  if (!norm_desc_ok(d)) return FO_ERR_ARG;
  if (d->hidden == 0) return FO_OK;
  const fo_type t = fo_type(d->type), s = fo_type(d->stream_type), p = fo_type(d->param_type);
  if ((post_gain && !dpost) || (gate && !dgate) || (pre_gain && !dpre)) return FO_ERR_ARG;
  if (!aligned_type(dpost, p) || !aligned_type(dgate, p) || !aligned_type(dpre, p))
    return FO_ERR_ARG;
  if (!workspace || !fo::aligned16(workspace)) return FO_ERR_ARG;
  if (d->tokens > 0) {
    if (!norm_inputs_ok(*d, x, x_stride, residual, residual_stride, post_gain, gate, gate_stride,
                        pre_gain, post_rstd, pre_rstd))
      return FO_ERR_ARG;
    if (dsum && (dsum_stride < d->hidden || !aligned_type(dsum, s))) return FO_ERR_ARG;
    if (pre_gain && (!dy || dy_stride < d->hidden || !aligned_type(dy, t))) return FO_ERR_ARG;
    if (!dx || dx_stride < d->hidden || !aligned_type(dx, t)) return FO_ERR_ARG;
    if (dresidual && (dresidual_stride < d->hidden || !aligned_type(dresidual, s)))
      return FO_ERR_ARG;
  }
  if (!walkable(d->tokens, d->hidden)) return FO_ERR_UNSUPPORTED;
  fo_status st;
  if (!device_ok(&st)) return st;
  fo::NormBackArgs a{};
  // (without the second norm no gradient takes a value of the stream)
  a.f = norm_args(*d, x, x_stride, pre_gain ? residual : nullptr, residual_stride, post_gain, gate,
                  gate_stride, pre_gain, post_rstd, pre_rstd);
  a.dsum = dsum, a.dsum_stride = dsum ? dsum_stride : 0;
  a.dy = pre_gain ? dy : nullptr, a.dy_stride = pre_gain ? dy_stride : 0;
  a.dx = dx, a.dx_stride = dx_stride;
  a.dresidual = dresidual, a.dresidual_stride = dresidual ? dresidual_stride : 0;
  a.dpost = dpost, a.dgate = dgate, a.dpre = dpre;
  a.workspace = static_cast<float*>(workspace);
  return fo::launch_block_norm_backward(a, t, s, d->gates, stream);
}

}  // extern "C"
