// The extern "C" entry points of the expert layer's operators (declared in
// include/fo.h): argument checks and dispatch to the kernel launchers.
#include <cuda_runtime.h>

#include "fo_internal.h"
#include "moe_internal.h"

namespace {

constexpr int64_t kMaxBytes = int64_t(1) << 62;

bool type_ok(fo_type t) { return t == FO_TYPE_BF16 || t == FO_TYPE_F32; }

// Padded rows x columns of a batch: false when the bytes pass 2^62.
bool mx_elements(int64_t batch, int64_t rows, int64_t cols, int64_t* n) {
  if (batch < 0 || rows < 0 || cols < 0) return false;
  if (rows > kMaxBytes - 127 || cols > kMaxBytes - 127) return false;
  const int64_t r = (rows + 127) / 128 * 128, c = (cols + 127) / 128 * 128;
  int64_t a, b;
  if (__builtin_mul_overflow(r, c, &a) || __builtin_mul_overflow(a, batch, &b)) return false;
  if (b >= kMaxBytes) return false;
  *n = b;
  return true;
}

// Sizes that the kernels index with 32-bit rows and columns.
bool fits_int32(int64_t n) { return n >= 0 && n <= (int64_t(1) << 31) - 256; }

bool device_ok(fo_status* st) {
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
    *st = FO_ERR_CUDA;
    return false;
  }
  *st = FO_ERR_UNSUPPORTED;
  return major == 10 && minor == 3;
}

bool aligned_type(const void* p, fo_type t) {
  return (reinterpret_cast<uintptr_t>(p) & (t == FO_TYPE_BF16 ? 1u : 3u)) == 0;
}

bool few_desc_ok(const fo_moe_few_desc* d) {
  if (!d || d->tokens < 0 || d->tokens > FO_MOE_FEW_TOKENS) return false;
  if (d->hidden < 8 || d->hidden % 8 || d->inter < 8 || d->inter % 8) return false;
  if (!fits_int32(d->hidden) || !fits_int32(2 * int64_t(d->inter))) return false;
  if (d->experts < 1 || d->experts > fo::kRouteExperts) return false;
  if (d->top_k < 1 || d->top_k > fo::kRouteTopK || d->top_k > d->experts) return false;
  if (d->act < FO_ACT_NONE || d->act > FO_ACT_SILU) return false;
  return d->weights == FO_TYPE_BF16 || d->weights == FO_TYPE_MX4;
}

bool route_shape_ok(int64_t tokens, int32_t experts, int32_t top_k) {
  return tokens >= 0 && experts >= 1 && experts <= fo::kRouteExperts && top_k >= 1 &&
         top_k <= fo::kRouteTopK && top_k <= experts;
}

}  // namespace

extern "C" {

fo_status fo_mx_sizes(int64_t batch, int64_t rows, int64_t cols, int64_t* code_bytes,
                      int64_t* scale_bytes) {
  int64_t n = 0;
  if (!mx_elements(batch, rows, cols, &n)) return FO_ERR_ARG;
  if (code_bytes) *code_bytes = n / 2;
  if (scale_bytes) *scale_bytes = n / 32;
  return FO_OK;
}

fo_status fo_mx_quantize(const void* src, fo_type type, int64_t batch, int64_t batch_stride,
                         int64_t rows, int64_t cols, int64_t row_stride, int32_t transpose,
                         const int32_t* row_index, int64_t src_rows, void* codes, void* scales,
                         void* stream) {
  int64_t n = 0;
  if (!type_ok(type) || !mx_elements(batch, rows, cols, &n)) return FO_ERR_ARG;
  if (n == 0) return FO_OK;
  // (a matrix without rows has no address to gather from)
  if ((!src && !(row_index && src_rows == 0)) || !codes || !scales || !fo::aligned16(codes) ||
      !fo::aligned16(scales))
    return FO_ERR_ARG;
  if (!aligned_type(src, type) || !fo::aligned4(row_index)) return FO_ERR_ARG;
  if (row_stride < (transpose ? rows : cols) || batch_stride < 0) return FO_ERR_ARG;
  if (row_index && (batch != 1 || transpose || src_rows < 0)) return FO_ERR_ARG;
  if (!fits_int32(rows) || !fits_int32(cols)) return FO_ERR_UNSUPPORTED;
  fo_status st;
  if (!device_ok(&st)) return st;
  return fo::launch_mx_quantize(src, type, batch, batch_stride, rows, cols, row_stride,
                                transpose != 0, row_index, src_rows, codes, scales, stream);
}

fo_status fo_mx_dequantize(const void* codes, const void* scales, int64_t batch, int64_t rows,
                           int64_t cols, void* dst, fo_type type, int64_t batch_stride,
                           int64_t row_stride, void* stream) {
  int64_t n = 0;
  if (!type_ok(type) || !mx_elements(batch, rows, cols, &n)) return FO_ERR_ARG;
  if (n == 0) return FO_OK;
  if (!dst || !codes || !scales || !fo::aligned16(codes) || !fo::aligned16(scales))
    return FO_ERR_ARG;
  if (!aligned_type(dst, type) || row_stride < cols || batch_stride < 0) return FO_ERR_ARG;
  if (!fits_int32(rows) || !fits_int32(cols)) return FO_ERR_UNSUPPORTED;
  fo_status st;
  if (!device_ok(&st)) return st;
  return fo::launch_mx_dequantize(codes, scales, batch, rows, cols, dst, type, batch_stride,
                                  row_stride, stream);
}

fo_status fo_mx_gemm(int64_t M, int64_t N, int64_t K, const void* A_codes, const void* A_scales,
                     const void* B_codes, const void* B_scales, int32_t n_groups,
                     const int32_t* group_first, const int32_t* group_rows, void* D,
                     fo_type type, int64_t row_stride, int32_t* dev_status, void* stream) {
  if (!type_ok(type) || M < 0 || N < 0 || K < 0 || row_stride < N) return FO_ERR_ARG;
  if (n_groups < 0 || n_groups > fo::kRouteExperts) return FO_ERR_ARG;
  if ((group_first != nullptr) != (n_groups > 0) || (group_rows != nullptr) != (n_groups > 0))
    return FO_ERR_ARG;
  if (!fo::aligned4(group_first) || !fo::aligned4(group_rows)) return FO_ERR_ARG;
  if (!dev_status || !fo::aligned4(dev_status)) return FO_ERR_ARG;
  if (M == 0 || N == 0) return FO_OK;
  if (!D || !aligned_type(D, type)) return FO_ERR_ARG;
  if (K > 0) {
    if (!A_codes || !A_scales || !B_codes || !B_scales) return FO_ERR_ARG;
    if (!fo::aligned16(A_codes) || !fo::aligned16(A_scales) || !fo::aligned16(B_codes) ||
        !fo::aligned16(B_scales))
      return FO_ERR_ARG;
  }
  const int64_t groups = n_groups > 0 ? n_groups : 1;
  if (!fits_int32(M) || !fits_int32(K) || !fits_int32(N) || !fits_int32((N + 127) / 128 * 128 * groups))
    return FO_ERR_UNSUPPORTED;
  fo_status st;
  if (!device_ok(&st)) return st;
  return fo::launch_mx_gemm(M, N, K, A_codes, A_scales, B_codes, B_scales, n_groups, group_first,
                            group_rows, D, type, row_stride, dev_status, stream);
}

fo_status fo_moe_route_sizes(int64_t tokens, int32_t experts, int32_t top_k, int64_t capacity,
                             int64_t* table_rows, int64_t* workspace_bytes) {
  if (!route_shape_ok(tokens, experts, top_k) || capacity < 0) return FO_ERR_ARG;
  if (!fits_int32(tokens) || !fits_int32(tokens * top_k + int64_t(experts) * 128))
    return FO_ERR_UNSUPPORTED;
  if (!fits_int32(capacity) || !fits_int32(capacity * experts)) return FO_ERR_UNSUPPORTED;
  if (table_rows)
    *table_rows = capacity > 0 ? capacity * experts
                               : (tokens * top_k + int64_t(experts) * 127) / 128 * 128;
  if (workspace_bytes) *workspace_bytes = fo::route_workspace_bytes(experts);
  return FO_OK;
}

fo_status fo_moe_route(const void* logits, fo_type type, int64_t tokens, int32_t experts,
                       int64_t row_stride, int32_t top_k, int32_t renormalize, int64_t capacity,
                       int32_t* ids, float* weights, int32_t* row_token, int32_t* row_slot,
                       int32_t* token_row, int32_t* expert_first, int32_t* expert_rows,
                       void* workspace, int32_t* dev_status, void* stream) {
  int64_t table_rows = 0;
  fo_status st = fo_moe_route_sizes(tokens, experts, top_k, capacity, &table_rows, nullptr);
  if (st != FO_OK) return st;
  if (!type_ok(type) || row_stride < experts) return FO_ERR_ARG;
  if (!expert_first || !expert_rows || !workspace || !dev_status) return FO_ERR_ARG;
  if (tokens > 0 && (!logits || !ids || !weights || !token_row)) return FO_ERR_ARG;
  if (table_rows > 0 && (!row_token || !row_slot)) return FO_ERR_ARG;
  if (!aligned_type(logits, type) || !fo::aligned4(ids) || !fo::aligned4(weights) ||
      !fo::aligned4(row_token) || !fo::aligned4(row_slot) || !fo::aligned4(token_row) ||
      !fo::aligned4(expert_first) || !fo::aligned4(expert_rows) || !fo::aligned4(dev_status) ||
      !fo::aligned16(workspace))
    return FO_ERR_ARG;
  if (!device_ok(&st)) return st;
  return fo::launch_moe_route(logits, type, tokens, experts, row_stride, top_k, renormalize != 0,
                              capacity, table_rows, ids, weights, row_token, row_slot, token_row,
                              expert_first, expert_rows, workspace, dev_status, stream);
}

fo_status fo_moe_route_backward(const void* logits, fo_type type, int64_t tokens,
                                int32_t experts, int64_t row_stride, int32_t top_k,
                                int32_t renormalize, const int32_t* ids, const float* weights,
                                const float* dweights, void* dlogits, int64_t dlogits_stride,
                                void* stream) {
  if (!type_ok(type) || !route_shape_ok(tokens, experts, top_k)) return FO_ERR_ARG;
  if (row_stride < experts || dlogits_stride < experts) return FO_ERR_ARG;
  if (tokens == 0) return FO_OK;
  if (!logits || !ids || !weights || !dweights || !dlogits) return FO_ERR_ARG;
  if (!aligned_type(logits, type) || !aligned_type(dlogits, type) || !fo::aligned4(ids) ||
      !fo::aligned4(weights) || !fo::aligned4(dweights))
    return FO_ERR_ARG;
  if (!fits_int32(tokens)) return FO_ERR_UNSUPPORTED;
  fo_status st;
  if (!device_ok(&st)) return st;
  return fo::launch_moe_route_backward(logits, type, tokens, experts, row_stride, top_k,
                                       renormalize != 0, ids, weights, dweights, dlogits,
                                       dlogits_stride, stream);
}

fo_status fo_moe_few_workspace(const fo_moe_few_desc* d, int64_t* bytes) {
  if (!few_desc_ok(d) || !bytes) return FO_ERR_ARG;
  *bytes = fo::few_workspace_bytes(*d);
  return FO_OK;
}

fo_status fo_moe_few(const fo_moe_few_desc* d, const void* x, int64_t x_stride,
                     const void* router, const void* W1, const void* W1_scales, const void* W2,
                     const void* W2_scales, void* y, int64_t y_stride, void* workspace,
                     int32_t* dev_status, void* stream) {
  if (!few_desc_ok(d)) return FO_ERR_ARG;
  const bool mx = d->weights == FO_TYPE_MX4;
  if (mx != (W1_scales != nullptr) || mx != (W2_scales != nullptr)) return FO_ERR_ARG;
  if (x_stride < d->hidden || x_stride % 8 || y_stride < d->hidden) return FO_ERR_ARG;
  if (!router || !W1 || !W2 || !workspace || !dev_status) return FO_ERR_ARG;
  if (d->tokens > 0 && (!x || !y)) return FO_ERR_ARG;
  if (!fo::aligned16(x) || !fo::aligned16(router) || !fo::aligned16(W1) || !fo::aligned16(W2) ||
      !fo::aligned16(W1_scales) || !fo::aligned16(W2_scales) || !fo::aligned16(workspace) ||
      !fo::aligned4(dev_status) || !aligned_type(y, FO_TYPE_BF16))
    return FO_ERR_ARG;
  // rows of all experts are indexed with 32 bits
  if (!fits_int32(int64_t(d->experts) * ((2 * int64_t(d->inter) + 127) / 128 * 128)) ||
      !fits_int32(int64_t(d->experts) * ((int64_t(d->hidden) + 127) / 128 * 128)))
    return FO_ERR_UNSUPPORTED;
  if (d->tokens == 0) return FO_OK;
  fo_status st;
  if (!device_ok(&st)) return st;
  return fo::launch_moe_few(*d, x, x_stride, router, W1, W1_scales, W2, W2_scales, y, y_stride,
                            workspace, dev_status, stream);
}

}  // extern "C"
