// Launchers of the expert layer's operators, called by their C entry points
// after the arguments have been checked.
#pragma once

#include <cstdint>

#include "fo.h"

namespace fo {

constexpr int kRouteExperts = 1024;   // experts a router may choose from
constexpr int kRouteTopK = 32;        // slots of a token
constexpr int kRouteGroups = 32;      // groups of experts

// mx_quantize.cu
fo_status launch_mx_quantize(const void* src, fo_type type, int64_t batch, int64_t batch_stride,
                             int64_t rows, int64_t cols, int64_t row_stride, bool transpose,
                             const int32_t* row_index, int64_t src_rows, void* codes,
                             void* scales, void* stream);
fo_status launch_mx_dequantize(const void* codes, const void* scales, int64_t batch,
                               int64_t rows, int64_t cols, void* dst, fo_type type,
                               int64_t batch_stride, int64_t row_stride, void* stream);

// mx_gemm.cu
fo_status launch_mx_gemm(int64_t M, int64_t N, int64_t K, const void* a_codes,
                         const void* a_scales, const void* b_codes, const void* b_scales,
                         int32_t n_groups, const int32_t* group_first,
                         const int32_t* group_rows, void* D, fo_type type, int64_t row_stride,
                         int32_t* dev_status, void* stream);

// moe_route.cu
int64_t route_workspace_bytes(int experts);
fo_status launch_moe_route(const void* logits, fo_type type, int64_t tokens, int32_t experts,
                           int64_t row_stride, int32_t top_k, bool renormalize,
                           int64_t capacity, int64_t table_rows, int32_t* ids, float* weights,
                           int32_t* row_token, int32_t* row_slot, int32_t* token_row,
                           int32_t* expert_first, int32_t* expert_rows, void* workspace,
                           int32_t* dev_status, void* stream);
fo_status launch_moe_route_backward(const void* logits, fo_type type, int64_t tokens,
                                    int32_t experts, int64_t row_stride, int32_t top_k,
                                    bool renormalize, const int32_t* ids, const float* weights,
                                    const float* dweights, void* dlogits,
                                    int64_t dlogits_stride, void* stream);

fo_status launch_moe_route_scored(const fo_route_desc& d, const void* logits, fo_type type,
                                  int64_t tokens, int64_t row_stride, const float* bias,
                                  int64_t table_rows, int32_t* ids, float* weights,
                                  int32_t* row_token, int32_t* row_slot, int32_t* token_row,
                                  int32_t* expert_first, int32_t* expert_rows, void* workspace,
                                  int32_t* dev_status, void* stream);

// moe_route_scored_backward.cu
fo_status launch_moe_route_scored_backward(const fo_route_desc& d, const void* logits,
                                           fo_type type, int64_t tokens, int64_t row_stride,
                                           const int32_t* ids, const float* weights,
                                           const float* dweights, void* dlogits,
                                           int64_t dlogits_stride, void* stream);

// moe_few.cu
int64_t few_workspace_bytes(const fo_moe_few_desc& d);
fo_status launch_moe_few(const fo_moe_few_desc& d, const void* x, int64_t x_stride,
                         const void* router, const void* W1, const void* S1, const void* W2,
                         const void* S2, void* y, int64_t y_stride, void* workspace,
                         int32_t* dev_status, void* stream);

}  // namespace fo
