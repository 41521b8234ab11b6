// Launchers of the operators around the expert layer's products, called by
// their C entry points after the arguments have been checked.
#pragma once

#include <cstdint>

#include "fo.h"

namespace fo {

constexpr int kCombineSlots = 32;     // slots of a token
constexpr int kCheckpointBlock = 32;  // values of a checkpoint that share a scale

// block_combine.cu
fo_status launch_combine(const void* rows, fo_type type, int64_t table_rows, int64_t hidden,
                         int64_t row_stride, const int32_t* token_row, const float* weights,
                         int64_t tokens, int32_t top_k, void* y, fo_type y_type,
                         int64_t y_stride, int32_t* dev_status, void* stream);
fo_status launch_combine_backward(const void* dy, fo_type dy_type, int64_t dy_stride,
                                  const void* rows, fo_type type, int64_t table_rows,
                                  int64_t hidden, int64_t row_stride, const int32_t* token_row,
                                  const int32_t* row_token, const float* weights,
                                  int64_t tokens, int32_t top_k, void* drows,
                                  int64_t drows_stride, float* dweights, int32_t* dev_status,
                                  void* stream);

// block_act.cu
fo_status launch_gated_act(const void* u, fo_type type, int64_t rows, int64_t inter,
                           int64_t u_stride, fo_activation act, void* h, int64_t h_stride,
                           void* codes, void* scales, void* stream);
fo_status launch_gated_act_backward(const void* dh, fo_type type, int64_t rows, int64_t inter,
                                    int64_t dh_stride, fo_activation act, const void* codes,
                                    const void* scales, void* du, int64_t du_stride,
                                    void* stream);

// block_norm.cu
struct NormArgs {
  const void* x;          // the block's output
  const void* residual;   // NULL: none
  const void* post;       // NULL: no norm after the block
  const void* gate;       // NULL: none
  const void* pre;        // NULL: no norm before the next block
  int64_t x_stride, residual_stride, gate_stride;
  void* sum;              // the stream after the block; NULL: not written
  void* y;
  int64_t sum_stride, y_stride;
  float* post_rstd;
  float* pre_rstd;
  int32_t tokens, hidden;
  int32_t gate_rows;      // consecutive tokens that share a row of the gate
  int32_t params_f32;
  float scale, eps;
};
fo_status launch_block_norm(const NormArgs& a, fo_type type, fo_type stream_type, void* stream);

// block_norm_backward.cu
struct NormBackArgs {
  NormArgs f;             // the forward call's inputs; post_rstd and pre_rstd are read
  const void* dsum;       // NULL: zeros
  const void* dy;         // NULL where pre is
  int64_t dsum_stride, dy_stride;
  void* dx;
  void* dresidual;
  int64_t dx_stride, dresidual_stride;
  void* dpost;
  void* dgate;
  void* dpre;
  float* workspace;
};
int64_t block_norm_workspace_bytes(int64_t tokens, int64_t hidden, int64_t gates);
fo_status launch_block_norm_backward(const NormBackArgs& a, fo_type type, fo_type stream_type,
                                     int64_t gates, void* stream);

}  // namespace fo
