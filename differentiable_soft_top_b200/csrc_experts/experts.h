// experts.h -- host-side interface between the C ABI (experts_abi.cu) and the
// kernels of the experts' operators.  Not part of the public boundary.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "lapsum_experts.h"
#include "launch.h"

namespace lapsum {

struct RouteFwd {
  const void* scores;
  int dtype;
  int64_t tokens, stride;
  int experts, k, score;
  const float* bias;
  int groups, groups_kept, group_top, renormalize;
  float scale;
  float* weights;
  int32_t* chosen;
  bool vec, bias_vec;  // set by the launcher
};
cudaError_t launch_route_fwd(RouteFwd a, cudaStream_t st);

struct RouteBwd {
  const void* scores;
  int dtype;
  int64_t tokens, stride;
  int experts, k, score;
  const float* bias;
  int renormalize;
  float scale;
  const int32_t* chosen;
  const float* weights;
  const float* grad_weights;
  void* grad;
  int64_t grad_stride;
  bool vec, bias_vec, grad_vec;  // set by the launcher
};
cudaError_t launch_route_bwd(RouteBwd a, cudaStream_t st);

size_t plan_workspace(int64_t slots, int experts);
cudaError_t launch_plan(const int32_t* chosen, int64_t slots, int experts, int32_t* offsets, int32_t* rows,
                        int32_t* slot_of, void* ws, cudaStream_t st);
cudaError_t launch_dispatch(const void* x, int dtype, int64_t tokens, int k, int64_t dim, int64_t x_stride,
                            const int32_t* slot_of, void* out, int64_t out_stride, int sms, cudaStream_t st);
cudaError_t launch_combine(const void* y, int dtype, int64_t tokens, int k, int64_t dim, int64_t y_stride,
                           const float* weights, const int32_t* rows, const void* residual, int64_t res_stride,
                           void* out, int64_t out_stride, int sms, cudaStream_t st);
cudaError_t launch_combine_bwd(const void* grad, int dtype, int64_t tokens, int k, int64_t dim, int64_t grad_stride,
                               const void* y, int64_t y_stride, const float* weights, const int32_t* rows,
                               const int32_t* slot_of, void* grad_y, int64_t grad_y_stride, float* grad_weights,
                               int sms, cudaStream_t st);

// One launch of the experts' products (linear.cuh).
struct Product {
  int64_t rows;
  int experts, activation;
  int64_t in, out;             // of the weights
  const int32_t* offsets;      // or null: one expert owns all rows
  const void* x;               // forward, weight gradient: [rows, in]
  int64_t x_stride;
  const void* grad_h;          // gradients: [rows, out]
  int64_t grad_h_stride;
  const void* weight;          // forward, input gradient
  const void* bias;
  const void* residual;
  int64_t residual_stride;
  void* y;                     // output of each direction
  int64_t y_stride;
  void* preact;
  int64_t preact_stride;
  uint32_t* status;
  uint32_t polls;              // of a bounded device wait
  int starve;                  // test knob: copy nothing
};
// kernel attributes, once per device
cudaError_t exchange_init();
cudaError_t linear_init_bf16();
cudaError_t linear_init_f16();
cudaError_t launch_linear_fwd_bf16(const Product& p, int sms, cudaStream_t st);
cudaError_t launch_linear_fwd_f16(const Product& p, int sms, cudaStream_t st);
cudaError_t launch_linear_dx_bf16(const Product& p, int sms, cudaStream_t st);
cudaError_t launch_linear_dx_f16(const Product& p, int sms, cudaStream_t st);
cudaError_t launch_linear_dweight_bf16(const Product& p, int sms, cudaStream_t st);
cudaError_t launch_linear_dweight_f16(const Product& p, int sms, cudaStream_t st);

size_t act_bwd_workspace(int64_t rows, int experts, int64_t out);
cudaError_t launch_act_bwd(const void* grad_y, int bf16, int64_t rows, int64_t out, int64_t grad_y_stride,
                           const void* preact, int64_t preact_stride, int experts, const int32_t* offsets,
                           int activation, void* grad_h, int64_t grad_h_stride, void* grad_bias, void* ws, int sms,
                           cudaStream_t st);

}  // namespace lapsum
