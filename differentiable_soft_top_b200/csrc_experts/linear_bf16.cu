// linear_bf16.cu -- the experts' products for bf16 (linear.cuh).
#include "linear.cuh"

namespace lapsum {

cudaError_t linear_init_bf16() { return init_as<__nv_bfloat16>(); }
cudaError_t launch_linear_fwd_bf16(const Product& p, int sms, cudaStream_t st) { return fwd_as<__nv_bfloat16>(p, sms, st); }
cudaError_t launch_linear_dx_bf16(const Product& p, int sms, cudaStream_t st) { return dx_as<__nv_bfloat16>(p, sms, st); }
cudaError_t launch_linear_dweight_bf16(const Product& p, int sms, cudaStream_t st) {
  return dweight_as<__nv_bfloat16>(p, sms, st);
}

}  // namespace lapsum
