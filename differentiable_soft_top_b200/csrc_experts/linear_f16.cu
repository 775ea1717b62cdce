// linear_f16.cu -- the experts' products for fp16 (linear.cuh).
#include "linear.cuh"

namespace lapsum {

cudaError_t linear_init_f16() { return init_as<__half>(); }
cudaError_t launch_linear_fwd_f16(const Product& p, int sms, cudaStream_t st) { return fwd_as<__half>(p, sms, st); }
cudaError_t launch_linear_dx_f16(const Product& p, int sms, cudaStream_t st) { return dx_as<__half>(p, sms, st); }
cudaError_t launch_linear_dweight_f16(const Product& p, int sms, cudaStream_t st) {
  return dweight_as<__half>(p, sms, st);
}

}  // namespace lapsum
