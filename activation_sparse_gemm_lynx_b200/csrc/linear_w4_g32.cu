// linear_w4_g32.cu -- lynx_linear_w4 for scale groups of 32.
#include "linear_w4.cuh"

namespace lynx {

cudaError_t launch_linear_w4_g32(const LinearW4Launch& p, int sms, cudaStream_t s) {
  return launch_linear_w4_group<32>(p, sms, s);
}

}  // namespace lynx
