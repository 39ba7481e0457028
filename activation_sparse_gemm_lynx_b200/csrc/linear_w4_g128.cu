// linear_w4_g128.cu -- lynx_linear_w4 for scale groups of 128.
#include "linear_w4.cuh"

namespace lynx {

cudaError_t launch_linear_w4_g128(const LinearW4Launch& p, int sms, cudaStream_t s) {
  return launch_linear_w4_group<128>(p, sms, s);
}

}  // namespace lynx
