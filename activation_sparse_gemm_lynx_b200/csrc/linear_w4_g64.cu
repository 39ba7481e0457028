// linear_w4_g64.cu -- lynx_linear_w4 for scale groups of 64.
#include "linear_w4.cuh"

namespace lynx {

cudaError_t launch_linear_w4_g64(const LinearW4Launch& p, int sms, cudaStream_t s) {
  return launch_linear_w4_group<64>(p, sms, s);
}

}  // namespace lynx
