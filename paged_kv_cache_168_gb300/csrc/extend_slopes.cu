// extend_slopes.cu -- attention of new tokens with scores that fall with distance (extend_tc.cuh).
#include "extend_tc.cuh"

namespace pkv {

cudaError_t launch_extend_slopes(const ExtendParams& p, void* workspace, int sms, int act_dtype, int head_size, bool i8,
                             cudaStream_t stream) {
  return launch<kSlope>(p, workspace, sms, act_dtype, head_size, i8, stream);
}

}  // namespace pkv
