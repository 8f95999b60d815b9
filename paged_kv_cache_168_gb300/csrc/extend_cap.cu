// extend_cap.cu -- attention of new tokens with capped scores (extend_tc.cuh).
#include "extend_tc.cuh"

namespace pkv {

cudaError_t launch_extend_cap(const ExtendParams& p, void* workspace, int sms, int act_dtype, int head_size, bool i8,
                             cudaStream_t stream) {
  return launch<kCap>(p, workspace, sms, act_dtype, head_size, i8, stream);
}

}  // namespace pkv
