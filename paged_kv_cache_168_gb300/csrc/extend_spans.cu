// extend_spans.cu -- attention of new tokens with spans of positions for each query and plain scores (extend_tc.cuh).
#include "extend_tc.cuh"

namespace pkv {

cudaError_t launch_extend_spans(const ExtendParams& p, void* workspace, int sms, int act_dtype, int head_size, bool i8,
                             cudaStream_t stream) {
  return launch<kSpans>(p, workspace, sms, act_dtype, head_size, i8, stream);
}

}  // namespace pkv
