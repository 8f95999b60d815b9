// rope_cache.cu -- rotary positions on q and k and the cache write (rope_cache.cuh).
#include "rope_cache.cuh"

namespace pkv {

cudaError_t launch_rope_cache(const RopeParams& p, int act_dtype, bool i8, int sms, cudaStream_t stream) {
  return launch<false>(p, act_dtype, i8, sms, stream);
}

}  // namespace pkv
