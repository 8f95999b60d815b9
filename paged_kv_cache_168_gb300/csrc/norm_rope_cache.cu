// norm_rope_cache.cu -- norms of q and k for each head before the rotary positions and the cache write
// (rope_cache.cuh).
#include "rope_cache.cuh"

namespace pkv {

cudaError_t launch_norm_rope_cache(const RopeParams& p, int act_dtype, bool i8, int sms, cudaStream_t stream) {
  return launch<true>(p, act_dtype, i8, sms, stream);
}

}  // namespace pkv
