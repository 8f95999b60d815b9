// extend_tc.cu -- attention of a chunk of new tokens per sequence (extend_tc.cuh).
#include "extend_tc.cuh"

namespace pkv {

size_t extend_workspace(int num_seqs, int num_tokens, int num_kv_heads, int group, int max_query_len, int head_size,
                        int sms, bool scored) {
  size_t bytes;
  lay_out(nullptr, num_seqs, num_tokens, num_kv_heads, group, max_query_len, head_size, sms, scored, &bytes);
  return bytes;
}

cudaError_t launch_extend(const ExtendParams& p, void* workspace, int sms, int act_dtype, int head_size, bool i8,
                          cudaStream_t stream) {
  return launch<kNone>(p, workspace, sms, act_dtype, head_size, i8, stream);
}

}  // namespace pkv
