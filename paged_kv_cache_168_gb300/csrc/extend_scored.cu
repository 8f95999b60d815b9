// extend_scored.cu -- attention of new tokens with capped scores, scores that fall with distance and spans of each
// query (extend_tc.cuh, kScored).
#include "extend_tc.cuh"

namespace pkv {

ScoreShape score_shape(float scale, float softcap, const float* slopes) {
  // tanh(y) / y in powers of y^2 on [0, 1]
  const double fit[6] = {0.9999994039535522, -0.3332904279232025, 0.13281433284282684, -0.051605675369501114,
                         0.016743116080760956, -0.0030670606065541506};
  const double half[4] = {0.999999463558197, -0.33326318860054016, 0.13190296292304993, -0.04440222680568695};    // the same on [0, 1/2]
  const double log2e = 1.4426950408889634;
  ScoreShape w;
  w.slopes = slopes;
  w.capped = softcap > 0.f;
  if (!w.capped) return w;
  w.cap_in = (float)((double)scale / softcap);
  w.cap_log2 = (float)(softcap * log2e);
  for (int i = 0; i < 6; ++i) w.poly[i] = (float)(fit[i] * softcap * log2e);
  for (int i = 0; i < 4; ++i) w.half[i] = (float)(half[i] * softcap * log2e);
  return w;
}

cudaError_t launch_extend_scored(const ExtendParams& p, void* workspace, int sms, int act_dtype, int head_size, bool i8,
                                 cudaStream_t stream) {
  return launch<true>(p, workspace, sms, act_dtype, head_size, i8, stream);
}

}  // namespace pkv
