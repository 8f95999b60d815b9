// extend_scored.cu -- attention of new tokens with shaped scores (extend_tc.cuh): which kernel a call takes, and those
// for caps and slopes together.
#include "extend_tc.cuh"

namespace pkv {

ScoreShape score_shape(float scale, float softcap, const float* slopes) {
  // tanh(y) / y in powers of y^2 on [0, 1]
  const double fit[6] = {0.9999994039535522, -0.3332904279232025, 0.13281433284282684, -0.051605675369501114,
                         0.016743116080760956, -0.0030670606065541506};
  // the same on [0, 3/4]
  const double near[5] = {0.999999463558197, -0.3332825303077698, 0.13258983194828033, -0.05005630478262901,
                          0.01292963232845068};
  const double log2e = 1.4426950408889634;
  ScoreShape w;
  w.slopes = slopes;
  w.capped = softcap > 0.f;
  if (!w.capped) return w;
  w.cap_in = (float)((double)scale / softcap);
  w.cap_out = (float)((double)softcap / scale);
  w.cap_log2 = (float)(softcap * log2e);
  for (int i = 0; i < 6; ++i) w.poly[i] = (float)(fit[i] * softcap * log2e);
  double in = w.cap_in;
  for (int i = 0; i < 5; ++i, in *= (double)w.cap_in * w.cap_in) {
    w.three_quarters[i] = (float)(near[i] * softcap * log2e);
    w.folded[i] = (float)(near[i] * softcap * log2e * in);
  }
  // (the fifth term, cap_in^9 in it, is the smallest; where it is a normal number the squares, up to 2^42 with those of
  // masked places, stay in range as well)
  w.folds = w.cap_in <= 0x1p10f && w.folded[4] >= 0x1p-120f;
  return w;
}

cudaError_t launch_extend_scored(const ExtendParams& p, void* workspace, int sms, int act_dtype, int head_size, bool i8,
                                 cudaStream_t stream) {
  const bool capped = p.shape.capped, sloped = p.shape.slopes != nullptr;
  if (!capped && !sloped) return launch_extend_spans(p, workspace, sms, act_dtype, head_size, i8, stream);
  if (!capped && !p.last_pos) return launch_extend_slopes(p, workspace, sms, act_dtype, head_size, i8, stream);
  const bool in_range = act_dtype == PA_F16 || i8 || p.shape.cap_log2 <= 80.f;
  if (!sloped && p.shape.folds && in_range) return launch_extend_cap(p, workspace, sms, act_dtype, head_size, i8, stream);
  return launch<kAny>(p, workspace, sms, act_dtype, head_size, i8, stream);
}

}  // namespace pkv
