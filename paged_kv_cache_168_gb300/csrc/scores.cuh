// scores.cuh -- what happens to a score between q.k and the softmax where it is
// capped or falls with distance: the same arithmetic in every kernel.
//
// With y = scale q.k / c, a cap c makes c tanh(y) of it.  Up to |y| = 1 that is y
// P(y^2) with a polynomial P of degree 5, fitted to tanh(y) / y by weighted least
// squares until its relative error is level (6.1e-7); beyond, c (1 - 2 / (1 +
// e^(2y))), whose absolute error of a few 2^-24 c is as small beside a result of
// at least 0.76 c.  Everything is in base-2 units (times log2 e) and fp32.  Up to
// |y| = 3/4 five terms do as well (5.9e-7): scores are rarely nearer to their cap.
#pragma once

#include <cuda_runtime.h>

#include "kernels.h"

namespace pkv {
namespace score {

constexpr float kLog2e = 1.4426950408889634f;

// c tanh(y) for |y| <= 1.
__device__ __forceinline__ float near_cap(const ScoreShape& w, float y) {
  const float s = y * y;
  float v = w.poly[5];
#pragma unroll
  for (int k = 4; k >= 0; --k) v = fmaf(v, s, w.poly[k]);
  return v * y;
}

// The same for two |y| <= 3/4, a step less and two operations an instruction; a and b are multiplied by unit first, and
// more is added to the results.
__device__ __forceinline__ void nearer_cap2(const ScoreShape& w, float unit, float more, float& a, float& b, float& ca, float& cb) {
  uint64_t y, u, s, v, c;
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(a), "f"(b));
  asm("mov.b64 %0, {%1, %1};" : "=l"(u) : "f"(unit));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(y) : "l"(u));
  asm("mul.rn.f32x2 %0, %1, %1;" : "=l"(s) : "l"(y));
  asm("mov.b64 %0, {%1, %1};" : "=l"(v) : "f"(w.three_quarters[4]));
#pragma unroll
  for (int k = 3; k >= 0; --k) {
    asm("mov.b64 %0, {%1, %1};" : "=l"(c) : "f"(w.three_quarters[k]));
    asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(v) : "l"(s), "l"(c));
  }
  asm("mov.b64 %0, {%1, %1};" : "=l"(c) : "f"(more));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(v) : "l"(y), "l"(c));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(y));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(ca), "=f"(cb) : "l"(v));
}

// c tanh(y) for any y (NaN stays NaN, infinities become -c and c).
__device__ __forceinline__ float any_cap(const ScoreShape& w, float y) {
  const float v = near_cap(w, y);
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fminf(y * (2.f * kLog2e), 64.f)));
  return fabsf(y) > 1.f ? w.cap_log2 * (1.f - __fdividef(2.f, 1.f + e)) : v;
}

// any_cap as a call, for where it is rarely needed: inlined it takes the place of code that is (8-bit decode of 8 columns:
// 715 us against 691).
static __device__ __noinline__ float any_cap_call(const ScoreShape& w, float y) { return any_cap(w, y); }

}  // namespace score
}  // namespace pkv
