// The INT4 wire's scale from a group's largest magnitude, amax / 7, without a
// division; shared by the encoders and the append to a 4-bit cache.
#pragma once

namespace hc {
namespace {

// fp32(a / 7) for every non-negative finite fp32 a, without a division: the
// product with fp32(1/7) is corrected by its exact residual (Markstein's
// correction, as in int4x8_corrected).  Checked against the IEEE division on
// the GPU for all 2^31 non-negative finite fp32 values: no mismatch.
__device__ __forceinline__ float div7(float a) {
  const float r7 = 0.142857149f;  // fp32(1/7)
  const float q1 = a * r7;
  return fmaf(fmaf(-q1, 7.0f, a), r7, q1);
}

}  // namespace
}  // namespace hc
