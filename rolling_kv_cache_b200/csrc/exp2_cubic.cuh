// 2^x on the FMA pipe for the attention kernels' softmax.
#pragma once

#include "ptx.cuh"

namespace rc {

// 2^x for a pair of lanes on the FMA pipe, in packed f32x2 steps: n =
// round(x) by the 1.5 * 2^23 shift, f = x - n in [-1/2, 1/2], 2^f by a cubic,
// n added to the exponent field. The cubic's coefficients are the minimax fit
// of the relative error on [-1/2, 1/2] (Remez exchange in fp64, each rounded
// to fp32): relative error within 7.5e-5, below the 2^-9 of the bf16 P it
// feeds. x is clamped at -126 so the exponent field cannot wrap; below that
// the result is at most 2^-126, as the SFU's flush-to-zero gives 0.
__device__ __forceinline__ float2 exp2_cubic2(float2 x) {
  x.x = fmaxf(x.x, -126.f);
  x.y = fmaxf(x.y, -126.f);
  const float2 t = ptx::fadd2(x, make_float2(12582912.f, 12582912.f));
  const float2 n = ptx::fadd2(t, make_float2(-12582912.f, -12582912.f));
  const float2 f = ptx::ffma2(n, make_float2(-1.f, -1.f), x);
  float2 q = ptx::ffma2(make_float2(5.517166853e-02f, 5.517166853e-02f), f,
                        make_float2(2.426111251e-01f, 2.426111251e-01f));
  q = ptx::ffma2(q, f, make_float2(6.932609677e-01f, 6.932609677e-01f));
  q = ptx::ffma2(q, f, make_float2(9.999280572e-01f, 9.999280572e-01f));
  return make_float2(__uint_as_float(__float_as_uint(q.x) + (__float_as_uint(t.x) << 23)),
                     __uint_as_float(__float_as_uint(q.y) + (__float_as_uint(t.y) << 23)));
}
// pairs k of a 16-pair chunk with (k % 8) < kCubicPairs take exp2_cubic2;
// the rest the SFU's ex2 (16 per clock per SM, the bound of the exponential
// phase when it runs alone)
constexpr int kCubicPairs = 2;

}  // namespace rc
