// gated_device.h -- gfx950 numerics of the gated linear recurrence.
//
// Per token and channel, with kappa = c softplus(lam) of the channel:
//     l = -kappa sigma(ra),  a = e^l,  s = sqrt(1 - a^2),  b = s sigma(rx) u,  h' = a h + b.
// A slow channel has 1 - a near 1e-4 or less, so there a is formed as 1 - m from
// m = -expm1(l): the subtraction rounds once, without the bias that an exp near
// 1 carries through thousands of products, and 1 - a^2 = m (2 - m) keeps its
// relative accuracy where 1 - a*a would cancel.  A fast channel's a is the exponential
// itself: 1 - m would hold it to 2^-25 of 1, which is nothing of a at l = -17.
#pragma once

#include "s6_device.h"

namespace s6 {

// Two bf16 values in a word, the first in the low half (one instruction).
__device__ __forceinline__ uint32_t f32x2_to_bf16(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// a = e^y and m = 1 - a for y <= 0, relative errors about 2e-7 (a's beyond y = -4: 2^-24 |y|):
//   y > -0.35 : m = -y (1 + y/2 (1 + y/3 (1 + ... y/7))), truncation below 2e-8; a = 1 - m
//   otherwise : a = e^y; m = 1 - a, cancellation below 2^-24 * 0.7 / 0.3
// near: the caller knows the first to hold in the whole wave (kappa < 0.35 bounds -l, the
// usual case: a channel that forgets within a few tokens is rare), which saves 7 of some
// 40 instruction slots per element.
constexpr float kNearExp = 0.35f;
__device__ __forceinline__ void decay_pair(float y, bool near, float& a, float& m) {
  float p = __builtin_fmaf(y, 1.0f / 5040.0f, 1.0f / 720.0f);
  p = __builtin_fmaf(y, p, 1.0f / 120.0f);
  p = __builtin_fmaf(y, p, 1.0f / 24.0f);
  p = __builtin_fmaf(y, p, 1.0f / 6.0f);
  p = __builtin_fmaf(y, p, 0.5f);
  p = __builtin_fmaf(y, p, 1.0f);
  m = -y * p;
  a = 1.0f - m;
  if (!near) {
    float e = ex2(y * kLog2e);
    asm volatile("" : "+v"(e));  // a branch, not a select
    m = y > -kNearExp ? m : 1.0f - e;
    a = y > -kNearExp ? a : e;
  }
}

// The decay e^y of a whole run from the sum y of its l (-inf after a reset: exactly 0).  A
// product of the run's decays would lose the second-order terms that are below an ulp of 1,
// all with the same sign, which a channel of long memory adds up over the sequence.  Only a reset's
// is 0, the sign to drop an older state: one that underflows is the least normal number, nothing
// of a state that is a number, while an infinite or NaN one stays what it is.
constexpr float kLeastDecay = 1.17549435e-38f;
__device__ __forceinline__ float run_decay(float y) {
  float a, m;
  decay_pair(y, false, a, m);
  return y == -__builtin_inff() ? 0.0f : fmaxf(a, kLeastDecay);
}

// sigma(v) and 1 - sigma(v), each to a few ulp relative; saturates without NaN, a NaN stays one.
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.0f + ex2(-v * kLog2e)); }
__device__ __forceinline__ void sigmoid_pair(float v, float& sg, float& om) {
  // finite, so that e * sg is a number; of a NaN and a number, `minimum` takes the NaN
  const float e = ex2(__builtin_elementwise_minimum(-v * kLog2e, 126.0f));
  sg = rcp(1.0f + e);
  om = e * sg;
}

// Decay and input of one token: h' = a h + b.  slow: kappa < kNearExp in the whole wave.
// l: the decay's logarithm (not that of a reset).
__device__ __forceinline__ void gated_token(float ra, float rx, float u, float kappa, bool slow, bool reset, float& a,
                                            float& b, float& l) {
  l = -kappa * sigmoid(ra);
  float m;
  decay_pair(l, slow, a, m);
  const float s = __builtin_amdgcn_sqrtf(m * (2.0f - m));
  const float x = sigmoid(rx) * u;
  a = reset ? 0.0f : a;
  b = reset ? x : s * x;
}

// The same with what the backward needs:
//   s, sx = sigma(rx), ox = 1 - sx, oa = 1 - sigma(ra), l (both 0 on a reset), and
//   q = a^2 l / s, 0 where s is 0 (l/s -> 0 with l) and on a reset.
struct GatedGrad {
  float a, s, sx, ox, oa, l, q;
};
__device__ __forceinline__ GatedGrad gated_grad(float ra, float rx, float kappa, bool slow, bool reset) {
  GatedGrad g;
  float sa, oa;
  sigmoid_pair(ra, sa, oa);
  sigmoid_pair(rx, g.sx, g.ox);
  const float l = -kappa * sa;
  float a, m;
  decay_pair(l, slow, a, m);
  const float s2 = m * (2.0f - m);
  const float rs = __builtin_amdgcn_rsqf(fmaxf(s2, 1.0e-37f));  // l and s2 are 0 together, then so are s and q
  const float s = s2 * rs;
  const float q = a * a * (l * rs);
  g.a = reset ? 0.0f : a;
  g.s = reset ? 1.0f : s;
  g.l = reset ? 0.0f : l;
  g.oa = reset ? 0.0f : oa;  // (a NaN gate left out by a reset does not reach its gradient)
  g.q = reset ? 0.0f : q;
  return g;
}

// d kappa / d lam / kappa = sigma(lam) / softplus(lam); the sums of e = dL/dl * l times this are dlam.
// Where softplus underflows, e^lam / e^lam = 1.
__device__ __forceinline__ float dlam_factor(float lam) {
  const float sp = softplus(lam);
  return sp > 0.0f ? sigmoid(lam) / sp : 1.0f;
}

// SiLU(z) and its derivative sigma(z) (1 + z (1 - sigma(z))).
__device__ __forceinline__ void silu_pair(float z, float& f, float& df) {
  float sg, om;
  sigmoid_pair(z, sg, om);
  f = z * sg;
  df = sg * __builtin_fmaf(z, om, 1.0f);
}

}  // namespace s6
