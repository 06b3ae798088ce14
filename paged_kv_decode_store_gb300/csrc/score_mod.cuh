// Attention scores after the dot product, shared by the decode and prefill
// kernels: capped by a tanh, biased by distance, opened to a prefix.
//   s' = cap * tanh(s / cap)            (softcap > 0)
//   s'' = s' - slope_h * |p - j|        (alibi_slopes)
// in the log2 domain: cap and slope come multiplied by log2(e), the softmax
// scale and 1 / cap are one factor on the raw dot product.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace pkvd {

__device__ __forceinline__ float mod_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float mod_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(y) = 1 - 2 / (1 + e^2y): right at both ends (e^2y = 0 or inf) and to a
// few 2^-24 of 1 everywhere, hence relative to the value only where |y| is
// not small.
__device__ __forceinline__ float tanh_large(float y) {
  return fmaf(-2.f, mod_rcp(1.f + mod_ex2(y * 2.885390081777927f)), 1.f);   // 2 log2(e)
}

// tanh(y) / y as a polynomial in z = y^2 (relative minimax, found by an
// exchange iteration): off by 5.9e-7 of the value for |y| <= 1 with six terms,
// by 7.2e-6 for |y| <= kTanhNear with four.  tanh's nearest pole is at z =
// -(pi / 2)^2, so each term gains a factor of about 12 on [0, 1].
#define PKVD_TANH_RATIO4 {0.999992801f, -0.332866126f, 0.128479621f, -0.0370293619f}
constexpr float kTanhNear = 0.707f;

__device__ __forceinline__ float tanh_ratio6(float z) {
  float r = fmaf(z, -0.00306706033f, 0.0167431151f);
  r = fmaf(z, r, -0.051605674f);
  r = fmaf(z, r, 0.132814339f);
  r = fmaf(z, r, -0.333290424f);
  return fmaf(z, r, 0.999999414f);
}

// tanh to 1e-6 of the value: a score's error stays relative to the score
// whatever the cap.
__device__ __forceinline__ float tanh_fast(float y) {
  const float z = y * y;
  const float small = y * tanh_ratio6(z), large = tanh_large(y);
  return z <= 1.f ? small : large;
}

// The score of a raw dot product, in log2 units, without its bias.
template <bool EXACT>
__device__ __forceinline__ float capped(float raw, float scale_log2, const ScoreMod& m) {
  if (m.cap_in == 0.f) return raw * scale_log2;
  const float y = raw * m.cap_in;
  return (EXACT ? tanhf(y) : tanh_fast(y)) * m.cap_out_log2;
}

// -slope * log2(e) of a query head, 0 without slopes.  At most 2^90 either way,
// so that its product with any distance is finite (an infinite one makes NaN at
// distance 0, or where a row starts with keys at -inf): a key is then 2^90
// ahead of the next, which no other score makes up for.
__device__ __forceinline__ float bias_slope(const ScoreMod& m, int head) {
  return m.slopes ? fminf(fmaxf(-m.slopes[head] * 1.4426950408889634f, -0x1p90f), 0x1p90f) : 0.f;
}

// Exponent that the mma.sync paths add to a weight of at most 1 before it is
// rounded to the cache's type (the sum of the weights has it too, so it
// cancels): f16 is normal down to 2^-14 only, and many small weights beside a
// large one have to add up to what they are.
template <typename T>
constexpr float kWeightLift = std::is_same<T, __half>::value ? 15.f : 0.f;

// Tokens of sequence `seq` that every row may see, clamped to its length.
__device__ __forceinline__ int prefix_of(const ScoreMod& m, int seq, int klen) {
  return m.prefix ? min(max(m.prefix[seq], 0), klen) : 0;
}

}  // namespace pkvd
