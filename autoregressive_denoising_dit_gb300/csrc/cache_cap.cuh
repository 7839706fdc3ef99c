// The score cap of the cache operators: cap log2(e) tanh(scale s / cap) of raw
// products s, to f32's relative accuracy whatever the cap, so that a cap far
// above the scores leaves them as they are.
//
// With x = s inv, inv = scale / cap, and z = x^2:
//   |x| <= 1   s P(z), P = scale log2(e) tanh(sqrt z) / sqrt z interpolated at the
//              Chebyshev points of [0, 1] with 7 coefficients (5e-8 of P).  The cap
//              enters by inv alone, and where inv underflows P is its constant.
//   |x| > 1    cap log2(e) (1 - a) / (1 + a), a = exp(-2 |x|), which does not
//              cancel there (for small x it would lose 2^-22 of the cap).
// A score's value then depends on the score alone, not on which of the two forms
// the rest of its warp needs.  Where the cap is at most kCapLow, 2^-21 of it is
// below 2^-14, an eighth of a weight's rounding to f16, and many-row kernels take
// the cheaper cap log2(e) (1 - 2 / (1 + exp(2 x))) for all scores of a warp that has
// one over the cap (prefix case with a cap of 5 and scores of deviation 8: 1175
// us, with the two forms 1916).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "psv_device.cuh"

namespace psv {

constexpr float kCapLow = 128.0f;

struct CapForm {
  float inv, c2;    // scale / cap and cap log2(e), both kept finite
  float two;        // 2 log2(e) inv, for caps up to kCapLow; else 0
  float2 poly[7];   // P's coefficients, each twice
};

// Sets `f` for a cap > 0.
void set_cap_form(CapForm& f, float scale, float cap);

__device__ __forceinline__ uint64_t pair_bits(const float2& v) { return *reinterpret_cast<const uint64_t*>(&v); }

// N scores (an even number) of which none passes the cap.
template <int N>
__device__ __forceinline__ void cap_within(float* s, const CapForm& f) {
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    uint64_t v, z, y, inv;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(s[c]), "f"(s[c + 1]));
    asm("mov.b64 %0, {%1, %1};" : "=l"(inv) : "f"(f.inv));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(z) : "l"(v), "l"(inv));
    asm("mul.rn.f32x2 %0, %0, %0;" : "+l"(z));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(z), "l"(pair_bits(f.poly[6])), "l"(pair_bits(f.poly[5])));
#pragma unroll
    for (int k = 4; k >= 0; --k) asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(y) : "l"(z), "l"(pair_bits(f.poly[k])));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(v) : "l"(y));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(s[c]), "=f"(s[c + 1]) : "l"(v));
  }
}

// N scores of which some may pass the cap.
template <int N>
__device__ __forceinline__ void cap_any(float* s, const CapForm& f) {
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const float x = __fmul_rn(s[c], f.inv), z = __fmul_rn(x, x);
    float y = __fmaf_rn(z, f.poly[6].x, f.poly[5].x);
#pragma unroll
    for (int k = 4; k >= 0; --k) y = __fmaf_rn(y, z, f.poly[k].x);
    const float a = fast_exp2(-2.885390081777927f * fabsf(x));
    const float t = (1.0f - a) * fast_rcp(1.0f + a);
    s[c] = fabsf(x) <= 1.0f ? __fmul_rn(s[c], y) : copysignf(f.c2 * t, x);
  }
}

// The cheaper form (f.two > 0).
template <int N>
__device__ __forceinline__ void cap_low(float* s, const CapForm& f) {
#pragma unroll
  for (int c = 0; c < N; ++c) s[c] = fmaf(-2.0f * f.c2, fast_rcp(1.0f + fast_exp2(s[c] * f.two)), f.c2);
}

}  // namespace psv
