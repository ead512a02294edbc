// Activations and the 8-bit checkpoint format of the linear operators
// (mx_gemm_act, mx_checkpoint_*, mx_quantize_saved): binary32 device
// functions.
//
// With z = 2u = 2 sqrt(2/pi) (x + 0.044715 x^3) for the tanh form of GELU and
// z = x for SiLU, and s = 1 / (1 + exp(-z)), (1 + tanh u) / 2 = s, so
//   act(x)  = x s,
//   act'(x) = s + x z'(x) s (1 - s).
// exp2 and the reciprocal are the hardware's (each within 1 ulp), not the
// packers' bit-exact contract (mx_device.h), which takes several times the
// instructions.  The exponent carries at most four roundings, an error of
// 4 |z| 2^-24 in exp(-z); the exponential, the sum, the reciprocal and the last
// product add 6 2^-24: act is within (4 |z| + 6) 2^-24 of itself.  In act' the
// largest error is the 2 2^-24 of s where it is next to 1, times x z' (33 for
// GELU at z = 17): under 2^-17.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"

namespace mx {

enum Act { kActNone = 0, kActGelu = 1, kActSilu = 2 };

// 1 / (1 + 2^(-t))
__device__ __forceinline__ float sigmoid2(float t) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-t));
#else
  return t;
#endif
}

// z(x) log2(e): the exponent of sigmoid2
template <int ACT>
__device__ __forceinline__ float act_exponent(float x) {
  if constexpr (ACT == kActGelu) {
    const float A = 0x1.26aec2p+1f;   // 2 sqrt(2/pi) log2(e)
    const float B = 0x1.a5a7d0p-4f;   // 0.044715 A
    return x * __builtin_fmaf(x * x, B, A);
  } else {
    return x * 0x1.715476p+0f;  // log2(e)
  }
}

template <int ACT>
__device__ __forceinline__ float act_value(float x) {
  if constexpr (ACT == kActNone) return x;
  return x * sigmoid2(act_exponent<ACT>(x));
}

template <int ACT>
__device__ __forceinline__ float act_slope(float x) {
  if constexpr (ACT == kActNone) return 1.0f;
  const float s = sigmoid2(act_exponent<ACT>(x));
  // s (1 - s): exactly 0 where s rounds to 1 (z past 17) or to 0 (z below
  // about -88).  Its other factor overflows only for |z| far beyond both, so
  // the product is the one whose zeros win
  const float w = __builtin_fmaf(-s, s, s);
  float xz = x;
  if constexpr (ACT == kActGelu) {
    const float C = 0x1.988454p+0f, D = 0x1.b6676cp-3f;  // z' = C + D x^2
    xz = x * __builtin_fmaf(x * x, D, C);
  }
#if defined(__HIP_DEVICE_COMPILE__)
  float term;  // xz w, 0 wherever w is 0
  asm("v_mul_legacy_f32 %0, %1, %2" : "=v"(term) : "v"(xz), "v"(w));
  return term + s;
#else
  return xz * w + s;
#endif
}

// 2^(byte - 127) of an E8M0 scale; 0 gives 2^-127 (a subnormal), 0xff NaN, so
// that every code of a NaN block decodes to NaN.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 0xffu ? 0x7fc00000u : byte << 23);
}

// Four E4M3 codes (one dword) times a scale.
__device__ __forceinline__ void e4m3_decode4(uint32_t w, float scale, float (&v)[4]) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef float f2 __attribute__((ext_vector_type(2)));
  const f2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const f2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  v[0] = lo.x * scale;
  v[1] = lo.y * scale;
  v[2] = hi.x * scale;
  v[3] = hi.y * scale;
#endif
}

// N values to E4M3 codes (four a dword) under scale byte `s` (RCEIL: |v| <=
// 448 2^X, so nothing saturates); the values may be rescaled in place.  The
// conversion divides by 2^X exactly; a block with X = -127, whose scale is no
// normal binary32, is converted as (v 2^64) / 2^-63 (only a wavefront that
// holds such a block pays), and a NaN block's codes are 0.
template <int N>
__device__ __forceinline__ void e4m3_encode(float (&v)[N], uint32_t s, uint32_t (&w)[N / 4]) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef short s2 __attribute__((ext_vector_type(2)));
  const bool tiny = s == 0u;
  const float sc = __uint_as_float((tiny ? 64u : (s == 0xffu ? 127u : s)) << 23);
  if (__builtin_amdgcn_ballot_w64(tiny) != 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = tiny ? v[i] * 0x1p64f : v[i];
  }
#pragma unroll
  for (int d = 0; d < N / 4; ++d) {
    s2 q = {0, 0};
    q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(q, v[4 * d + 0], v[4 * d + 1], sc, false);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(q, v[4 * d + 2], v[4 * d + 3], sc, true);
    w[d] = s == 0xffu ? 0u : __builtin_bit_cast(uint32_t, q);
  }
#endif
}

// Largest |v| as a bit pattern (a NaN sorts above infinity).  Positive
// values order as signed integers, negative ones as unsigned integers above
// every positive one, so two integer maxima (three operands an instruction)
// need no absolute values.
template <int N>
__device__ __forceinline__ uint32_t abs_max(const float (&v)[N]) {
  int32_t pos = 0;
  uint32_t neg = 0u;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t b = __float_as_uint(v[i]);
    pos = pos > (int32_t)b ? pos : (int32_t)b;
    neg = neg > b ? neg : b;
  }
  neg &= 0x7fffffffu;
  return (uint32_t)pos > neg ? (uint32_t)pos : neg;
}

// One step of a reduction within a row of 16 lanes: the value of the lane
// that DPP control `CTRL` names.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_move(uint32_t v) {
#if defined(__HIP_DEVICE_COMPILE__)
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
#else
  return v;
#endif
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppHalfMirror = 0x141, kDppRor4 = 0x124, kDppRor8 = 0x128;

__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Maximum over the 4 (8) lanes of an aligned group.
__device__ __forceinline__ uint32_t max_over4(uint32_t v) {
  v = max_u32(v, dpp_move<kDppXor1>(v));
  return max_u32(v, dpp_move<kDppXor2>(v));
}
__device__ __forceinline__ uint32_t max_over8(uint32_t v) {
  v = max_over4(v);
  return max_u32(v, dpp_move<kDppHalfMirror>(v));  // lane i of 8 takes lane 7 - i's: the other four
}

}  // namespace mx
