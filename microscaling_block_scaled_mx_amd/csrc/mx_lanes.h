// Eight values a lane: loads and stores of bf16 or binary32 rows, sums over a
// wavefront, and the packing of 32-element blocks held by four adjacent lanes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_act.h"
#include "mx_device.h"

namespace mx {

// Eight consecutive values as they lie in memory: one 16-byte load of bf16, two
// of binary32.
template <int F32>
struct Lane8 {
  uint4 w[F32 ? 2 : 1];
};
template <int F32>
__device__ __forceinline__ Lane8<F32> lane8_load(const void* base, int64_t at) {
  Lane8<F32> q;
  if constexpr (F32) {
    const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(base) + at);
    q.w[0] = src[0];
    q.w[1] = src[1];
  } else {
    q.w[0] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + at);
  }
  return q;
}
template <int F32>
__device__ __forceinline__ Lane8<F32> lane8_zero() {
  Lane8<F32> q;
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) q.w[i] = make_uint4(0u, 0u, 0u, 0u);
  return q;
}
template <int F32>
__device__ __forceinline__ void lane8_values(const Lane8<F32>& q, float (&v)[8]) {
  if constexpr (F32) {
    const uint32_t a[8] = {q.w[0].x, q.w[0].y, q.w[0].z, q.w[0].w, q.w[1].x, q.w[1].y, q.w[1].z, q.w[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(a[i]);
  } else {
    const uint32_t a[4] = {q.w[0].x, q.w[0].y, q.w[0].z, q.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(a[i]);
      v[2 * i + 1] = bf16_hi(a[i]);
    }
  }
}
// The same from a type known at run time only (uniform).
__device__ __forceinline__ void lane8_read(const void* base, int64_t at, int f32, float (&v)[8]) {
  if (f32) lane8_values<1>(lane8_load<1>(base, at), v);
  else lane8_values<0>(lane8_load<0>(base, at), v);
}
__device__ __forceinline__ uint4 lane8_bf16(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void lane8_store(void* base, int64_t at, int f32, const float (&v)[8]) {
  if (f32) {
    float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + at);
    dst[0] = make_float4(v[0], v[1], v[2], v[3]);
    dst[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(base) + at) = lane8_bf16(v);
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp_float(float v) {
  return __uint_as_float(dpp_move<CTRL>(__float_as_uint(v)));
}
constexpr int kDppMirror = 0x140;  // lane i of 16 takes lane 15 - i's

// Sum over the 64 lanes, the same bits in each (every step adds a pair's two
// values, in either order).  All lanes take part.
__device__ __forceinline__ float wave_sum(float v) {
#if defined(__HIP_DEVICE_COMPILE__)
  v = v + dpp_float<kDppXor1>(v);
  v = v + dpp_float<kDppXor2>(v);
  v = v + dpp_float<kDppHalfMirror>(v);
  v = v + dpp_float<kDppMirror>(v);
  const uint32_t b = __float_as_uint(v);
  const auto x = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  const uint32_t h = __float_as_uint(__uint_as_float(x[0]) + __uint_as_float(x[1]));
  const auto y = __builtin_amdgcn_permlane32_swap(h, h, false, false);
  return __uint_as_float(y[0]) + __uint_as_float(y[1]);
#else
  return v;
#endif
}

// ------------------------------------------------------------------ packing
// The 32-point rotation of a block whose elements 8 c .. 8 c + 7 the lane c =
// lane % 4 holds: hadamard32's butterfly, its strides 8 and 16 across lanes.
__device__ __forceinline__ void hadamard_lanes(float (&v)[8], int lane) {
#pragma unroll
  for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
    for (int i = 0; i < 8; i += 2 * h) {
#pragma unroll
      for (int j = i; j < i + h; ++j) {
        const float a = v[j], b = v[j + h];
        v[j] = a + b;
        v[j + h] = a - b;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float o = dpp_float<kDppXor1>(v[i]);
    v[i] = (lane & 1) ? o - v[i] : v[i] + o;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float o = dpp_float<kDppXor2>(v[i]);
    v[i] = (lane & 2) ? o - v[i] : v[i] + o;
  }
  const float c = __uint_as_float(0x3e3504f3u);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] * c;
}

// E2M3 code of v / 2^X given 2^-X: nearest, ties to even, saturating at 7.5
// (the spacing is 1/8 below 2, 1/4 below 4, then 1/2).
__device__ __forceinline__ uint32_t e2m3_code(float v, float inv) {
  const float a = __builtin_fabsf(v) * inv;
  const float step = a < 2.0f ? 8.0f : a < 4.0f ? 4.0f : 2.0f;
  const uint32_t base = a < 2.0f ? 0u : a < 4.0f ? 8u : 16u;
  const uint32_t c = base + (uint32_t)__builtin_rintf(a * step);
  return (c < 31u ? c : 31u) | ((__float_as_uint(v) >> 26) & 32u);
}

// Quantize blocks of 32 held by four adjacent lanes (16 lanes: one row's K
// group) and store this lane's codes at the group's base `g`, and the group's
// four scale bytes from its first lane: the bytes that quant_store writes.
// `row` is the operand's row.  Every lane takes part; `in` says whether it
// stores.
template <int FMT, int MODE, int HAD>
__device__ __forceinline__ void lane8_quantize(float (&v)[8], uint8_t* g, uint8_t* scales, int64_t row, bool in) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int lane = threadIdx.x & 63, ch = lane & 15, blk = ch >> 2, c = ch & 3;
  if constexpr (HAD) hadamard_lanes(v, lane);
  const uint32_t s = scale_byte<FMT, MODE>(max_over4(abs_max(v)));
  if constexpr (FMT == kE2M3) {
    const float inv = __uint_as_float((254u - (s == 0xffu ? 127u : s)) << 23);  // 2^-X (X is at most 125 here)
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = s == 0xffu ? 0u : e2m3_code(v[i], inv);
    // 48 bits a lane; the block's six dwords are 0, 1 from lane 0, 2 from lane
    // 1, 3 from lane 2 and 4, 5 from lane 3
    const uint32_t lo = q[0] | q[1] << 6 | q[2] << 12 | q[3] << 18 | q[4] << 24 | q[5] << 30;
    const uint32_t hi = q[5] >> 2 | q[6] << 4 | q[7] << 10;  // 16 bits
    const uint32_t other_lo = dpp_move<kDppXor1>(lo), other_hi = dpp_move<kDppXor1>(hi);
    const uint32_t even1 = hi | other_lo << 16;              // second dword of an even lane's pair
    const uint32_t odd1 = lo >> 16 | hi << 16;               // third
    const uint32_t odd0 = other_hi | lo << 16;               // second, from the odd lane
    if (in) {
      if (c == 0) *reinterpret_cast<uint2*>(g + 16 * blk) = make_uint2(lo, even1);
      else if (c == 1) *reinterpret_cast<uint32_t*>(g + 16 * blk + 8) = odd1;
      else if (c == 2) *reinterpret_cast<uint32_t*>(g + 16 * blk + 12) = lo;
      else *reinterpret_cast<uint2*>(g + 64 + 8 * (blk ^ (int)((row >> 4) & 1))) = make_uint2(odd0, odd1);
    }
  } else if constexpr (FMT == kE2M1) {
    const bool tiny = s == 0u;
    const float sc = __uint_as_float((tiny ? 64u : (s == 0xffu ? 127u : s)) << 23);
    if (__builtin_amdgcn_ballot_w64(tiny) != 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = tiny ? v[i] * 0x1p64f : v[i];
    }
    uint32_t q = 0u;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], sc, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], sc, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], sc, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], sc, 3);
    if (in) *reinterpret_cast<uint32_t*>(g + 4 * ch) = s == 0xffu ? 0u : q;
  } else {
    if constexpr (MODE == kFloor) {  // 2^8 2^X <= amax < 2^9 2^X: clamped to 448 2^X
      // (X = -127: the block's values lie below 2^-118, where 448 2^-127 is
      // still formed exactly from 448 2^-63 2^-64)
      const bool tiny = s == 0u;
      const float bound = tiny ? 448.0f * 0x1p-63f * 0x1p-64f : 448.0f * __uint_as_float((s == 0xffu ? 127u : s) << 23);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = s == 0xffu ? v[i] : __builtin_fminf(__builtin_fmaxf(v[i], -bound), bound);
    }
    uint32_t w[2];
    e4m3_encode(v, s, w);
    if (in) *reinterpret_cast<uint2*>(g + 8 * ch) = make_uint2(w[0], w[1]);
  }
  uint32_t d = s << (8 * blk);
  d |= dpp_move<kDppRor8>(d);
  d |= dpp_move<kDppRor4>(d);
  if (in && ch == 0) *reinterpret_cast<uint32_t*>(scales) = d;
#endif
}

}  // namespace mx
