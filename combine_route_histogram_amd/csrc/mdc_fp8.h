// fp8 (e4m3, OCP) with one scale per 128 consecutive values, shared by the
// norm, the row quantiser and the fp8 products.
#pragma once

#include "mdc_ops.h"

namespace {

constexpr int kFp8Block = 128;          // values that share a scale
constexpr float kFp8Max = 448.0f;       // largest e4m3 value
constexpr float kFp8AmaxMin = 0x1p-110f;   // a non-zero block's amax counts as at least this (1 / amax stays finite)

// max over the 16 lanes of a DPP row (xor 1, xor 2, half mirror, mirror).
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));
  return v;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Scale of a block whose largest |value| has the bits amax_bits (unsigned
// maxima of such bits put NaN above infinity above every number), and the
// codes of its values: rne_e4m3(448 v / amax).  The quotient is rounded
// correctly where it matters: v 7/8 is exact for values of up to 21
// significant bits, and the correction q + (v' - q d) / d leaves a quotient
// that fp32 holds exact, so that halves between two codes stay halves.
struct Fp8Scaler {
  float scale;      // amax / 448
  float den, inv;   // amax / 512 and its reciprocal; 448 v / amax = (7/8 v) / den
  __device__ __forceinline__ explicit Fp8Scaler(uint32_t amax_bits) {
    const float amax = __uint_as_float(amax_bits);
    const float a = amax_bits != 0u && amax < kFp8AmaxMin ? kFp8AmaxMin : amax;
    scale = a / kFp8Max;
    den = a * 0x1p-9f;
    inv = amax_bits != 0u ? __builtin_amdgcn_rcpf(den) : 0.f;
  }
  __device__ __forceinline__ float quotient(float v) const {
    const float t = v * 0.875f;
    const float q = t * inv;
    return __builtin_fmaf(__builtin_fmaf(-q, den, t), inv, q);
  }
  // codes of four values, the first in the lowest byte
  __device__ __forceinline__ uint32_t codes4(float v0, float v1, float v2, float v3) const {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v0), quotient(v1), 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v2), quotient(v3), w, true);
    return (uint32_t)w;
  }
};

}  // namespace
