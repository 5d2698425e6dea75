// e4m3 codes with a scale, for the kernels that quantise what they just computed.
#pragma once

#include "quantize.cuh"

namespace dsa {
namespace quant {

// The smallest scale.  amax / 448 rounds to 0 below 448 * 2^-150, and 0 / 0 would be a NaN code; over this
// scale such values (multiples of 2^-149) are exact quotients of at most 224.
constexpr float kLeastScale = 0x1p-149f;

// The scale of values with this largest magnitude (1 for none).
__device__ __forceinline__ float scale_of(float amax) { return amax > 0.f ? fmaxf(__fdiv_rn(amax, kE4m3Max), kLeastScale) : 1.f; }

// 1 / s for over(), or 0 where s is so small that 1 / s could overflow.
__device__ __forceinline__ float inverse_of(float s) { return s > 0x1p-120f ? __fdiv_rn(1.f, s) : 0.f; }

// v / s as v * (1 / s): two fp32 roundings (2^-23 relative) before the one to e4m3 (2^-4), which can
// differ from the exact quotient's code only next to a tie; a division per element was the largest
// part of the kernels' instructions.  Tiny scales take the division.
__device__ __forceinline__ float over(float v, float s, float inv) { return inv > 0.f ? v * inv : __fdiv_rn(v, s); }

}  // namespace quant
}  // namespace dsa
