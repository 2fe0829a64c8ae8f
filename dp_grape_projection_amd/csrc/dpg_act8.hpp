// Activations in 8 bits: 32 consecutive channels of a row share a power of two.
//
// With b = max(7, the exponent field of the block's largest magnitude as fp32), a
// value is held as the integer q = clamp(round(x 2^(133 - b)), -127, 127), ties to
// even, and b as one byte; it stands for q 2^(b - 133). The largest magnitude lies in
// [64, 128) steps, so a value is off by at most half a step, 2^-7 of the block's
// largest (fp32 values in a block's last half step by up to one). b >= 7 keeps both
// factors normal numbers; a block with an infinity or NaN gets b = 255 and reads as
// NaN. Every value q 2^(b - 133) is a bf16 number: reading it back, or feeding it to
// the bf16 matrix instructions, rounds nothing.
#pragma once

#include "dpg_device.hpp"

namespace dpg {

constexpr int kBlock8 = 32;  // channels that share an exponent

// Exponent byte from the largest magnitude's bits (fp32, sign cleared).
__device__ __forceinline__ uint32_t exponent8(uint32_t top) { return max(top >> 23, 7u); }
// 2^(133 - b) and 2^(b - 133), with NaN for b = 255.
__device__ __forceinline__ float to_steps8(uint32_t b) {
  return __builtin_bit_cast(float, (260u - b) << 23);
}
__device__ __forceinline__ float step8(uint32_t b) {
  return __builtin_bit_cast(float, b == 255u ? 0x7FC00000u : (max(b, 7u) - 6u) << 23);
}
__device__ __forceinline__ uint32_t magnitude_bits(float x) {
  return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu;
}
// The codes of four values, the first in the lowest byte; zero where b = 255. Adding 1.5
// 2^23 to x in steps rounds it to an integer, ties to even, whose low byte is the code.
__device__ __forceinline__ uint32_t codes8(float x0, float x1, float x2, float x3, uint32_t b) {
  const float s = to_steps8(b), top = 127.0f * step8(b);
  auto code = [&](float x) {
    return __builtin_bit_cast(uint32_t, fmaf(__builtin_amdgcn_fmed3f(x, -top, top), s, 12582912.0f));
  };
  const uint32_t lo = __builtin_amdgcn_perm(code(x1), code(x0), 0x0c0c0400u),
                 hi = __builtin_amdgcn_perm(code(x3), code(x2), 0x04000c0cu);
  return b == 255u ? 0u : lo | hi;
}
// The value of byte i of `codes`.
__device__ __forceinline__ float value8(uint32_t codes, int i, float step) {
  return static_cast<float>(static_cast<int>(codes << (24 - 8 * i)) >> 24) * step;
}

inline int64_t blocks8(int64_t d) { return (d + kBlock8 - 1) / kBlock8; }

}  // namespace dpg
