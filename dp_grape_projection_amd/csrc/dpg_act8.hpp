// Activations in 8 bits: 32 consecutive channels of a row share a power of two.
//
// With b = max(7, the exponent field of the block's largest magnitude as fp32), a
// value is held as the integer q = clamp(round(x 2^(133 - b)), -127, 127), ties to
// even, and b as one byte; it stands for q 2^(b - 133). The largest magnitude lies in
// [64, 128) steps, so a value is off by at most half a step, 2^-7 of the block's
// largest (fp32 values in a block's last half step by up to one). b >= 7 keeps both
// factors normal numbers, at steps of 2^-126: a block whose largest is below 2^-120 is
// off by up to 2^-127, whatever part of it that is. A block with an infinity or NaN gets
// b = 255 and reads as NaN. Every value q 2^(b - 133) is a bf16 number: reading it back, or feeding it to
// the bf16 matrix instructions, rounds nothing.
#pragma once

#include "dpg_device.hpp"
#include "dpg_internal.hpp"
#include "dpg_tile.hpp"

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

constexpr int kPer = 8;      // channels of a lane
constexpr int kFlight = 4;   // a lane's pieces in flight

struct Act8Args {
  const void* X;
  void* out;         // unpack: rows of ldo elements
  int8_t* codes;     // [N][32 * blocks]
  uint8_t* exps;     // [N][blocks]
  int64_t N;
  int64_t d;         // channels
  int64_t ldo;       // unpack: elements of an output row, >= d
  int64_t blocks;    // blocks of a row
  uint32_t pieces;   // pieces of 8 channels of a row that are written
  uint32_t total;    // N * pieces, below 2^31
  uint32_t magic;    // t / pieces = (t * magic) >> 32 >> shift for t < 2^31
  uint32_t shift;
};

struct Place {
  int64_t row;
  int c;       // the piece's first channel
  bool there;
};
__device__ __forceinline__ Place place_of(const Act8Args& a, uint32_t block, int u) {
  const uint32_t t = (block * kFlight + u) * kThreads + threadIdx.x;
  const uint32_t row = __umulhi(t, a.magic) >> a.shift;
  return {row, static_cast<int>(t - row * a.pieces) * kPer, t < a.total};
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 any_u32x2 __attribute__((aligned(1)));

__device__ __forceinline__ void store8(bf16* row, int c, int64_t n, const float (&x)[8]) {
  bf16x8 v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = from_float<bf16>(x[i]);
  store_row(row + c, static_cast<int>(n), v);
}
__device__ __forceinline__ void store8(float* row, int c, int64_t n, const float (&x)[8]) {
  store_row(row + c, static_cast<int>(n), f32x4{x[0], x[1], x[2], x[3]});
  if (n > 4) store_row(row + c + 4, static_cast<int>(n) - 4, f32x4{x[4], x[5], x[6], x[7]});
}

// Reads back the pieces of one block of threads.
template <typename T>
__device__ __forceinline__ void unpack8_block(const Act8Args& a, uint32_t block) {
  u32x2 q[kFlight];
  uint32_t b[kFlight];
#pragma unroll
  for (int u = 0; u < kFlight; ++u) {
    const Place p = place_of(a, block, u);
    q[u] = u32x2{0u, 0u};
    b[u] = 7u;
    if (p.there && p.c < a.d) {
      q[u] = *reinterpret_cast<const any_u32x2*>(a.codes + p.row * a.blocks * kBlock8 + p.c);
      b[u] = a.exps[p.row * a.blocks + p.c / kBlock8];
    }
  }
#pragma unroll
  for (int u = 0; u < kFlight; ++u) {
    const Place p = place_of(a, block, u);
    if (!p.there) continue;
    const float s = step8(b[u]);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (what pads a row's last block stands for nothing)
      x[i] = p.c + i < a.d ? value8(q[u].x, i, s) : 0.0f;
      x[4 + i] = p.c + 4 + i < a.d ? value8(q[u].y, i, s) : 0.0f;
    }
    store8(static_cast<T*>(a.out) + p.row * a.ldo, p.c, a.ldo - p.c, x);
  }
}

inline int64_t blocks8(int64_t d) { return (d + kBlock8 - 1) / kBlock8; }

// Sets how the grid covers a.N rows, and returns its blocks; N pieces is below 2^31 less
// a block's.
inline int64_t cover_rows(Act8Args& a) {
  uint32_t bits = 0;
  while (int64_t{1} << bits < a.pieces) ++bits;
  // ceil(2^(31 + bits) / pieces): off by less than 2^bits in all, which t < 2^31 forgives
  a.magic = static_cast<uint32_t>(((uint64_t{1} << (31 + bits)) + a.pieces - 1) / a.pieces);
  a.shift = bits - 1;
  a.total = static_cast<uint32_t>(a.N * a.pieces);
  return ceil_div(a.total, kThreads * kFlight);
}
// Rows of d channels read back into rows of ldo elements.
inline Act8Args unpack_args(const int8_t* codes, const uint8_t* exps, int64_t N, int64_t d, void* X,
                            int64_t ldo) {
  Act8Args a{};
  a.out = X, a.codes = const_cast<int8_t*>(codes), a.exps = const_cast<uint8_t*>(exps);
  a.N = N, a.d = d, a.ldo = ldo, a.blocks = blocks8(d);
  a.pieces = static_cast<uint32_t>(ldo <= kPer ? 2 : ceil_div(ldo, kPer));
  return a;
}

}  // namespace dpg
