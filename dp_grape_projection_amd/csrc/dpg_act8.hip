// Writing activations in 8 bits and reading them back: dpg_pack_act, dpg_unpack_act.
// The format and its reasons stand in dpg_act8.hpp.
//
// Both kernels are bound by memory: a row of d bf16 values is 2 d bytes against 1.03 d
// of codes and exponents. A lane takes 8 channels (16 or 32 bytes of X, 8 bytes of
// codes), four such pieces in flight; the four lanes of a block find its largest magnitude
// between them. 8192 x 8192 bf16: written in 47 us (4.3 TB/s), read back in 31 (6.6 TB/s,
// part of it from the memory-side cache), where a large copy moves 5.2 TB/s; 16384 x 11008:
// 119 and 86 us.
#include <cmath>
#include <string>

#include "dpg.h"
#include "dpg_act8.hpp"
#include "dpg_internal.hpp"
#include "dpg_tile.hpp"

namespace dpg {
namespace {

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
__device__ __forceinline__ Place place_of(const Act8Args& a, int u) {
  const uint32_t t = (blockIdx.x * kFlight + u) * kThreads + threadIdx.x;
  const uint32_t row = __umulhi(t, a.magic) >> a.shift;
  return {row, static_cast<int>(t - row * a.pieces) * kPer, t < a.total};
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 any_u32x2 __attribute__((aligned(1)));

// Eight channels of a row from c on, zero beyond it.
__device__ __forceinline__ void load8(const bf16* row, int c, int64_t d, float (&x)[8]) {
  const bf16x8 v = load_row(row, c, static_cast<int>(d));
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(v[i]);
}
__device__ __forceinline__ void load8(const float* row, int c, int64_t d, float (&x)[8]) {
  const f32x4 v = load_row(row, c, static_cast<int>(d)),
              w = load_row(row, c + 4, static_cast<int>(d));
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = v[i], x[4 + i] = w[i];
}

template <typename T>
__global__ __launch_bounds__(kThreads) void pack8_kernel(const Act8Args a) {
  float x[kFlight][8];
#pragma unroll
  for (int u = 0; u < kFlight; ++u) {
    const Place p = place_of(a, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[u][i] = 0.0f;
    if (p.there) load8(static_cast<const T*>(a.X) + p.row * a.d, p.c, a.d, x[u]);
  }
#pragma unroll
  for (int u = 0; u < kFlight; ++u) {
    const Place p = place_of(a, u);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, magnitude_bits(x[u][i]));
    // (a block's four lanes are neighbours: pieces are whole blocks)
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 1, 64)));
    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 2, 64)));
    const uint32_t b = exponent8(top);
    if (!p.there) continue;
    u32x2 q;
    q.x = codes8(x[u][0], x[u][1], x[u][2], x[u][3], b);
    q.y = codes8(x[u][4], x[u][5], x[u][6], x[u][7], b);
    *reinterpret_cast<any_u32x2*>(a.codes + p.row * a.blocks * kBlock8 + p.c) = q;
    if ((p.c & (kBlock8 - 1)) == 0) a.exps[p.row * a.blocks + p.c / kBlock8] = static_cast<uint8_t>(b);
  }
}

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

template <typename T>
__global__ __launch_bounds__(kThreads) void unpack8_kernel(const Act8Args a) {
  u32x2 q[kFlight];
  uint32_t b[kFlight];
#pragma unroll
  for (int u = 0; u < kFlight; ++u) {
    const Place p = place_of(a, u);
    q[u] = u32x2{0u, 0u};
    b[u] = 7u;
    if (p.there && p.c < a.d) {
      q[u] = *reinterpret_cast<const any_u32x2*>(a.codes + p.row * a.blocks * kBlock8 + p.c);
      b[u] = a.exps[p.row * a.blocks + p.c / kBlock8];
    }
  }
#pragma unroll
  for (int u = 0; u < kFlight; ++u) {
    const Place p = place_of(a, u);
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

// fn(arguments, grid) for runs of rows of at most 2^31 pieces.
template <class F>
hipError_t for_rows(Act8Args a, int64_t x_row, int64_t out_row, F fn) {
  uint32_t bits = 0;
  while (int64_t{1} << bits < a.pieces) ++bits;
  // ceil(2^(31 + bits) / pieces): off by less than 2^bits in all, which t < 2^31 forgives
  a.magic = static_cast<uint32_t>(((uint64_t{1} << (31 + bits)) + a.pieces - 1) / a.pieces);
  a.shift = bits - 1;
  const int64_t N = a.N, per = ((int64_t{1} << 31) - kThreads * kFlight) / a.pieces;
  for (int64_t n0 = 0; n0 < N; n0 += per) {
    a.N = std::min(per, N - n0);
    a.total = static_cast<uint32_t>(a.N * a.pieces);
    fn(a, dim3(static_cast<unsigned>(ceil_div(a.total, kThreads * kFlight))));
    a.X = static_cast<const char*>(a.X) + a.N * x_row;
    a.out = static_cast<char*>(a.out) + a.N * out_row;
    a.codes += a.N * a.blocks * kBlock8, a.exps += a.N * a.blocks;
  }
  return hipGetLastError();
}

int check_shape(int64_t N, int64_t d, int32_t dtype) {
  if (N < 1 || N > (1ll << 30)) return fail(DPG_ERR_INVALID_ARG, "N must be in [1, 2^30]");
  if (d < 1 || d > (1ll << 20)) return fail(DPG_ERR_INVALID_ARG, "d must be in [1, 2^20]");
  if (dtype != DPG_FP32 && dtype != DPG_BF16) return fail(DPG_ERR_INVALID_ARG, "unknown dtype");
  return DPG_OK;
}

}  // namespace

hipError_t launch_pack8(const void* X, bool bf16_in, int64_t N, int64_t d, int8_t* codes,
                        uint8_t* exps, hipStream_t s) {
  Act8Args a{};
  a.X = X, a.codes = codes, a.exps = exps;
  a.N = N, a.d = d, a.blocks = blocks8(d);
  a.pieces = static_cast<uint32_t>(a.blocks * (kBlock8 / kPer));
  return for_rows(a, d * (bf16_in ? 2 : 4), 0, [&](const Act8Args& r, dim3 grid) {
    if (bf16_in) hipLaunchKernelGGL(pack8_kernel<bf16>, grid, dim3(kThreads), 0, s, r);
    else hipLaunchKernelGGL(pack8_kernel<float>, grid, dim3(kThreads), 0, s, r);
  });
}

hipError_t launch_unpack8(const int8_t* codes, const uint8_t* exps, int64_t N, int64_t d,
                          void* X, bool bf16_out, int64_t ldo, hipStream_t s) {
  Act8Args a{};
  a.out = X, a.codes = const_cast<int8_t*>(codes), a.exps = const_cast<uint8_t*>(exps);
  a.N = N, a.d = d, a.ldo = ldo, a.blocks = blocks8(d);
  a.pieces = static_cast<uint32_t>(std::max<int64_t>(2, ceil_div(ldo, kPer)));
  return for_rows(a, 0, ldo * (bf16_out ? 2 : 4), [&](const Act8Args& r, dim3 grid) {
    if (bf16_out) hipLaunchKernelGGL(unpack8_kernel<bf16>, grid, dim3(kThreads), 0, s, r);
    else hipLaunchKernelGGL(unpack8_kernel<float>, grid, dim3(kThreads), 0, s, r);
  });
}

}  // namespace dpg

using namespace dpg;

extern "C" {

int dpg_pack_act(const void* X, int64_t N, int64_t d, int32_t dtype, int8_t* codes, uint8_t* exps,
                 void* stream) {
  record_error(DPG_OK, "");
  if (const int st = check_shape(N, d, dtype)) return st;
  if (!X || !codes || !exps) return fail(DPG_ERR_INVALID_ARG, "NULL data pointer");
  if (launch_pack8(X, dtype == DPG_BF16, N, d, codes, exps, static_cast<hipStream_t>(stream)) !=
      hipSuccess)
    return fail(DPG_ERR_HIP, "pack_act: launch failed");
  return DPG_OK;
}

int dpg_unpack_act(const int8_t* codes, const uint8_t* exps, int64_t N, int64_t d, int32_t dtype,
                   void* X, void* stream) {
  record_error(DPG_OK, "");
  if (const int st = check_shape(N, d, dtype)) return st;
  if (!X || !codes || !exps) return fail(DPG_ERR_INVALID_ARG, "NULL data pointer");
  if (launch_unpack8(codes, exps, N, d, X, dtype == DPG_BF16, d,
                     static_cast<hipStream_t>(stream)) != hipSuccess)
    return fail(DPG_ERR_HIP, "unpack_act: launch failed");
  return DPG_OK;
}

}  // extern "C"
