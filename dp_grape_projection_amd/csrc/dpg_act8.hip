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
    const Place p = place_of(a, blockIdx.x, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[u][i] = 0.0f;
    if (p.there) load8(static_cast<const T*>(a.X) + p.row * a.d, p.c, a.d, x[u]);
  }
#pragma unroll
  for (int u = 0; u < kFlight; ++u) {
    const Place p = place_of(a, blockIdx.x, u);
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

template <typename T>
__global__ __launch_bounds__(kThreads) void unpack8_kernel(const Act8Args a) {
  unpack8_block<T>(a, blockIdx.x);
}

// fn(arguments, grid) for runs of rows of at most 2^31 pieces.
template <class F>
hipError_t for_rows(Act8Args a, int64_t x_row, int64_t out_row, F fn) {
  const int64_t N = a.N, per = ((int64_t{1} << 31) - kThreads * kFlight) / a.pieces;
  for (int64_t n0 = 0; n0 < N; n0 += per) {
    a.N = std::min(per, N - n0);
    const int64_t blocks = cover_rows(a);
    fn(a, dim3(static_cast<unsigned>(blocks)));
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
  const Act8Args a = unpack_args(codes, exps, N, d, X, ldo);
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
