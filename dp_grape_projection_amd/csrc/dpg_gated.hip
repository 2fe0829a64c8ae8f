// The gated feed-forward block and its gradients: dpg_gated, dpg_gated_grad.
//
//   G = X W_gate, U = X W_up   (W_in = [W_gate | W_up], [d][2f])
//   H = act(G) * U             [N][f]
//   Y = H W_out                [N][d]
//   dH = dY W_out^T, dU = dH act(G), dG = dH U act'(G)
//   dX = [dG | dU] W_in^T, dW_in = X^T [dG | dU], dW_out = H^T dY
//
// All products run in the tiles of dpg_tile.hpp. The first computes both projections:
// a wave's 16-column blocks are half of the gate's and half of the same columns of the
// up projection, so that a lane holds G and U of the same places and H leaves the tile
// without either being stored. What the backward pass keeps of them is the caller's
// choice: their 8-bit form (dpg_act8.hpp), written by the same epilogue, or nothing, in
// which case they are computed again, without a rounding, by the blocks that need them.
// dH is not stored as a matrix either: what computes it has G and U of the same places
// and writes dG, dU and H.
//
// Epilogues keep to registers: quarters of a wave change places with four registers
// (dpg_tile.hpp), so that a lane stores 16 bytes of one row where it held four columns of
// four blocks, without LDS, barriers or the copies' space (forward and backward of 8192 x
// 2048 x 8192, 8-bit projections: 2.28 ms staged in LDS, 2.13 so).
//
// Inside, Z = [G | U] and dZ have their halves fq columns apart, f rounded up to 8, so
// that both halves' rows can be copied 16 bytes at a time; what lies between and after
// is zero, and so are dZ's and H's rows from N up to whole K steps, which the weights'
// gradients sum over.
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <string>

#include "dpg.h"
#include "dpg_act8.hpp"
#include "dpg_device.hpp"
#include "dpg_internal.hpp"
#include "dpg_tile.hpp"

namespace dpg {
namespace {

constexpr int kPad = 256;  // rows of a product's partial sums are padded to whole tiles
constexpr float kLog2e = 1.4426950408889634f;

// A matrix as operands of 16 bits see it: rows of ld elements, in one or three parts.
struct Mat {
  const bf16* p;
  int64_t ld;
  int64_t part;   // elements between the parts
  int32_t rows, cols;
};

struct GatedArgs {
  Mat x, w_in, w_out, dy, h, dz;
  int32_t N, d, f, fq, act;
  int32_t ldh;          // f rounded up to 64
  int32_t fp;           // f rounded up to 32: the codes of one half of a row of Z
  int32_t np;           // rows of dz and h that are written: N up to whole K steps
  int8_t* codes;        // [N][2][fp], or null
  uint8_t* exps;        // [N][2][fp / 32]
  bool two;             // bf16: h and dz in two parts
  f32x4* scratch;       // a tile of dH for every resident block, where Z is computed again
  void* dz_out;         // [N][2f] the caller's dZ where dz is in the workspace, h_out likewise
  void* h_out;          // [N][f]
};

// ------------------------------------------------------------ activations --

__device__ __forceinline__ float exp_(float x) { return exp2_(x * kLog2e); }
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + exp_(-x));
}

// Phi(x), with e = exp(-x^2 / 2), which the slope needs too. The tail Phi(-|x|) is e times
// a slowly falling function of |x|, here a polynomial in 1 / (1 + |x| / 3) fitted for the
// least relative error over [0, 13.4] (7e-9; beyond, e is zero). 1 + erf(x / sqrt 2) would
// cancel: a gate of -4 is off by 3e-4 of its value that way, one of -5 by 4 %. The
// library's erfc keeps the tail too, at 3 % of a step of 16384 x 768 x 2048 (690 us, 667
// with 1 + erf).
__device__ __forceinline__ float normal_cdf(float x, float& e) {
  e = exp_(-0.5f * x * x);
  const float w = __builtin_amdgcn_rcpf(fmaf(fabsf(x), 0.33333334f, 1.0f));
  const float c[] = {6.01766197e-06f, 1.32818176e-01f,  1.34891244e-01f, 1.05370570e-01f,  1.43067443e-01f,
                     -1.01843256e-01f, 2.83787339e-01f, -3.24841814e-01f, 1.54469604e-01f, -2.77253265e-02f};
  float r = c[9];
#pragma unroll
  for (int i = 8; i >= 0; --i) r = fmaf(r, w, c[i]);
  return x < 0.0f ? e * r : 1.0f - e * r;
}

// act(x), and with it act'(x). The exponential and reciprocal instructions are off by 1 ulp;
// e^x also by the rounding of its argument, 2^-24 |x| of the result, which is what the last
// bit of x itself moves it by (silu(-20): 1e-6).
template <int ACT>
__device__ __forceinline__ float act_of(float x) {
  if constexpr (ACT == DPG_ACT_SILU) {
    return x * sigmoid(x);
  } else if constexpr (ACT == DPG_ACT_GELU) {
    float e;
    return x * normal_cdf(x, e);
  } else {
    // (1 + tanh t) / 2 = sigmoid(2 t)
    return x * sigmoid(1.5957691216f * (x + 0.044715f * x * x * x));
  }
}
template <int ACT>
__device__ __forceinline__ float act_of(float x, float& slope) {
  if constexpr (ACT == DPG_ACT_SILU) {
    const float s = sigmoid(x);
    slope = s * (1.0f + x * (1.0f - s));
    return x * s;
  } else if constexpr (ACT == DPG_ACT_GELU) {
    float e;
    const float c = normal_cdf(x, e);
    slope = c + x * (0.3989422804f * e);
    return x * c;
  } else {
    // beyond 20 the sigmoid is 0 or 1 and the slope's second term nothing (the median of a
    // NaN would be -20, and its slope 0)
    const float y = x != x ? x : __builtin_amdgcn_fmed3f(x, -20.0f, 20.0f);
    const float s = sigmoid(1.5957691216f * (y + 0.044715f * y * y * y));
    slope = s + y * s * (1.0f - s) * (1.5957691216f * (1.0f + 0.134145f * y * y));
    return x * s;
  }
}
template <class F>
__host__ __device__ __forceinline__ void with_act(int act, F fn) {
  if (act == DPG_ACT_SILU) fn(std::integral_constant<int, DPG_ACT_SILU>{});
  else if (act == DPG_ACT_GELU) fn(std::integral_constant<int, DPG_ACT_GELU>{});
  else fn(std::integral_constant<int, DPG_ACT_GELU_TANH>{});
}

// ---------------------------------------------------------------- packing --

// Copies of matrices as parts, zero-padded to rows of whole K steps: up to four of them
// in one launch, a wave a row (or half of one, whose halves go fq columns apart).
struct PackJob {
  const void* src;   // [rows][halves][cols]
  bf16* dst;         // rows of ld elements
  int64_t ld, part;
  int32_t rows, cols, halves, fq;
  int64_t wave0;     // first wave of the job
};
struct PackArgs {
  PackJob job[4];
  int32_t n;
  int64_t waves;
};

template <typename T>
__global__ __launch_bounds__(kThreads) void pack_mat_kernel(const PackArgs a) {
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (w >= a.waves) return;
  int j = 0;
  while (j + 1 < a.n && w >= a.job[j + 1].wave0) ++j;
  const PackJob& o = a.job[j];
  const int64_t at = w - o.wave0, r = at / o.halves;
  const int h = static_cast<int>(at - r * o.halves);
  const int width = h + 1 < o.halves ? o.fq : static_cast<int>(o.ld) - h * o.fq;
  pack_row(static_cast<const T*>(o.src) + at * o.cols, o.dst + r * o.ld + h * o.fq, o.cols, width,
           o.part, threadIdx.x & 63);
}

// --------------------------------------------------------------- products --

// LDS of a kernel of tiles, and its blocks on a CU.
template <class G, int PARTS> constexpr int kLdsOf = PARTS == 3 ? kPartsLds<G> : G::kLds;
template <class G, int PARTS>
constexpr int kBlocksOf = PARTS != 3 ? G::kBlocks : G::kTile == TinyTile::kTile ? 2 : 1;

template <class G, int PARTS, bool KA, bool KB, bool AGAIN = false>
__device__ __forceinline__ void product(const Operand& a, const Operand& b, int n_k, char* smem,
                                        typename G::Acc& acc) {
  if constexpr (PARTS == 3) parts_product<G, KA, KB>(a, b, n_k, smem, acc);
  else tile_product<G, PARTS, KA, KB, AGAIN>(a, b, n_k, smem, acc);
}

__device__ __forceinline__ Operand rows_of(const Mat& m, int r0, int k0) {
  return rows_operand(m.p + static_cast<int64_t>(r0) * m.ld + k0, m.ld, m.part, m.rows - r0, m.cols - k0);
}
__device__ __forceinline__ Operand kmajor_of(const Mat& m, int k0, int c0) {
  return rows_operand(m.p + static_cast<int64_t>(k0) * m.ld + c0, m.ld, m.part, m.rows - k0, m.cols - c0);
}

typedef uint32_t any_u32 __attribute__((aligned(1)));
typedef uint32_t any_u32x4 __attribute__((ext_vector_type(4), aligned(1)));

// The codes of a lane's eight values of a block of 32 columns, which four lanes share.
__device__ __forceinline__ void codes_of_block(const f32x4& x, const f32x4& y, uint32_t& cx,
                                               uint32_t& cy, uint32_t& b) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(magnitude_bits(x[i]), magnitude_bits(y[i])));
  uint32_t other = top;
  swap16(top, other);
  top = max(top, other);
  other = top;
  swap32(top, other);
  b = exponent8(max(top, other));
  cx = codes8(x[0], x[1], x[2], x[3], b);
  cy = codes8(y[0], y[1], y[2], y[3], b);
}

// Four values, rounded, at any element's address.
__device__ __forceinline__ void store_any4(bf16* p, const f32x4& x) {
  typedef __bf16 any4 __attribute__((ext_vector_type(4), aligned(2)));
  any4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = from_float<bf16>(x[i]);
  *reinterpret_cast<any4*>(p) = v;
}

// MB blocks of 16 columns of one row, rounded (or, of several parts, the next one taken
// off x), to dst of n columns.
template <int MB, int PARTS>
__device__ __forceinline__ void store_strip(bf16* dst, f32x4 (&x)[MB], int kq, bool row, int n) {
#pragma unroll
  for (int p = 0; p < MB / 2; ++p) {
    Vec4<bf16>::type v[2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[m][i] = PARTS == 1 ? from_float<bf16>(x[2 * p + m][i]) : take_part(x[2 * p + m], i);
    const bf16x8 w = pair_cols(v[0], v[1]);
    const int c = 32 * p + pair_col(kq);
    if (row && c < n) store_row(dst + c, n - c, w);
  }
}

// store_strip of values in bf16: once, and with `two` (TWO: it may be set) what that left
// over to dst + part.
template <int MB, bool TWO>
__device__ __forceinline__ void store_strips(bf16* dst, int64_t part, bool two, f32x4 (&x)[MB], int kq,
                                             bool row, int n) {
  store_strip<MB, 1>(dst, x, kq, row, n);
  if (!TWO || !two) return;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = static_cast<float>(from_float<bf16>(x[mb][i]));
      x[mb][i] = fabsf(v) < INFINITY ? x[mb][i] - v : 0.0f;  // (an infinity leaves nothing)
    }
  store_strip<MB, 1>(dst + part, x, kq, row, n);
}

// A tile of G and U: TILE / 2 columns of each by TILE rows. Bound by the products: 16384 x
// 4096 x 11008 in 2.13 to 2.20 ms, 1390 to 1340 TFLOP/s; with the 8-bit form written,
// 8192 x 2048 x 8192 in 484 us, 1140 TFLOP/s (the epilogue rounds and packs 128 values a
// lane, 10 us of a tile's 60).
template <class G, int PARTS, int ACT, bool CODES>
__global__ __launch_bounds__(G::kThreads, (kBlocksOf<G, PARTS>)) void gate_up_kernel(const GatedArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[kLdsOf<G, PARTS>];
  constexpr int kCols = G::kTile / 2, kHB = G::kMB / 2;  // columns of H; blocks of a half
  int mt, nt;
  if (!tile_of_block(blockIdx.x, (a.ldh + kCols - 1) / kCols, (a.N + G::kTile - 1) / G::kTile, mt, nt))
    return;
  const int c0 = mt * kCols, r0 = nt * G::kTile;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave % G::kWavesM, wn = wave / G::kWavesM, r16 = lane & 15, kq = lane >> 4;
  // (a tile of padding alone computes the last columns, and writes zeros)
  Operand w = kmajor_of(a.w_in, 0, min(c0, a.fq - 8));
  w.cols = a.fq - min(c0, a.fq - 8);
  w.half = a.fq;
  typename G::Acc acc;
  product<G, PARTS, true, false>(w, rows_of(a.x, r0, 0), (a.d + kStepK - 1) / kStepK, smem, acc);
  const int cw = c0 + 16 * kHB * wm;  // the wave's first column of H
  with_edge(r0 + G::kTile > a.N || c0 + kCols > a.f, [&](auto edge) {
    constexpr bool E = decltype(edge)::value;
    each<G::kNB>([&](auto at) {
      constexpr int nb = decltype(at)::value;
      const int r = r0 + G::kWaveN * wn + 16 * nb + r16;
      const bool row = !E || r < a.N;
      f32x4 g[kHB], u[kHB];
#pragma unroll
      for (int mb = 0; mb < kHB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool there = !E || cw + 16 * mb + 4 * kq + i < a.f;
          g[mb][i] = there ? acc.v[mb][nb][i] : 0.0f;
          u[mb][i] = there ? acc.v[kHB + mb][nb][i] : 0.0f;
        }
      if constexpr (CODES) {
        uint32_t code[2][kHB], e[2][kHB / 2];
#pragma unroll
        for (int p = 0; p < kHB / 2; ++p) {
          codes_of_block(g[2 * p], g[2 * p + 1], code[0][2 * p], code[0][2 * p + 1], e[0][p]);
          codes_of_block(u[2 * p], u[2 * p + 1], code[1][2 * p], code[1][2 * p + 1], e[1][p]);
        }
        const int64_t rz = 2 * static_cast<int64_t>(r);
        // 64 bytes of a row by four lanes: of one half, or half of that of both
#pragma unroll
        for (int o = 0; o < kHB / 2; ++o) {
          u32x4 x = kHB == 4 ? u32x4{code[o][0], code[o][1], code[o][2], code[o][3]}
                             : u32x4{code[0][0], code[0][1], code[1][0], code[1][1]};
          transpose4(x);
          const int h = kHB == 4 ? o : kq >> 1, c = cw + 16 * (kHB == 4 ? kq : kq & 1);
          if (row && (!E || c < a.fp)) *reinterpret_cast<any_u32x4*>(a.codes + (rz + h) * a.fp + c) = x;
        }
        // and the exponents of its blocks by as many lanes as there are
        constexpr int kP = kHB / 2;
        const int h = kq / kP, p = kq % kP, c = cw + 32 * p;
        const uint32_t b = h == 0 ? (p == 0 ? e[0][0] : e[0][kP - 1]) : (p == 0 ? e[1][0] : e[1][kP - 1]);
        if (h < 2 && row && (!E || c < a.fp))
          a.exps[(rz + h) * (a.fp / kBlock8) + c / kBlock8] = static_cast<uint8_t>(b);
      }
#pragma unroll
      for (int mb = 0; mb < kHB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i) g[mb][i] = act_of<ACT>(g[mb][i]) * u[mb][i];
      bf16* const dst = const_cast<bf16*>(a.h.p) + static_cast<int64_t>(r) * a.h.ld + cw;
      const int n = E ? a.ldh - cw : 16 * kHB;
      if constexpr (PARTS == 1) {
        store_strips<kHB, (G::kTile < BigTile::kTile)>(dst, a.h.part, a.two, g, kq, row, n);
      } else {
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
          store_strip<kHB, PARTS>(dst + part * a.h.part, g, kq, row, n);
      }
    });
  });
}

// From G, U and dH of MB blocks of 16 columns of row r from column co on: dG, dU and H,
// written. E: the tile has rows or columns that do not exist, which are zero.
template <int MB, int PARTS, int ACT, bool TWO, bool E>
__device__ __forceinline__ void grad_strip(const GatedArgs& a, int r, int co, int kq, f32x4 (&dg)[MB],
                                           f32x4 (&du)[MB], const f32x4 (&dh)[MB]) {
  constexpr int kAll = 16 * MB;
  const bool row = !E || r < a.N;
  f32x4 hv[MB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool there = !E || (row && co + 16 * mb + 4 * kq + i < a.f);
      const float u = du[mb][i];
      float slope;
      const float v = act_of<ACT>(dg[mb][i], slope);
      hv[mb][i] = there ? v * u : 0.0f;
      du[mb][i] = there ? dh[mb][i] * v : 0.0f;
      dg[mb][i] = there ? dh[mb][i] * u * slope : 0.0f;
    }
  // the caller's own arrays, rows of 2 f and of f
  const int64_t own = static_cast<int64_t>(r) * a.f + co;
  if (!a.dz_out && !a.h_out) {
  } else if constexpr (PARTS == 3) {
    auto store = [&](float* p, const f32x4 (&x)[MB]) {
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        const int c = 16 * mb + 4 * kq;
        if (row && co + c < a.f) store_row(p + c, a.f - co - c, x[mb]);
      }
    };
    if (float* const z = static_cast<float*>(a.dz_out)) {
      store(z + own + static_cast<int64_t>(r) * a.f, dg);
      store(z + own + static_cast<int64_t>(r + 1) * a.f, du);
    }
    if (a.h_out) store(static_cast<float*>(a.h_out) + own, hv);
  } else {
    const int n = E ? a.f - co : kAll;
    if (bf16* const z = static_cast<bf16*>(a.dz_out)) {
      store_strip<MB, 1>(z + own + static_cast<int64_t>(r) * a.f, dg, kq, row, n);
      store_strip<MB, 1>(z + own + static_cast<int64_t>(r + 1) * a.f, du, kq, row, n);
    }
    if (a.h_out) store_strip<MB, 1>(static_cast<bf16*>(a.h_out) + own, hv, kq, row, n);
  }
  // (rows from N on are written up to np, columns up to the end of the padding)
  const bool there = !E || r < a.np;
  bf16* const dz = const_cast<bf16*>(a.dz.p) + static_cast<int64_t>(r) * a.dz.ld + co;
  bf16* const h = const_cast<bf16*>(a.h.p) + static_cast<int64_t>(r) * a.h.ld + co;
  const int ng = E ? a.fq - co : kAll, nu = E ? static_cast<int>(a.dz.ld) - a.fq - co : kAll,
            nh = E ? static_cast<int>(a.h.ld) - co : kAll;
  if constexpr (PARTS == 1) {
    store_strips<MB, TWO>(dz, a.dz.part, a.two, dg, kq, there, ng);
    store_strips<MB, TWO>(dz + a.fq, a.dz.part, a.two, du, kq, there, nu);
    store_strips<MB, TWO>(h, a.h.part, a.two, hv, kq, there, nh);
  } else {
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
      store_strip<MB, PARTS>(dz + part * a.dz.part, dg, kq, there, ng);
      store_strip<MB, PARTS>(dz + part * a.dz.part + a.fq, du, kq, there, nu);
      store_strip<MB, PARTS>(h + part * a.h.part, hv, kq, there, nh);
    }
  }
  __builtin_amdgcn_sched_barrier(0);  // (interleaved strips would need more registers)
}

// Columns that the gradient's tiles cover: up to the end of the padding of H and of dZ's
// second half.
__host__ __device__ __forceinline__ int grad_cols(const GatedArgs& a) {
  const int u = static_cast<int>(a.dz.ld) - a.fq;
  return a.ldh > u ? a.ldh : u;
}

// A tile of dH, from which with G and U in their 8-bit form dG, dU and H follow. 8192 x
// 2048 x 8192: 328 us, of which the product is 215; the rest is the epilogues' 540 MB,
// which all CUs read and write at the same time, and 20 vector instructions a value. (564
// us with strips staged in LDS and registers spilled; 354 with the activation chosen
// inside the kernel.)
template <class G, int PARTS, int ACT>
__global__ __launch_bounds__(G::kThreads, (kBlocksOf<G, PARTS>)) void gate_up_grad_kernel(const GatedArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[kLdsOf<G, PARTS>];
  int mt, nt;
  if (!tile_of_block(blockIdx.x, (grad_cols(a) + G::kTile - 1) / G::kTile,
                     (a.np + G::kTile - 1) / G::kTile, mt, nt))
    return;
  const int c0 = mt * G::kTile, r0 = nt * G::kTile;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave % G::kWavesM, wn = wave / G::kWavesM, r16 = lane & 15, kq = lane >> 4;
  typename G::Acc acc;
  // (columns past the last compute the last ones again, and are written as zero)
  product<G, PARTS, false, false>(rows_of(a.w_out, min(c0, a.f - 1), 0), rows_of(a.dy, r0, 0),
                                  (a.d + kStepK - 1) / kStepK, smem, acc);
  const int cw = c0 + G::kWaveM * wm;  // the wave's first column
  with_edge(r0 + G::kTile > a.N || c0 + G::kTile > a.f, [&](auto edge) {
    constexpr bool E = decltype(edge)::value;
    // 64 columns of the wave's 16 rows at a time, the next ones' codes in flight
    constexpr int kO = G::kMB / 4;
    u32x4 code[2][2];
    uint32_t e[2][2][2];
    auto load = [&](int nb, int o, int to) {
      const int r = r0 + G::kWaveN * wn + 16 * nb + r16, c = cw + 64 * o;
      const int64_t rz = 2 * static_cast<int64_t>(E ? min(r, a.N - 1) : r);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int cc = c + 16 * kq;
        code[to][h] = *reinterpret_cast<const any_u32x4*>(a.codes + (rz + h) * a.fp +
                                                          (E ? min(cc, a.fp - 16) : cc));
#pragma unroll
        for (int p = 0; p < 2; ++p)
          e[to][h][p] = a.exps[(rz + h) * (a.fp / kBlock8) +
                               (E ? min(c + 32 * p, a.fp - 32) : c + 32 * p) / kBlock8];
      }
    };
    load(0, 0, 0);
    each<G::kNB * kO>([&](auto at) {
      constexpr int t = decltype(at)::value, nb = t / kO, o = t % kO, cur = t & 1;
      if constexpr (t + 1 < G::kNB * kO) load((t + 1) / kO, (t + 1) % kO, cur ^ 1);
      transpose4(code[cur][0]);
      transpose4(code[cur][1]);
      f32x4 g[4], u[4], dh[4];
#pragma unroll
      for (int mb = 0; mb < 4; ++mb) {
        const float sg = step8(e[cur][0][mb / 2]), su = step8(e[cur][1][mb / 2]);
        dh[mb] = acc.v[4 * o + mb][nb];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[mb][i] = value8(code[cur][0][mb], i, sg);
          u[mb][i] = value8(code[cur][1][mb], i, su);
        }
      }
      grad_strip<4, PARTS, ACT, (G::kTile < BigTile::kTile), E>(a, r0 + G::kWaveN * wn + 16 * nb + r16, cw + 64 * o, kq, g, u, dh);
    });
  });
}

// The same with G and U computed again: a block takes tiles in turn, computes dH, puts it
// where only it reads, and then both projections of the same columns, half of a wave's
// at a time, in the places where the wave had dH. Two kernels with G and U in fp32 between
// them write and read 16 bytes for every element of dH (16384 x 768 x 2048: 274 us so, 213
// in one; 16384 x 4096 x 11008: 4.15 and 3.59 ms). What bounds it is the products, at 1230
// TFLOP/s of the 1250 to 1340 that a large one of the library reaches, and for short K the
// epilogues between them, which nothing overlaps in a block that has all of LDS. In tiles of
// 256 x 256 it spills 54 to 70 registers (220 to 284 bytes a thread), stored and loaded in
// the epilogues and between the products, none of it in a K loop.
template <class G, int PARTS, int ACT>
__global__ __launch_bounds__(G::kThreads, (kBlocksOf<G, PARTS>)) void gate_up_again_kernel(const GatedArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[kLdsOf<G, PARTS>];
  constexpr int kHB = G::kMB / 2;
  const int mts = (grad_cols(a) + G::kTile - 1) / G::kTile, nts = (a.np + G::kTile - 1) / G::kTile;
  const int steps = (a.d + kStepK - 1) / kStepK, all = (mts * nts + 7) / 8 * 8;
  // the block's dH: 16 bytes a thread for every 16 x 16 block of its wave (through a
  // buffer resource, whose offsets cost no registers)
  const __amdgpu_buffer_rsrc_t mine =
      tile_rsrc(a.scratch + static_cast<int64_t>(blockIdx.x) * (G::kMB * G::kNB * G::kThreads));
  constexpr int kEach = G::kThreads * 16;
  for (int block = blockIdx.x; block < all; block += gridDim.x) {
    int mt, nt;
    if (!tile_of_block(block, mts, nts, mt, nt)) continue;
    const int c0 = mt * G::kTile, r0 = nt * G::kTile;
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));  // (nothing of it is kept from tile to tile)
    const int lane = tid & 63, wave = tid >> 6;
    const int wm = wave % G::kWavesM, wn = wave / G::kWavesM, r16 = lane & 15, kq = lane >> 4;
    typename G::Acc acc;
    __syncthreads();  // the last tile's fragments have been read
    product<G, PARTS, false, false, true>(rows_of(a.w_out, min(c0, a.f - 1), 0), rows_of(a.dy, r0, 0),
                                         steps, smem, acc);
#pragma unroll
    for (int mb = 0; mb < G::kMB; ++mb)
#pragma unroll
      for (int nb = 0; nb < G::kNB; ++nb)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc.v[mb][nb]), mine, tid * 16,
                                               (mb * G::kNB + nb) * kEach, 0);
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      const int ch = c0 + half * (G::kWaveM / 2), cb = min(ch, a.fq - 8);
      Operand w = kmajor_of(a.w_in, 0, cb);
      w.cols = a.fq - cb;
      w.half = a.fq;
      w.apart = true;
      __syncthreads();
      product<G, PARTS, true, false, true>(w, rows_of(a.x, r0, 0), steps, smem, acc);
      const int cw = ch + G::kWaveM * wm;  // the wave's first column of this half
      with_edge(r0 + G::kTile > a.N || c0 + G::kTile > a.f, [&](auto edge) {
        constexpr bool E = decltype(edge)::value;
        f32x4 dh[2][kHB];
        auto load = [&](int nb, int to) {
#pragma unroll
          for (int mb = 0; mb < kHB; ++mb)
            dh[to][mb] = __builtin_bit_cast(
                f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                           mine, tid * 16, ((half * kHB + mb) * G::kNB + nb) * kEach, 0));
        };
        load(0, 0);
        each<G::kNB>([&](auto at) {
          constexpr int nb = decltype(at)::value;
          if constexpr (nb + 1 < G::kNB) load(nb + 1, (nb + 1) & 1);
          f32x4 g[kHB], u[kHB];
#pragma unroll
          for (int mb = 0; mb < kHB; ++mb) g[mb] = acc.v[mb][nb], u[mb] = acc.v[kHB + mb][nb];
          grad_strip<kHB, PARTS, ACT, (G::kTile < BigTile::kTile), E>(a, r0 + G::kWaveN * wn + 16 * nb + r16, cw, kq, g, u, dh[nb & 1]);
        });
      });
    }
  }
}

// out[n][h m + c] = sum_k b[n][k] a[h][c][k] for the halves h of A (its columns or rows
// half apart): one product, or a part of its K whose sums are added afterwards.
struct ProductArgs {
  Mat a, b;
  int32_t half, halves;
  int32_t m, n;        // columns of a half of the output, rows
  int32_t steps;       // of K
  int32_t splits;
  void* out;           // [n][halves m]
  float* acc;          // [splits][np][ldm], where splits > 1
  int32_t np, ldm;     // rows, and halves times m rounded up to 64
};

template <class G, typename T, int PARTS, bool KA, bool KB>
__device__ __forceinline__ void product_tile(const ProductArgs& a, int block, char* smem) {
  const int mh = (a.m + G::kTile - 1) / G::kTile, nh = (a.n + G::kTile - 1) / G::kTile;
  int mt, nt;
  if (!tile_of_block(block, mh * a.halves, nh * a.splits, mt, nt)) return;
  const int split = nt / nh, half = mt / mh;
  const int m0 = (mt - half * mh) * G::kTile, n0 = (nt - split * nh) * G::kTile;
  const int per = (a.steps + a.splits - 1) / a.splits;
  const int k0 = min(a.steps, split * per), k1 = min(a.steps, k0 + per), kk = k0 * kStepK;
  Operand oa, ob;
  if constexpr (KA) {
    oa = kmajor_of(a.a, kk, half * a.half + m0);
  } else {
    oa = rows_of(a.a, m0, kk);
  }
  if constexpr (KB) ob = kmajor_of(a.b, kk, n0);
  else ob = rows_of(a.b, n0, kk);
  typename G::Acc acc;
  product<G, PARTS, KA, KB>(oa, ob, k1 - k0, smem, acc);
  if (a.splits > 1) {
    const int c = half * (a.ldm / a.halves) + m0;
    add_tile<G>(a.acc + (static_cast<int64_t>(split) * a.np + n0) * a.ldm + c, a.ldm,
                a.ldm / a.halves - m0, false, acc);
    return;
  }
  const int64_t ld = static_cast<int64_t>(a.halves) * a.m;
  T* dst = static_cast<T*>(a.out) + n0 * ld + half * a.m + m0;
  const int n_rows = a.n - n0, n_cols = a.m - m0;
  if constexpr (sizeof(T) == 2) {
    write_tile<G>(smem, dst, ld, n_rows, n_cols,
                  [&](int nb, int mb, int i) { return from_float<bf16>(acc.v[mb][nb][i]); });
  } else {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave % G::kWavesM, wn = wave / G::kWavesM, r16 = lane & 15, kq = lane >> 4;
#pragma unroll
    for (int nb = 0; nb < G::kNB; ++nb) {
      const int r = G::kWaveN * wn + 16 * nb + r16;
      if (r >= n_rows) continue;
#pragma unroll
      for (int mb = 0; mb < G::kMB; ++mb) {
        const int c = G::kWaveM * wm + 16 * mb + 4 * kq;
        if (c < n_cols) store_row(dst + r * ld + c, n_cols - c, acc.v[mb][nb]);
      }
    }
  }
}

template <class G, typename T, int PARTS, bool KA, bool KB>
__global__ __launch_bounds__(G::kThreads, (kBlocksOf<G, PARTS>)) void product_kernel(const ProductArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[kLdsOf<G, PARTS>];
  product_tile<G, T, PARTS, KA, KB>(a, blockIdx.x, smem);
}

// The three products of the gradients in one launch, where none of them takes big tiles:
// each alone leaves CUs idle, and a launch is 3 us of host time (forward and backward of
// 128 x 64 x 256, fp32: 40 us, 45 with three launches).
template <class G, typename T, int PARTS>
__global__ __launch_bounds__(G::kThreads, (kBlocksOf<G, PARTS>)) void three_products_kernel(
    const ProductArgs dx, const ProductArgs dw_in, const ProductArgs dw_out, int first_in, int first_out) {
  __shared__ __attribute__((aligned(1024))) char smem[kLdsOf<G, PARTS>];
  const int block = blockIdx.x;
  if (block < first_in) product_tile<G, T, PARTS, false, false>(dx, block, smem);
  else if (block < first_out) product_tile<G, T, PARTS, true, true>(dw_in, block - first_in, smem);
  else product_tile<G, T, PARTS, true, true>(dw_out, block - first_out, smem);
}

// Sums over the splits of K, rounded: four columns a thread.
template <typename T>
__global__ __launch_bounds__(kThreads) void splits_kernel(const ProductArgs a) {
  const int quads = (a.m + 3) / 4;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t rh = t / quads;
  if (rh >= static_cast<int64_t>(a.n) * a.halves) return;
  const int64_t n = rh / a.halves;
  const int h = static_cast<int>(rh - n * a.halves), c = static_cast<int>(t - rh * quads) * 4;
  const float* src = a.acc + n * a.ldm + h * (a.ldm / a.halves) + c;
  const int64_t stride = static_cast<int64_t>(a.np) * a.ldm;
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < a.splits; s0 += 8) {  // (eight loads in flight)
    f32x4 y[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      y[u] = *reinterpret_cast<const f32x4*>(src + min(s0 + u, a.splits - 1) * stride);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (s0 + u < a.splits) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] += y[u][i];
      }
  }
  T* p = static_cast<T*>(a.out) + rh * a.m + c;
  if (c + 4 <= a.m && is_aligned(p, 4 * sizeof(T))) {
    store4<T>(p, x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < a.m) p[i] = from_float<T>(x[i]);
  }
}

// ---------------------------------------------------------------- few rows --
//
// At most 16 rows (tokens being answered): the weights' bytes are the time, and what
// counts is how many of them are in flight. A block takes 64 columns (of the up and gate
// projections 32 each), its four waves every fourth K step of 32, each on its own: a wave
// copies a step's 32 rows of 128 bytes and 16 rows of X into its own LDS, five steps
// ahead, and waits for nothing but its copies; no barrier until the waves' sums meet.
// H stays in two bf16 parts (2^-17 of it), which costs a product but no bytes that count.

constexpr int kFewRows = 16, kFewK = 32, kFewCols = 64, kFewStages = 6;

struct FewArgs {
  const bf16* w;       // [K][ldw], K-major
  const bf16* x;       // [parts][16 or more][ldx]
  int64_t ldw, ldx, part;
  int32_t N, K, cols;  // rows, columns of a half
  int32_t half;        // columns from a half to the other (gate and up)
  int32_t tiles, splits;
  int32_t act;
  bf16* h;             // gate and up: [2][16][cols]
  int8_t* codes;       // and [N][2][cols], or null
  uint8_t* exps;
  float* acc;          // [splits][16][ldm], or, with one split,
  bf16* out;           // [N][cols]
  int32_t ldm;
};

// Nothing in memory or on the matrix cores moves across.
__device__ __forceinline__ void keep_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

template <bool GATED>
__global__ __launch_bounds__(kThreads, 1) void few_rows_kernel(const FewArgs a) {
  constexpr int kParts2 = GATED ? 1 : 2;         // parts of the rows
  constexpr int kCopies = 4 + kParts2;           // a step's
  constexpr int kStage = 4096 + 1024 * kParts2;  // 32 rows of 64 columns, 16 rows of 32 K
  __shared__ __attribute__((aligned(1024))) char smem[4 * kFewStages * kStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, kq = lane >> 4;
  const int total = a.tiles * a.splits, per = (total + 7) >> 3;
  const int at = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if (static_cast<int>(blockIdx.x >> 3) >= per || at >= total) return;
  const int split = at / a.tiles, tile = at - split * a.tiles;
  const int c0 = tile * (GATED ? kFewCols / 2 : kFewCols);
  const int all = a.K / kFewK, some = (all + a.splits - 1) / a.splits;
  const int s0 = min(all, split * some) + wave, s1 = min(all, (split + 1) * some);
  const int n = s0 < s1 ? (s1 - s0 + 3) / 4 : 0;  // this wave's steps: s0, s0 + 4, ...
  char* const mine = smem + wave * kFewStages * kStage;
  // a copy is 8 rows of 8 chunks; slots as in any k-major tile of 64 columns
  uint32_t off_w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int k = 8 * q + (lane >> 3), c = kslot<8>(k, lane & 7);
    const int col = GATED ? c0 + 8 * (c & 3) + (c >> 2) * a.half : min(c0 + 8 * c, a.cols - 8);
    off_w[q] = static_cast<uint32_t>(k) * static_cast<uint32_t>(a.ldw) * 2u + static_cast<uint32_t>(col) * 2u;
  }
  // and 16 rows of 4 chunks, chunk c of row r in slot c ^ (r / 4 mod 4)
  const int xr = lane >> 2, xc = (lane & 3) ^ ((xr >> 2) & 3);
  const uint32_t off_x = static_cast<uint32_t>(min(xr, a.N - 1)) * static_cast<uint32_t>(a.ldx) * 2u +
                         static_cast<uint32_t>(xc) * 16u;
  auto issue = [&](int i) {  // the wave's step i
    char* const to = mine + (i % kFewStages) * kStage;
    const int64_t k = static_cast<int64_t>(s0 + 4 * i) * kFewK;
    const __amdgpu_buffer_rsrc_t rw = tile_rsrc(a.w + k * a.ldw), rx = tile_rsrc(a.x + k);
#pragma unroll
    for (int q = 0; q < 4; ++q) copy_to_lds(rw, off_w[q], 0, to + q * 1024);
#pragma unroll
    for (int q = 0; q < kParts2; ++q)
      copy_to_lds(q ? tile_rsrc(a.x + a.part + k) : rx, off_x, 0, to + 4096 + q * 1024);
  };
  f32x4 acc[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto use = [&](int i) {
    const char* const from = mine + (i % kFewStages) * kStage;
    bf16x8 fw[4], fx[kParts2];
#pragma unroll
    for (int q = 0; q < kParts2; ++q)
      fx[q] = lds_read_b128(from + 4096 + q * 1024 + r16 * 64 + (kq ^ ((r16 >> 2) & 3)) * 16);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      v4i16 h[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = 8 * kq + 4 * j + (r16 >> 2), c = 16 * m + 4 * (r16 & 3);
        h[j] = lds_read_tr(from + k * 128 + kslot<8>(k, c >> 3) * 16 + (c & 7) * 2);
      }
      fw[m] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
#pragma unroll
    for (int q = kParts2 - 1; q >= 0; --q)
#pragma unroll
      for (int m = 0; m < 4; ++m) acc[m] = mfma<1>(fw[m], fx[q], acc[m]);
  };
  // a step is used once at most the copies of the ones after it are in flight: loads
  // return in order
#pragma unroll
  for (int i = 0; i < kFewStages - 1; ++i)
    if (i < n) issue(i);
  int i = 0;
  for (; i + kFewStages - 1 < n; ++i) {
    issue(i + kFewStages - 1);
    wait_vm_all<kCopies * (kFewStages - 1)>();
    keep_order();
    use(i);
    wait_lgkm0();  // the next step's copies go where this one's were
    keep_order();
  }
  wait_vm_all<0>();
  keep_order();
  for (; i < n; ++i) use(i);
  // the waves' sums, in their order
  __syncthreads();
  f32x4* const sums = reinterpret_cast<f32x4*>(smem);
#pragma unroll
  for (int m = 0; m < 4; ++m) sums[(wave * 4 + m) * 64 + lane] = acc[m];
  __syncthreads();
  // wave w's lanes hold columns 16 w + 4 kq .. + 3 of row r16
  f32x4 x = sums[wave * 64 + lane];
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    const f32x4 y = sums[(w * 4 + wave) * 64 + lane];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] += y[j];
  }
  const int c = 16 * wave + 4 * kq;
  if constexpr (GATED) {
    __syncthreads();
    sums[wave * 64 + lane] = x;
    __syncthreads();
    if (wave >= 2) {  // the 8-bit form of G and of U
      if (!a.codes) return;
      const int h = wave - 2;
      uint32_t code[2], b;
      codes_of_block(sums[2 * h * 64 + lane], sums[(2 * h + 1) * 64 + lane], code[0], code[1], b);
      if (r16 >= a.N) return;
      const int64_t rz = 2 * r16 + h;
#pragma unroll
      for (int m = 0; m < 2; ++m)
        *reinterpret_cast<any_u32*>(a.codes + rz * a.cols + c0 + 16 * m + 4 * kq) = code[m];
      if (kq == 0) a.exps[(rz * a.cols + c0) / kBlock8] = static_cast<uint8_t>(b);
      return;
    }
    if (r16 >= a.N) return;
    const f32x4 u = sums[(wave + 2) * 64 + lane];
    f32x4 hv;
    with_act(a.act, [&](auto act) {
#pragma unroll
      for (int j = 0; j < 4; ++j) hv[j] = act_of<decltype(act)::value>(x[j]) * u[j];
    });
    bf16* const dst = a.h + static_cast<int64_t>(r16) * a.cols + c0 + c;
    f32x4 rest;
    Vec4<bf16>::type v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = from_float<bf16>(hv[j]);
      // (an infinity leaves nothing)
      rest[j] = fabsf(static_cast<float>(v[j])) < INFINITY ? hv[j] - static_cast<float>(v[j]) : 0.0f;
    }
    *reinterpret_cast<Vec4<bf16>::type*>(dst) = v;
    store4<bf16>(dst + kFewRows * static_cast<int64_t>(a.cols), rest[0], rest[1], rest[2], rest[3]);
  } else {
    if (r16 >= a.N || c0 + c >= a.cols) return;
    if (a.splits > 1)
      *reinterpret_cast<f32x4*>(a.acc + (static_cast<int64_t>(split) * kFewRows + r16) * a.ldm + c0 + c) = x;
    else
      store_any4(a.out + static_cast<int64_t>(r16) * a.cols + c0 + c, x);
  }
}

// ------------------------------------------------------------------- host --

enum Tile { kBig, kSmall, kTiny };
// (three parts have no big tiles: their six tiles of a K step would not fit LDS)
template <int PARTS, class F>
void with_tile(Tile t, F fn) {
  if constexpr (PARTS != 3) {
    if (t == kBig) return fn(BigTile());
  }
  if (t == kTiny) fn(TinyTile());
  else fn(SmallTile());
}

// Blocks that the chip holds.
int32_t resident(Tile t, int parts) {
  if (parts == 3) return t == kTiny ? 512 : 256;
  return t == kBig ? 256 : t == kSmall ? 512 : 1024;
}

// Tiles and splits of a product of m x n outputs over `steps` K steps, of operands in
// `parts`; of G and U together, whose tiles have half their width of columns of either
// and which needs all of K, as dH does (kWhole) and the three products of kAgain.
// Modelled on 400 measurements: with c blocks on a CU, a K step takes 1.05 + 0.5 c us in a
// big tile, 0.5 max(1, c) in a small one, 0.34 + 0.13 (c - 1) in a tiny one, a fifth more
// where both operands are read transposed; in three parts 2.5 us in a small tile, 1.05 max(1,
// c) in a tiny one; outputs and partial sums are written at 5.6 TB/s, and adding those up is a launch of 2.5 us and 6.5 TB/s.
// (dW_out of 16384 x 768 x 2048: 64 us in small tiles with 5 splits, 65 big with 10, 90
// tiny with 2; of 128 x 64 x 256: 3.6 tiny, 4.5 small, 7.9 big. dX of 2048 x 2048 x 4096:
// 67 us in small tiles, 73 big with 4 splits, 99 tiny.)
struct Choice {
  Tile tile;
  int32_t splits;
};
enum Kind { kPlain, kBothTransposed, kGateUp, kWhole, kAgain };
Choice choose(int64_t m, int64_t n, int64_t steps, int parts, Kind kind) {
  Choice best{kTiny, 1};
  double best_us = 1e30;
  const double mn = static_cast<double>(m) * static_cast<double>(n) / 1e6;
  for (const Tile t : {kBig, kSmall, kTiny}) {
    if (parts == 3 && t == kBig) continue;
    const uint32_t tile = t == kBig ? BigTile::kTile : t == kSmall ? SmallTile::kTile : TinyTile::kTile;
    const uint32_t slots = resident(t, parts), all_steps = static_cast<uint32_t>(steps);
    const uint32_t tiles = static_cast<uint32_t>(ceil_div(m, kind == kGateUp ? tile / 2 : tile) * ceil_div(n, tile));
    const uint32_t most = kind <= kBothTransposed ? std::max(1u, std::min(slots / tiles, all_steps)) : 1;
    // (a call searches every time: counts a quarter apart, from 4 on)
    for (uint32_t k = 1; k <= most; k += std::max(1u, k / 4)) {
      const uint32_t blocks = tiles * k, rounds = (blocks + slots - 1) / slots;
      const double c = static_cast<double>(std::min(blocks, slots)) / 256;
      double step = t == kBig ? 1.05 + 0.5 * c : t == kSmall ? 0.5 * std::max(1.0, c)
                                                             : 0.34 + 0.13 * std::max(0.0, c - 1.0);
      if (kind == kBothTransposed) step *= 1.2;
      if (parts == kTwo) step *= 2;
      if (parts == 3) step = (t == kSmall ? 2.5 : 1.05 * std::max(1.0, c)) * (kind == kBothTransposed ? 1.15 : 1.0);
      const double around = t == kBig ? 5.0 : t == kSmall ? 3.5 : 3.0;
      double us = static_cast<double>(rounds) *
                  (static_cast<double>((all_steps + k - 1) / k * (kind == kAgain ? 3 : 1)) * step + around);
      us += mn * (k > 1 ? 4.0 * static_cast<double>(k) : 2.0) / 5.6;
      if (k > 1) us += 2.5 + mn * (4.0 * static_cast<double>(k) + 2.0) / 6.5;
      if (us < best_us) best_us = us, best = {t, static_cast<int32_t>(k)};
    }
  }
  return best;
}

struct Call {
  int64_t N, d, f;
  int32_t dtype, act;
};

int check_call_shape(const Call& c) {
  if (c.N < 1 || c.N > (1ll << 22)) return fail(DPG_ERR_INVALID_ARG, "N must be in [1, 2^22]");
  if (c.d < 1 || c.d > (1ll << 16)) return fail(DPG_ERR_INVALID_ARG, "d must be in [1, 2^16]");
  if (c.f < 1 || c.f > (1ll << 16)) return fail(DPG_ERR_INVALID_ARG, "f must be in [1, 2^16]");
  if (c.dtype != DPG_FP32 && c.dtype != DPG_BF16) return fail(DPG_ERR_INVALID_ARG, "unknown dtype");
  return DPG_OK;
}
int check_call(const Call& c) {
  if (const int st = check_call_shape(c)) return st;
  if (c.act != DPG_ACT_SILU && c.act != DPG_ACT_GELU && c.act != DPG_ACT_GELU_TANH)
    return fail(DPG_ERR_INVALID_ARG, "unknown activation");
  return DPG_OK;
}

// bf16: H and dZ are rounded once where they enter their products, which with the rounding
// of the output makes its error 1.41 times that of one rounding, at any size (Y of 17 to 8192
// rows). In two parts it is 1.00 times, for products that cost twice as much. Up to a row of
// tiles of 64 the weights' bytes hide a part of that and the two parts are kept: 64 rows x
// 2048 x 8192: forward 40.4 us, 33.3 with one part, gradients 83 and 68; 32 x 768 x 2048: 16
// and 16, 26 and 23. Beyond they are not: 128 rows x 2048 x 8192: 43 and 37, 103 and 75; 256:
// 54 and 43, 129 and 91. A row's result so depends, by that rounding, on whether the call has
// more than 64 rows.
constexpr int64_t kTwoRows = 64;

// Where everything lies in the workspace. Copies of the operands are planned whatever
// their alignment, since a size depends on shapes alone.
struct Plan {
  int64_t parts, ldx, ldh, fq, ldz, np, fp;
  bool two;    // H and dZ in two parts
  bool whole;  // no rows of dZ and H need padding
  Choice y{}, x{}, wi{}, wo{}, again{};
  int64_t again_blocks = 0;
  int32_t few_splits = 0;  // few rows: parts of f in the second product
  size_t off_x, off_wi, off_wo, off_dy, off_h, off_dz = 0, off_scratch = 0, off_x8 = 0, off_acc = 0,
                                                  off_acc_wi = 0, off_acc_wo = 0, total;
};

// Few rows of bf16 in whole K steps go their own way where the weights are 16-byte
// aligned (4 rows x 2048 x 8192: 30 us, 42 in tiles; 16 rows x 4096 x 11008: 78, where 17
// rows take 88 in tiles; the weights alone are 19 and 52 us of a large copy).
bool few_rows(const Call& c) {
  return c.dtype == DPG_BF16 && c.N <= kFewRows && c.d % kFewK == 0 && c.f % kFewK == 0;
}

size_t acc_bytes(const Choice& c, int64_t halves, int64_t m, int64_t n) {
  return c.splits > 1 ? c.splits * round_up(n, kPad) * halves * round_up(m, 64) * 4 : 0;
}

// What a call needs of the workspace beside its shape.
struct Needs {
  bool grad, again, weights;
  bool layers;     // dZ and H are the caller's, both of them
  bool unaligned;  // some operand or output is not 16-byte aligned
};
Plan plan_gated(const Call& c, const Needs& w) {
  Plan p;
  p.parts = c.dtype == DPG_BF16 ? 1 : 3;
  p.ldx = round_up(c.d, kStepK);
  p.ldh = round_up(c.f, kStepK);
  p.fq = round_up(c.f, 8);
  p.ldz = round_up(2 * p.fq, kStepK);
  p.fp = round_up(c.f, kBlock8);
  // (no more: a tile of rows that do not exist takes as long as any; 1 row x 2048 x 8192, dX
  // with G and U computed again: 84 us with rows padded to 256, 75 so; 64 rows: 81 and 78)
  p.np = round_up(c.N, kStepK);
  static_assert(TinyTile::kTile % kStepK == 0, "every tile has a row of the block");
  const int parts = static_cast<int>(p.parts), later = c.dtype == DPG_BF16 && c.N <= kTwoRows ? kTwo : parts;
  size_t off = 0;
  auto take = [&](int64_t elems, int64_t size) {
    const size_t at = off;
    off += align_up(static_cast<size_t>(elems * size));
    return at;
  };
  // operands are copied where they are split, where their rows are no whole 16 bytes or
  // K steps, and where they do not start on 16 bytes
  const bool copy = p.parts == 3 || w.unaligned, copy_rows = copy || c.d % kStepK;
  p.off_x = take(copy_rows ? p.parts * c.N * p.ldx : 0, 2);
  p.off_wi = take(copy || c.f % 8 ? p.parts * c.d * p.ldz : 0, 2);
  p.off_wo = take(copy || c.d % 8 ? p.parts * c.f * p.ldx : 0, 2);
  p.off_dy = take(w.grad && copy_rows ? p.parts * c.N * p.ldx : 0, 2);
  p.two = c.dtype == DPG_BF16 && c.N <= kTwoRows;
  const int64_t made = p.two ? 2 : p.parts;  // parts of what the kernels make
  // dZ and H go straight to the caller where they need no padding
  p.whole = c.dtype == DPG_BF16 && !p.two && !w.unaligned && c.N % kStepK == 0;
  p.off_h = take(w.layers && p.whole && p.ldh == c.f ? 0 : made * p.np * p.ldh, 2);
  if (!w.grad) {
    p.y = choose(c.d, c.N, p.ldh / kStepK, later, kPlain);
    size_t acc = acc_bytes(p.y, 1, c.d, c.N);
    if (few_rows(c)) {
      // about a block for every CU, each wave with four steps at least
      const int64_t tiles = ceil_div(c.d, kFewCols);
      p.few_splits = static_cast<int32_t>(
          std::max<int64_t>(1, std::min(256 / tiles, c.f / (16 * kFewK))));
      acc = std::max<size_t>(acc, p.few_splits * kFewRows * round_up(c.d, 64) * 4);
    }
    p.off_acc = take(static_cast<int64_t>(acc), 1);
  } else {
    p.off_dz = take(w.layers && p.whole && p.ldz == 2 * c.f ? 0 : made * p.np * p.ldz, 2);
    if (w.again) {
      // three products in one kernel, whose blocks are as many as the chip holds at most
      const int64_t cols = std::max(p.ldh, p.ldz - p.fq);
      p.again = choose(cols, c.N, ceil_div(c.d, kStepK), parts, kAgain);
      auto blocks = [&](auto g) {
        typedef decltype(g) G;
        const int64_t tiles = round_up(ceil_div(cols, G::kTile) * ceil_div(p.np, G::kTile), 8);
        p.again_blocks = std::min<int64_t>(tiles, resident(p.again.tile, parts));
        p.off_scratch = take(p.again_blocks * G::kTile * G::kTile, 4);
      };
      if (p.parts == 3) with_tile<3>(p.again.tile, blocks);
      else with_tile<1>(p.again.tile, blocks);
    }
    p.x = choose(c.d, c.N, p.ldz / kStepK, later, kPlain);
    p.off_acc = take(static_cast<int64_t>(acc_bytes(p.x, 1, c.d, c.N)), 1);
    if (w.weights) {
      p.wi = choose(2 * c.f, c.d, ceil_div(c.N, kStepK), later, kBothTransposed);
      p.wo = choose(c.d, c.f, ceil_div(c.N, kStepK), later, kBothTransposed);
      p.off_acc_wi = take(static_cast<int64_t>(acc_bytes(p.wi, 2, c.f, c.d)), 1);
      p.off_acc_wo = take(static_cast<int64_t>(acc_bytes(p.wo, 1, c.d, c.f)), 1);
      // X read back from 8 bits, whether the call has it so or as it is (a size is asked for
      // without X); never where G and U are computed again, from X as it is
      p.off_x8 = take(w.again ? 0 : c.N * p.ldx, c.dtype == DPG_BF16 ? 2 : 4);
    }
  }
  p.total = off;
  return p;
}

// The operands of one call: the caller's matrices where their rows can be copied 16
// bytes at a time and K needs no padding, else copies in the workspace.
struct Operands {
  PackArgs pack{};
  char* ws;
  bool bf16_in;

  Mat bring(const void* src, int64_t rows, int64_t cols, int64_t halves, int64_t half, int64_t ld,
            size_t off, bool direct) {
    if (direct)
      return {static_cast<const bf16*>(src), halves * cols, 0, static_cast<int32_t>(rows),
              static_cast<int32_t>(halves * cols)};
    PackJob& j = pack.job[pack.n++];
    j = {src, reinterpret_cast<bf16*>(ws + off), ld, rows * ld, static_cast<int32_t>(rows),
         static_cast<int32_t>(cols), static_cast<int32_t>(halves), static_cast<int32_t>(half), pack.waves};
    pack.waves += rows * halves;
    // (one part has no other: 0 apart, for the products whose other operand has two)
    return {j.dst, ld, bf16_in ? 0 : j.part, static_cast<int32_t>(rows), static_cast<int32_t>(ld)};
  }
  void launch(hipStream_t s) {
    if (!pack.n) return;
    const dim3 grid(static_cast<unsigned>(ceil_div(pack.waves, 4)));
    if (bf16_in) hipLaunchKernelGGL(pack_mat_kernel<bf16>, grid, dim3(kThreads), 0, s, pack);
    else hipLaunchKernelGGL(pack_mat_kernel<float>, grid, dim3(kThreads), 0, s, pack);
    pack.n = 0, pack.waves = 0;
  }
};

GatedArgs make_args(const Call& c, const Plan& p) {
  GatedArgs a{};
  a.N = static_cast<int32_t>(c.N), a.d = static_cast<int32_t>(c.d), a.f = static_cast<int32_t>(c.f);
  a.fq = static_cast<int32_t>(p.fq), a.act = c.act;
  a.ldh = static_cast<int32_t>(p.ldh), a.fp = static_cast<int32_t>(p.fp);
  a.two = p.two;
  return a;
}

// The tiles of the kernels that need all of K: of G and U, of dH.
template <typename T>
Tile whole_tile(int64_t m, int64_t n, int64_t d, Kind kind) {
  return choose(m, n, ceil_div(d, kStepK), kParts<T>, kind).tile;
}

template <typename T, bool CODES>
void launch_gate_up(const GatedArgs& a, hipStream_t s) {
  with_tile<kParts<T>>(whole_tile<T>(a.ldh, a.N, a.d, kGateUp), [&](auto g) {
    typedef decltype(g) G;
    with_act(a.act, [&](auto act) {
      hipLaunchKernelGGL((gate_up_kernel<G, kParts<T>, decltype(act)::value, CODES>),
                         tile_grid(ceil_div(a.ldh, G::kTile / 2), ceil_div(a.N, G::kTile)),
                         dim3(G::kThreads), 0, s, a);
    });
  });
}

template <class F>
void with_small(Tile t, F fn) {
  if (t == kTiny) fn(TinyTile());
  else fn(SmallTile());
}

// out = B A^T.
ProductArgs product_args(const Choice& c, const Mat& ma, const Mat& mb, int64_t half, int64_t halves,
                         int64_t m, int64_t n, int64_t k, void* out, char* acc) {
  ProductArgs a{};
  a.a = ma, a.b = mb;
  a.half = static_cast<int32_t>(half), a.halves = static_cast<int32_t>(halves);
  a.m = static_cast<int32_t>(m), a.n = static_cast<int32_t>(n);
  a.steps = static_cast<int32_t>(ceil_div(k, kStepK));
  a.splits = c.splits;
  a.out = out, a.acc = reinterpret_cast<float*>(acc);
  a.np = static_cast<int32_t>(round_up(n, kPad));
  a.ldm = static_cast<int32_t>(halves * round_up(m, 64));
  return a;
}
dim3 product_grid(const ProductArgs& a, int64_t tile) {
  return tile_grid(ceil_div(a.m, tile) * a.halves, ceil_div(a.n, tile) * a.splits);
}
template <typename T>
void launch_splits(const ProductArgs& a, hipStream_t s) {
  if (a.splits > 1)
    hipLaunchKernelGGL(splits_kernel<T>, dim3(blocks_of(static_cast<int64_t>(a.n) * a.halves * ((a.m + 3) / 4), kThreads)),
                       dim3(kThreads), 0, s, a);
}
// fn with the parts of the operands of a product, one of which the kernels made.
template <typename T, class F>
void with_parts(bool two, F fn) {
  if constexpr (sizeof(T) == 2) {
    if (two) return fn(std::integral_constant<int, kTwo>{});
  }
  fn(std::integral_constant<int, kParts<T>>{});
}

// One product in one of the three orders of its operands.
template <typename T, bool KA, bool KB>
void launch_product(Tile tile, bool two, const ProductArgs& a, hipStream_t s) {
  with_tile<kParts<T>>(tile, [&](auto g) {
    typedef decltype(g) G;
    with_parts<T>(two, [&](auto parts) {
      hipLaunchKernelGGL((product_kernel<G, T, decltype(parts)::value, KA, KB>), product_grid(a, G::kTile),
                         dim3(G::kThreads), 0, s, a);
    });
  });
  launch_splits<T>(a, s);
}

template <typename T>
int run_forward(const Call& c, const Plan& p, const void* X, const void* W_in, const void* W_out,
                void* Y, int8_t* codes, uint8_t* exps, char* ws, hipStream_t s) {
  constexpr bool kHalf = sizeof(T) == 2;
  GatedArgs a = make_args(c, p);
  Operands o{{}, ws, kHalf};
  a.x = o.bring(X, c.N, c.d, 1, 0, p.ldx, p.off_x, kHalf && c.d % kStepK == 0 && aligned(X, 16));
  a.w_in = o.bring(W_in, c.d, c.f, 2, p.fq, p.ldz, p.off_wi, kHalf && c.f % 8 == 0 && aligned(W_in, 16));
  a.w_out = o.bring(W_out, c.f, c.d, 1, 0, p.ldx, p.off_wo, kHalf && c.d % 8 == 0 && aligned(W_out, 16));
  o.launch(s);
  a.h = {reinterpret_cast<bf16*>(ws + p.off_h), p.ldh, p.np * p.ldh, a.N, a.ldh};
  a.codes = codes, a.exps = exps;
  if (codes) launch_gate_up<T, true>(a, s);
  else launch_gate_up<T, false>(a, s);
  launch_product<T, true, false>(
      p.y.tile, p.two, product_args(p.y, a.w_out, a.h, 0, 1, c.d, c.N, p.ldh, Y, ws + p.off_acc), s);
  return check_launch("gated block");
}

// The forward pass of few rows. The two parts of H are where the tiles' H would be.
int run_few(const Call& c, const Plan& p, const void* X, const void* W_in, const void* W_out, void* Y,
            int8_t* codes, uint8_t* exps, char* ws, hipStream_t s) {
  FewArgs a{};
  a.N = static_cast<int32_t>(c.N), a.act = c.act;
  a.w = static_cast<const bf16*>(W_in), a.ldw = 2 * c.f;
  a.x = static_cast<const bf16*>(X), a.ldx = c.d;
  a.K = static_cast<int32_t>(c.d), a.cols = a.half = static_cast<int32_t>(c.f);
  a.h = reinterpret_cast<bf16*>(ws + p.off_h);
  a.codes = codes, a.exps = exps;
  a.tiles = static_cast<int32_t>(ceil_div(c.f, kFewCols / 2)), a.splits = 1;
  hipLaunchKernelGGL(few_rows_kernel<true>, tile_grid(a.tiles, 1), dim3(kThreads), 0, s, a);
  FewArgs b{};
  b.N = a.N;
  b.w = static_cast<const bf16*>(W_out), b.ldw = c.d;
  b.x = a.h, b.ldx = c.f, b.part = kFewRows * c.f;
  b.K = static_cast<int32_t>(c.f), b.cols = static_cast<int32_t>(c.d);
  b.tiles = static_cast<int32_t>(ceil_div(c.d, kFewCols)), b.splits = p.few_splits;
  b.acc = reinterpret_cast<float*>(ws + p.off_acc), b.out = static_cast<bf16*>(Y);
  b.ldm = static_cast<int32_t>(round_up(c.d, 64));
  hipLaunchKernelGGL(few_rows_kernel<false>, tile_grid(b.tiles, b.splits), dim3(kThreads), 0, s, b);
  if (b.splits > 1) {
    ProductArgs q{};
    q.m = b.cols, q.n = b.N, q.halves = 1, q.splits = b.splits;
    q.acc = b.acc, q.out = Y, q.np = kFewRows, q.ldm = b.ldm;
    hipLaunchKernelGGL(splits_kernel<bf16>, dim3(blocks_of(c.N * ceil_div(c.d, 4), kThreads)),
                       dim3(kThreads), 0, s, q);
  }
  return check_launch("gated block");
}

bool unaligned(std::initializer_list<const void*> pointers) {
  return std::any_of(pointers.begin(), pointers.end(), [](const void* p) { return !aligned(p, 16); });
}

struct Grads {
  void *dX, *dW_in, *dW_out, *dZ, *H;
};

template <typename T>
int run_backward(const Call& c, const Plan& p, const void* X, const int8_t* x_codes,
                 const uint8_t* x_exps, const void* W_in, const void* W_out, const int8_t* z_codes,
                 const uint8_t* z_exps, const void* dY, const Grads& g, char* ws, hipStream_t s) {
  constexpr bool kHalf = sizeof(T) == 2;
  GatedArgs a = make_args(c, p);
  Operands o{{}, ws, kHalf};
  const bool again = !z_codes;
  if (x_codes && g.dW_in) {
    if (launch_unpack8(x_codes, x_exps, c.N, c.d, ws + p.off_x8, kHalf, p.ldx, s) != hipSuccess)
      return fail(DPG_ERR_HIP, "gated gradient: launch failed");
    if (kHalf) {
      a.x = {reinterpret_cast<bf16*>(ws + p.off_x8), p.ldx, 0, a.N, static_cast<int32_t>(p.ldx)};
    } else {
      a.x = o.bring(ws + p.off_x8, c.N, p.ldx, 1, 0, p.ldx, p.off_x, false);
    }
  } else if (again || g.dW_in) {
    a.x = o.bring(X, c.N, c.d, 1, 0, p.ldx, p.off_x, kHalf && c.d % kStepK == 0 && aligned(X, 16));
  }
  if (again || g.dX)
    a.w_in = o.bring(W_in, c.d, c.f, 2, p.fq, p.ldz, p.off_wi, kHalf && c.f % 8 == 0 && aligned(W_in, 16));
  a.w_out = o.bring(W_out, c.f, c.d, 1, 0, p.ldx, p.off_wo, kHalf && c.d % 8 == 0 && aligned(W_out, 16));
  a.dy = o.bring(dY, c.N, c.d, 1, 0, p.ldx, p.off_dy, kHalf && c.d % kStepK == 0 && aligned(dY, 16));
  o.launch(s);
  const bool own_z = p.whole && g.dZ && p.ldz == 2 * c.f, own_h = p.whole && g.H && p.ldh == c.f;
  bf16* const dz = own_z ? static_cast<bf16*>(g.dZ) : reinterpret_cast<bf16*>(ws + p.off_dz);
  bf16* const h = own_h ? static_cast<bf16*>(g.H) : reinterpret_cast<bf16*>(ws + p.off_h);
  a.np = static_cast<int32_t>(p.np);
  a.dz = {dz, p.ldz, p.np * p.ldz, a.np, static_cast<int32_t>(p.ldz)};
  a.h = {h, p.ldh, p.np * p.ldh, a.np, static_cast<int32_t>(p.ldh)};
  a.codes = const_cast<int8_t*>(z_codes), a.exps = const_cast<uint8_t*>(z_exps);
  a.scratch = reinterpret_cast<f32x4*>(ws + p.off_scratch);
  a.dz_out = own_z ? nullptr : g.dZ;
  a.h_out = own_h ? nullptr : g.H;
  if (again) {
    with_tile<kParts<T>>(p.again.tile, [&](auto t) {
      typedef decltype(t) G;
      with_act(c.act, [&](auto act) {
        hipLaunchKernelGGL((gate_up_again_kernel<G, kParts<T>, decltype(act)::value>),
                           dim3(static_cast<unsigned>(p.again_blocks)), dim3(G::kThreads), 0, s, a);
      });
    });
  } else {
    const int64_t cols = grad_cols(a);
    with_tile<kParts<T>>(whole_tile<T>(cols, c.N, c.d, kWhole), [&](auto t) {
      typedef decltype(t) G;
      with_act(c.act, [&](auto act) {
        hipLaunchKernelGGL((gate_up_grad_kernel<G, kParts<T>, decltype(act)::value>),
                           tile_grid(ceil_div(cols, G::kTile), ceil_div(a.np, G::kTile)),
                           dim3(G::kThreads), 0, s, a);
      });
    });
  }
  // (K runs over the rows that are written: whole steps, zero from N on)
  const int64_t k = round_up(c.N, kStepK);
  const ProductArgs x = product_args(p.x, a.w_in, a.dz, 0, 1, c.d, c.N, p.ldz, g.dX, ws + p.off_acc);
  if (!g.dW_in && !g.dW_out) {
    if (g.dX) launch_product<T, false, false>(p.x.tile, p.two, x, s);
    return check_launch("gated gradient");
  }
  const ProductArgs wi = product_args(p.wi, a.dz, a.x, p.fq, 2, c.f, c.d, k, g.dW_in, ws + p.off_acc_wi);
  const ProductArgs wo = product_args(p.wo, a.dy, a.h, 0, 1, c.d, c.f, k, g.dW_out, ws + p.off_acc_wo);
  if (g.dX && g.dW_in && g.dW_out && p.x.tile != kBig && p.x.tile == p.wi.tile && p.x.tile == p.wo.tile) {
    with_small(p.x.tile, [&](auto t) {
      typedef decltype(t) G;
      const unsigned first_in = product_grid(x, G::kTile).x,
                     first_out = first_in + product_grid(wi, G::kTile).x;
      with_parts<T>(p.two, [&](auto parts) {
        hipLaunchKernelGGL((three_products_kernel<G, T, decltype(parts)::value>),
                           dim3(first_out + product_grid(wo, G::kTile).x), dim3(G::kThreads), 0, s, x, wi,
                           wo, static_cast<int>(first_in), static_cast<int>(first_out));
      });
    });
    launch_splits<T>(x, s), launch_splits<T>(wi, s), launch_splits<T>(wo, s);
    return check_launch("gated gradient");
  }
  if (g.dX) launch_product<T, false, false>(p.x.tile, p.two, x, s);
  if (g.dW_in) launch_product<T, true, true>(p.wi.tile, p.two, wi, s);
  if (g.dW_out) launch_product<T, true, true>(p.wo.tile, p.two, wo, s);
  return check_launch("gated gradient");
}

}  // namespace
}  // namespace dpg

using namespace dpg;

extern "C" {

int dpg_gated_workspace_size(int64_t N, int64_t d, int64_t f, int32_t dtype, int32_t unaligned,
                             size_t* bytes) {
  record_error(DPG_OK, "");
  if (!bytes) return fail(DPG_ERR_INVALID_ARG, "bytes is NULL");
  const Call c{N, d, f, dtype, DPG_ACT_SILU};
  if (const int st = check_call_shape(c)) return st;
  *bytes = plan_gated(c, {false, false, false, false, unaligned != 0}).total;
  return DPG_OK;
}

int dpg_gated(const void* X, const void* W_in, const void* W_out, int64_t N, int64_t d, int64_t f,
              int32_t dtype, int32_t act, void* Y, int8_t* z_codes, uint8_t* z_exps, void* workspace,
              size_t workspace_bytes, void* stream) {
  record_error(DPG_OK, "");
  const Call c{N, d, f, dtype, act};
  if (const int st = check_call(c)) return st;
  if (!X || !W_in || !W_out || !Y) return fail(DPG_ERR_INVALID_ARG, "NULL data pointer");
  if (!z_codes != !z_exps) return fail(DPG_ERR_INVALID_ARG, "z_codes and z_exps go together");
  const bool off = unaligned({X, W_in, W_out});
  const Plan p = plan_gated(c, {false, false, false, false, off});
  if (const int st = check_ws(workspace, workspace_bytes, p.total)) return st;
  char* ws = static_cast<char*>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (few_rows(c) && !off)
    return run_few(c, p, X, W_in, W_out, Y, z_codes, z_exps, ws, s);
  return dtype == DPG_BF16 ? run_forward<bf16>(c, p, X, W_in, W_out, Y, z_codes, z_exps, ws, s)
                           : run_forward<float>(c, p, X, W_in, W_out, Y, z_codes, z_exps, ws, s);
}

int dpg_gated_grad_workspace_size(int64_t N, int64_t d, int64_t f, int32_t dtype, int32_t have_z,
                                  int32_t weights, int32_t layers, int32_t unaligned, size_t* bytes) {
  record_error(DPG_OK, "");
  if (!bytes) return fail(DPG_ERR_INVALID_ARG, "bytes is NULL");
  const Call c{N, d, f, dtype, DPG_ACT_SILU};
  if (const int st = check_call_shape(c)) return st;
  *bytes = plan_gated(c, {true, !have_z, weights != 0, layers != 0, unaligned != 0}).total;
  return DPG_OK;
}

int dpg_gated_grad(const void* X, const int8_t* x_codes, const uint8_t* x_exps, const void* W_in,
                   const void* W_out, const int8_t* z_codes, const uint8_t* z_exps, const void* dY,
                   int64_t N, int64_t d, int64_t f, int32_t dtype, int32_t act, void* dX,
                   void* dW_in, void* dW_out, void* dZ, void* H, void* workspace,
                   size_t workspace_bytes, void* stream) {
  record_error(DPG_OK, "");
  const Call c{N, d, f, dtype, act};
  if (const int st = check_call(c)) return st;
  if (!W_in || !W_out || !dY) return fail(DPG_ERR_INVALID_ARG, "NULL data pointer");
  if (!x_codes != !x_exps) return fail(DPG_ERR_INVALID_ARG, "x_codes and x_exps go together");
  if (!z_codes != !z_exps) return fail(DPG_ERR_INVALID_ARG, "z_codes and z_exps go together");
  if (X && x_codes) return fail(DPG_ERR_INVALID_ARG, "X and its 8-bit form are both given");
  if (!z_codes && !X) return fail(DPG_ERR_INVALID_ARG, "the projections need X, or their 8-bit form");
  if (dW_in && !X && !x_codes) return fail(DPG_ERR_INVALID_ARG, "dW_in needs X, or its 8-bit form");
  if (!dX && !dW_in && !dW_out && !dZ && !H) return fail(DPG_ERR_INVALID_ARG, "no output is asked for");
  const Plan p = plan_gated(c, {true, !z_codes, dW_in || dW_out, dZ && H,
                                unaligned({X, W_in, W_out, dY, dZ, H})});
  if (const int st = check_ws(workspace, workspace_bytes, p.total)) return st;
  char* ws = static_cast<char*>(workspace);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Grads g{dX, dW_in, dW_out, dZ, H};
  return dtype == DPG_BF16
             ? run_backward<bf16>(c, p, X, x_codes, x_exps, W_in, W_out, z_codes, z_exps, dY, g, ws, s)
             : run_backward<float>(c, p, X, x_codes, x_exps, W_in, W_out, z_codes, z_exps, dY, g, ws, s);
}

}  // extern "C"
