// Losses of hidden states X [N][d] against a table E [V][d] of a large
// vocabulary, with their gradients, without an [N][V] array of logits:
// softmax cross entropy, and distillation from a teacher's top k logits.
//
// With z_nv = c x_n . e_v / tau, lse_n = ln sum_v exp z_nv and a sparse target
// distribution q_n (one-hot for cross entropy, tau = 1; softmax of t_n / tau
// over the teacher's entries for distillation):
//   loss_n = tau^2 (sum_j q_nj ln q_nj - sum_j q_nj z_n,id(j) + lse_n)
//   D_nv   = c tau g_n (exp(z_nv - lse_n) - q_nv)
//   dX = D E,  dE = D^T X.
// The logits are computed in tiles: the loss keeps each row's running maximum
// and sum of exponentials per tile, the gradient recomputes the logits of one
// piece of the vocabulary at a time and keeps that piece's D.
//
// Rows without a target take no part: the others are packed together first,
// so that masked rows cost nothing and their contents are never read.
#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include "dpg.h"
#include "dpg_device.hpp"
#include "dpg_internal.hpp"

namespace dpg {
namespace {

constexpr int kPad = 256;     // packed rows and pieces are padded to whole tiles
constexpr int kMaxTop = 1024; // entries of a teacher's row
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// fp32 products on the 16-bit matrix instructions, which are 16 times as fast as
// the fp32 ones.
//
// The logits: every row of X and of E is scaled by a power of two, so that its
// largest magnitude lies in [2^13, 2^14), and split into two fp16 parts of 11
// bits, x = h + l. What is left of an element is at most 2^-23 of it, or 2^-38 of
// its row's largest where that is more (fp16 has no smaller step). A product is
// three fp16 products, all pairs but l l, which is at most 2^-22 of it.
//
// dX and dE: a column of D may hold nothing but tiny entries (an unlikely token),
// which no scale of a row can keep, so the operands are split exactly into three
// bf16 parts of 8 bits, each part truncated, x = h + m + l, with fp32's exponent
// range. A product is six bf16 products, all pairs but m l, l m and l l, below
// 2^-22 of it.
//
// Small products are added first, so that the sum is rounded at its full size
// only in the last pass over K. Loss and dX at 999 x 768 x 32003: 643 us; 802
// with three bf16 parts in the logits too.
template <int PARTS> struct Combos;  // parts of an operand: 1 and 3 bf16, 2 fp16
template <> struct Combos<1> {
  static constexpr int n = 1;
  __device__ __forceinline__ static int a(int) { return 0; }
  __device__ __forceinline__ static int b(int) { return 0; }
};
template <> struct Combos<2> {
  static constexpr int n = 3;  // (l,h) (h,l) (h,h)
  __device__ __forceinline__ static int a(int c) { return (0x001 >> (4 * c)) & 15; }
  __device__ __forceinline__ static int b(int c) { return (0x010 >> (4 * c)) & 15; }
};
template <> struct Combos<3> {
  static constexpr int n = 6;  // (l,h) (h,l) (m,m) (m,h) (h,m) (h,h)
  __device__ __forceinline__ static int a(int c) { return (0x001102 >> (4 * c)) & 15; }
  __device__ __forceinline__ static int b(int c) { return (0x010120 >> (4 * c)) & 15; }
};
// Instead of a count of parts: fp32 operands of which the table is read as it is.
constexpr int kRaw = 0;
// Parts of the logits' operands where the others have PARTS.
template <int PARTS> constexpr int kLogitParts = PARTS == 3 ? 2 : 1;
__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
template <int PARTS>
__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  if constexpr (PARTS == 2)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
template <typename T> constexpr int kParts = sizeof(T) == 4 ? 3 : 1;

// Takes the leading part off a value: x becomes the rest (zero for infinities
// and NaN, whose other parts are zero).
__device__ __forceinline__ bf16 take_part(float& x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  x = (u & 0x7F800000u) == 0x7F800000u ? 0.0f : x - __builtin_bit_cast(float, u & 0xFFFF0000u);
  return __builtin_bit_cast(bf16, static_cast<unsigned short>(u >> 16));
}
__device__ __forceinline__ bf16 take_part(f32x4& v, int i) {
  float x = v[i];
  const bf16 p = take_part(x);
  v[i] = x;
  return p;
}
__device__ __forceinline__ void split3(float x, bf16 (&p)[3]) {
#pragma unroll
  for (int q = 0; q < 3; ++q) p[q] = take_part(x);
}

// Per-call tables in the workspace. Row i of the packed arrays is the i-th
// row that has a target.
struct VocabArgs {
  const void* X;        // [N][d]
  const void* E;        // [V][d]
  const int64_t* ids;   // [N][k] targets
  const float* t;       // [N][k] teacher logits, or null (cross entropy)
  const float* dloss;   // [N]
  int64_t N;
  int32_t V, d, k;
  int32_t ldx;          // row stride of Xp, Ep and dXacc: d rounded up to 64
  int32_t np;           // rows of Xp, D and dXacc: N rounded up to kPad
  float zscale;         // c / tau
  float dscale;         // c tau
  float tau;
  float* loss;          // [N]
  float* lse;           // [N]: written by the loss, read by the gradient
  // workspace
  int32_t* flag;        // [N] distillation: row has a target (kOn), or one whose
                        // entry j has nearly all the weight (kPeaked + j)
  int32_t* count;       // [1] packed rows
  int32_t* row;         // [N] packed -> row
  int32_t* inv;         // [N] row -> packed, -1
  int32_t* target;      // [np] packed: cross entropy's target, else -1
  float* g;             // [np] packed: the factor of dloss c tau that D carries, 0
                        // past the last row
  float* gx;            // bf16: [np] packed: the other one, which dX and Xg carry
  float* lse2;          // [np] packed: lse log2(e), 0 past the last row
  float* q;             // [N][k] target weights (distillation)
  float* ent;           // [N] sum q ln q (distillation)
  float* zt;            // [N][k] packed: logits of the target, or of the
                        // teacher's distinct ids in ascending order
  float* qu;            // [N][k] packed: weights of those ids
  int32_t* nu;          // [N] packed: how many of them the pieces so far held
  uint64_t* bits;       // [N][ldd / 64] packed: the piece's columns that are
                        // teacher ids
  uint16_t* before;     // [N][ldd / 64] packed: index in qu of a word's first
  bf16* Xp;             // [parts][np][ldx] packed rows of X, or null
  bf16* Xg;             // bf16: [np][ldx] packed rows of X times gx for dE, or null
  bf16* Ep;             // [parts][piece][ldx] the piece's rows of E, or null
  _Float16* Xh;         // fp32: [2][np][ldx] packed rows of X for the logits
  _Float16* Eh;         // fp32: [2][piece][ldx] the piece's rows of E for them
  float* sx;            // fp32: [np] scale of a row's logits
  float* se;            // fp32: [piece] scale of a column's logits
  float2* part;         // [col tiles][np] packed: tile maximum and sum, base 2
  bf16* D;              // [parts][np][ldd] packed: one piece of D
  float* dXacc;         // [splits][np][ldx] packed
  int32_t ldd;          // columns of a piece (a multiple of kPad)
  int32_t v0, vn;       // the piece: vocabulary rows v0 .. v0 + vn - 1
  int32_t splits;       // parts of the vocabulary piece dX is summed in
  int32_t splits_e;     // parts of the packed rows dE is summed in
  float* dEacc;         // [splits_e][ldd][ldx], where splits_e > 1
};

// ------------------------------------------------------------------- rows --

// Where a row's factor g = dloss c tau meets its D. With fp32 operands D carries it,
// in three exact parts. With bf16 operands D is rounded once. Where one entry of q has
// most of the weight (cross entropy; a teacher sure of its token), so has one entry of
// D, and all of the row's gradient is off by that entry's rounding: by up to 2^-8, and
// for a whole sample the same way, where its rows share g and p is small. There D
// carries t / (q - p) of that entry instead of g, which makes it -t, of 8 bits at most,
// and dX takes the rest of the factor in fp32 at its end, dE through a second copy of
// the row of X, rounded element by element. Other rows' D has several entries whose
// roundings are independent of each other, and carries g: a second rounding, of X,
// would only add to them. (Errors of dX and dE over those of gradients that are rounded
// once, in 150 cases of 1 to 8192 rows, mean and worst: cross entropy 1.43, 2.1 and 1.39,
// 2.2 with g in D, 1.00, 1.03 and 1.29, 1.48 so; teachers of which few are sure 1.41, 1.7
// and 1.38, 1.7 with g, 1.31, 1.52 and 1.36, 1.52 so. Finding p takes the packing 3 us.)
// kPeaked + j: entry j is that one, of at least kPeak; what D has there is at least
// kPeakD (or D's other entries count as much).
enum { kOff = 0, kOn = 1, kPeaked = 2 };
constexpr float kPeak = 0.75f, kPeakD = 0.25f;

// t for a row whose dE takes the factor g / t with X. 181/128 where g is close to a
// multiple of a quarter of its power of two: such a g moves all of the bf16 values of X
// the same way (1 / 511 none of them), and the rounded copies would be off together,
// by up to 1.9e-3 with t = 1, where 4.7e-4 is left so (400000 normal values, factors
// about every 1/128 of [1, 2) and 1/3). But 1 within 2^-11 of a power of two (g = 1, p
// small), which is then as near, and whose copy of X is exact.
__device__ __forceinline__ float peak_in_d(float g) {
  const float m = 8.0f * __builtin_amdgcn_frexp_mantf(fabsf(g));  // quarters, in [4, 8)
  const bool power = m < 4.0f + 0x1p-9f || m > 8.0f - 0x1p-8f;
  return !power && fabsf(m - rintf(m)) < 0.125f ? 181.0f / 128 : 1.0f;
}

// Distillation: one wave per row. q_j = exp(t_j / tau - m) / sum over the
// entries whose id lies in [0, V); entries outside get q = 0, and a row
// without any weight (no id, or every logit -inf) has no target.
__global__ __launch_bounds__(kThreads) void teacher_kernel(const VocabArgs a) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (n >= a.N) return;
  const int lane = threadIdx.x & 63;
  const int64_t* id = a.ids + n * a.k;
  const float* t = a.t + n * a.k;
  float* q = a.q + n * a.k;
  const float inv_tau = 1.0f / a.tau;
  float m = -INFINITY;
  bool nan = false;
  for (int j = lane; j < a.k; j += 64)
    if (id[j] >= 0 && id[j] < a.V) {
      m = fmaxf(m, t[j]);
      nan |= t[j] != t[j];
    }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  nan = __any(nan);
  const bool on = m > -INFINITY || nan;
  float s = 0.0f, e = 0.0f;
  int top = kMaxTop;  // the first entry with the largest logit
  for (int j = lane; j < a.k; j += 64) {
    float w = 0.0f;
    if (on && id[j] >= 0 && id[j] < a.V) {
      const float x = (t[j] - m) * inv_tau;
      w = expf(x);
      if (t[j] == m) top = min(top, j);
      if (w != 0.0f) e = fmaf(w, x, e);
    }
    q[j] = w;
    s += w;
  }
  s = wave_sum(s);
  e = wave_sum(e);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = min(top, __shfl_xor(top, off, 64));
  for (int j = lane; j < a.k; j += 64) q[j] = on ? q[j] / s : 0.0f;
  if (lane == 0) {
    a.flag[n] = !on ? kOff : 1.0f / s >= kPeak ? kPeaked + top : kOn;  // (the largest q is 1 / s)
    a.ent[n] = on ? e / s - logf(s) : 0.0f;  // sum q ln q, ln q = x - ln s
  }
}

// 16 bytes at any element's address: rows of an odd width start anywhere, and the
// global loads and stores take any address (216 MB of rows of 1001 bf16 packed:
// 145 us element by element, 73 us so).
template <typename T>
struct AnyVec16 {
  typedef typename Vec16<T>::type type __attribute__((aligned(sizeof(T))));
};
// Elements c .. of a row of d, zero beyond it.
template <typename T>
__device__ __forceinline__ typename Vec16<T>::type load_row(const T* src, int c, int d) {
  constexpr int VN = Vec16<T>::N;
  typename Vec16<T>::type x;
  if (c + VN <= d) {
    x = *reinterpret_cast<const typename AnyVec16<T>::type*>(src + c);
  } else {
#pragma unroll
    for (int q = 0; q < VN; ++q) x[q] = c + q < d ? src[c + q] : zero_val<T>();
  }
  return x;
}
// n of a row's elements from p on (all 16 bytes of them, or fewer at its end).
template <typename T>
__device__ __forceinline__ void store_row(T* p, int n, typename Vec16<T>::type x) {
  constexpr int VN = Vec16<T>::N;
  if (n >= VN) {
    *reinterpret_cast<typename AnyVec16<T>::type*>(p) = x;
  } else {
#pragma unroll
    for (int q = 0; q < VN; ++q)
      if (q < n) p[q] = x[q];
  }
}

// One row of d values as parts, zero beyond d, by 64 lanes.
template <typename T>
__device__ __forceinline__ void pack_row(const T* src, bf16* dst, int d, int ldx, int64_t part_stride,
                                         int lane) {
  constexpr int VN = Vec16<T>::N;
  for (int c = lane * VN; c < ldx; c += 64 * VN) {
    const typename Vec16<T>::type x = load_row(src, c, d);
    if constexpr (kParts<T> == 1) {
      *reinterpret_cast<bf16x8*>(dst + c) = x;
    } else {
      Vec4<bf16>::type y[3];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        bf16 p[3];
        split3(x[q], p);
#pragma unroll
        for (int j = 0; j < 3; ++j) y[j][q] = p[j];
      }
#pragma unroll
      for (int j = 0; j < 3; ++j)
        *reinterpret_cast<Vec4<bf16>::type*>(dst + j * part_stride + c) = y[j];
    }
  }
}

// One fp32 row for the logits: scaled, in two fp16 parts; returns the factor that
// undoes the scale. A row with an infinity or NaN is not scaled.
__device__ __forceinline__ float pack_row_half(const float* src, _Float16* dst, int d, int ldx,
                                               int64_t part_stride, int lane) {
  float m = 0.0f;
  for (int c = lane * 4; c < d; c += 256) {
    const f32x4 x = load_row(src, c, d);
#pragma unroll
    for (int q = 0; q < 4; ++q) m = fmaxf(m, fabsf(x[q]));
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  int e = 14;
  if (m > 0.0f && m < INFINITY) e = max(__builtin_amdgcn_frexp_expf(m), -100);
  for (int c = lane * 4; c < ldx; c += 256) {
    const f32x4 x = load_row(src, c, d);
    f16x4 h, l;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float y = ldexpf(x[q], 14 - e);
      h[q] = static_cast<_Float16>(y);
      const float r = y - static_cast<float>(h[q]);
      l[q] = static_cast<_Float16>(fabsf(y) < INFINITY ? r : 0.0f);
    }
    *reinterpret_cast<f16x4*>(dst + c) = h;
    *reinterpret_cast<f16x4*>(dst + part_stride + c) = l;
  }
  return ldexpf(1.0f, e - 14);
}

// Packs rows and table in one launch. Blocks [0, row_blocks - kPadBlocks):
// kPackRows rows of X each. A row's packed index is the number of rows before it that have a
// target, which each block counts for itself (8 bytes of L2 reads for every
// earlier row, instead of a launch that counts and one that waits for it). That
// grows with the square of the rows: with 64 columns 9 us for 8192 rows, 31 for 2^15,
// 0.31 ms for 2^17, and at 2^20 20 ms, more than the products of a small table. The
// kPad / kPackRows blocks after them zero Xp up to the next multiple of kPad.
// The rest: rows of the first piece of the table, where it is packed. Bound by memory
// with a table (107911 rows of 1001 bf16: 73 us, 5.9 TB/s), without by the counts and
// the rows' latency (8192 rows of 4096: 34 us for the loss, 75 for the gradients,
// with the targets' logits and the second copy).
constexpr int kPackRows = 16, kPadBlocks = kPad / kPackRows;
template <typename T>
__global__ __launch_bounds__(kThreads) void pack_kernel(const VocabArgs a, int row_blocks) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int block = static_cast<int>(blockIdx.x);
  if (block >= row_blocks) {
    const int i = (block - row_blocks) * 4 + wave, d = i < a.vn ? a.d : 0;
    const T* src = static_cast<const T*>(a.E) + (static_cast<int64_t>(a.v0) + i) * a.d;
    const int64_t at = static_cast<int64_t>(i) * a.ldx, stride = static_cast<int64_t>(a.ldd) * a.ldx;
    if constexpr (kParts<T> == 3) {
      const float f = pack_row_half(src, a.Eh + at, d, a.ldx, stride, lane);
      if (lane == 0) a.se[i] = f;
    }
    if (a.Ep) pack_row(src, a.Ep + at, d, a.ldx, stride, lane);
    return;
  }
  __shared__ int wave_cnt[4];
  const int n0 = min(block * kPackRows, static_cast<int>(a.N));
  const int64_t* ids = a.ids;
  auto on = [&](int n) {
    if (a.t) return a.flag[n] != kOff;
    const int64_t id = ids[n];
    return id >= 0 && id < a.V;
  };
  int c = 0;
  for (int j0 = tid; j0 < n0; j0 += 8 * kThreads) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int j = j0 + u * kThreads;
      c += on(min(j, n0 - 1)) && j < n0;
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) c += __shfl_xor(c, off, 64);
  if (lane == 0) wave_cnt[wave] = c;
  __syncthreads();
  const int before = (wave_cnt[0] + wave_cnt[1]) + (wave_cnt[2] + wave_cnt[3]);
  // a wave's rows: d columns from src[q] on, to packed row to[q] where it is not
  // negative, side by side, so that their latencies are
  constexpr int R = kPackRows / 4;
  auto pack = [&](const T* const (&src)[R], const int (&to)[R], int d, const float (&gx)[R]) {
    if constexpr (kParts<T> == 1) {
      constexpr int VN = Vec16<T>::N;
      for (int c = lane * VN; c < a.ldx; c += 64 * VN) {
        typename Vec16<T>::type x[R];
#pragma unroll
        for (int q = 0; q < R; ++q)
          if (to[q] >= 0) x[q] = load_row(src[q], c, d);
#pragma unroll
        for (int q = 0; q < R; ++q)
          if (to[q] >= 0) {
            const int64_t at = static_cast<int64_t>(to[q]) * a.ldx + c;
            *reinterpret_cast<bf16x8*>(a.Xp + at) = x[q];
            if (!a.Xg) continue;
#pragma unroll
            for (int i = 0; i < VN; ++i) x[q][i] = from_float<bf16>(gx[q] * static_cast<float>(x[q][i]));
            *reinterpret_cast<bf16x8*>(a.Xg + at) = x[q];
          }
      }
    } else {
#pragma unroll
      for (int q = 0; q < R; ++q) {
        if (to[q] < 0) continue;
        const int64_t at = static_cast<int64_t>(to[q]) * a.ldx, stride = static_cast<int64_t>(a.np) * a.ldx;
        if (a.Xh) {
          const float f = pack_row_half(src[q], a.Xh + at, d, a.ldx, stride, lane);
          if (lane == 0) a.sx[to[q]] = f;
        }
        if (a.Xp) pack_row(src[q], a.Xp + at, d, a.ldx, stride, lane);
      }
    }
  };
  const T* src[R];
  int to[R];
  float gx[R];
  const int pad = block - (row_blocks - kPadBlocks);
  if (pad >= 0) {
    if (tid == 0 && pad == 0) a.count[0] = before;
    const int end = (before + kPad - 1) / kPad * kPad;
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int i = before + pad * kPackRows + q * 4 + wave;
      if (i < end && lane == 0) {
        a.target[i] = -1;
        if (a.dloss) a.g[i] = a.lse2[i] = 0.0f;
      }
      src[q] = static_cast<const T*>(a.X), to[q] = i < end ? i : -1, gx[q] = 1.0f;
    }
    pack(src, to, 0, gx);
    return;
  }
  const int mine = n0 + lane;
  const bool mine_on = lane < kPackRows && mine < a.N && on(mine);
  const uint64_t b = __ballot(mine_on);
  if (wave == 0 && lane < kPackRows && mine < a.N) {
    const int at = before + __popcll(b & ((1ull << lane) - 1));
    if (mine_on) {
      a.row[at] = mine;
      a.target[at] = a.t ? -1 : static_cast<int32_t>(a.ids[mine]);
      if (a.dloss) a.lse2[at] = a.lse[mine] * kLog2e;
    }
    a.inv[mine] = mine_on ? at : -1;
  }
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const int r = q * 4 + wave;
    const bool there = (b >> r) & 1;
    src[q] = static_cast<const T*>(a.X) + static_cast<int64_t>(there ? n0 + r : 0) * a.d;
    to[q] = there ? before + __popcll(b & ((1ull << r) - 1)) : -1;
    gx[q] = 1.0f;
  }
  if (a.dloss) {
    // what D has, but for its factor, at the entry that has most of the weight of a
    // row's target; 0 where there is none
    float peak[R] = {};
    if constexpr (kParts<T> == 1) {
      constexpr int VN = Vec16<T>::N;
      const T* e[R];
      float z[R];
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const int n = n0 + q * 4 + wave;
        int64_t id = 0;
        if (to[q] >= 0 && (!a.t || a.flag[n] >= kPeaked)) {
          const int64_t at = a.t ? static_cast<int64_t>(n) * a.k + a.flag[n] - kPeaked : n;
          id = a.ids[at];
          peak[q] = a.t ? a.q[at] : 1.0f;
        }
        e[q] = static_cast<const T*>(a.E) + id * a.d;
        z[q] = 0.0f;
      }
      for (int c = lane * VN; c < a.d; c += 64 * VN) {
        typename Vec16<T>::type u[R], v[R];
#pragma unroll
        for (int q = 0; q < R; ++q)
          if (peak[q] > 0.0f) u[q] = load_row(src[q], c, a.d), v[q] = load_row(e[q], c, a.d);
#pragma unroll
        for (int q = 0; q < R; ++q)
          if (peak[q] > 0.0f) {
#pragma unroll
            for (int i = 0; i < VN; ++i)
              z[q] = fmaf(static_cast<float>(u[q][i]), static_cast<float>(v[q][i]), z[q]);
          }
      }
#pragma unroll
      for (int q = 0; q < R; ++q) z[q] = wave_sum(z[q]);
#pragma unroll
      for (int q = 0; q < R; ++q)
        if (peak[q] > 0.0f)
          peak[q] -= exp2_((z[q] * a.zscale - a.lse[n0 + q * 4 + wave]) * kLog2e);
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (to[q] < 0) continue;
      const float g = a.dloss[n0 + q * 4 + wave] * a.dscale;
      float gd = g;
      if (peak[q] >= kPeakD) {
        const float t = peak_in_d(g * peak[q]);
        gd = t / peak[q];
        gx[q] = g * peak[q] / t;
      }
      if (lane == 0) {
        a.g[to[q]] = gd;
        if (kParts<T> == 1) a.gx[to[q]] = gx[q];
      }
    }
  }
  pack(src, to, a.d, gx);
}

// Distillation: where a packed row's teacher ids lie in the piece, as one bit
// per column, so that the tiles' epilogues find them; one block per row. The
// row's distinct ids get consecutive places in qu, in ascending order; an id
// named more than once gets its weights' sum, in the order they are named. It writes
// 10 bytes per row and word (4096 rows of 786 words: 20 us, bound by the block's
// dependent phases).
constexpr int kMaxWords = 4096;  // 64-column words of a piece
__global__ __launch_bounds__(kThreads) void teacher_ids_kernel(const VocabArgs a) {
  __shared__ uint32_t half[2 * kMaxWords];
  __shared__ uint16_t first[kMaxWords];
  __shared__ int col[kMaxTop];  // column of entry j in the piece, or -1
  __shared__ float weight[kMaxTop];
  __shared__ int wave_cnt[4], named;
  const int i = blockIdx.x;
  if (i >= a.count[0]) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int words = a.ldd / 64;
  const int64_t n = a.row[i];
  for (int w = tid; w < 2 * words; w += kThreads) half[w] = 0;
  if (tid == 0) named = 0;
  __syncthreads();
  for (int j = tid; j < a.k; j += kThreads) {
    const float q = a.q[n * a.k + j];
    const int64_t at = a.ids[n * a.k + j] - a.v0;
    const int c = at >= 0 && at < a.vn && q != 0.0f ? static_cast<int>(at) : -1;
    col[j] = c;
    weight[j] = q;
    if (c >= 0) {
      atomicOr(&half[c >> 5], 1u << (c & 31));
      atomicAdd(&named, 1);
    }
  }
  __syncthreads();
  auto word = [&](int w) {
    return static_cast<uint64_t>(half[2 * w + 1]) << 32 | half[2 * w];
  };
  int base = a.v0 == 0 ? 0 : a.nu[i];
  const int per = (words + kThreads - 1) / kThreads, w0 = min(words, tid * per),
            w1 = min(words, w0 + per);
  int c = 0;
  for (int w = w0; w < w1; ++w) c += __popcll(word(w));
  int x = c;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(x, off, 64);
    if (lane >= off) x += y;
  }
  if (lane == 63) wave_cnt[wave] = x;
  __syncthreads();
  int at = base + x - c, all = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < wave) at += wave_cnt[w];
    all += wave_cnt[w];
  }
  for (int w = w0; w < w1; ++w) {
    first[w] = static_cast<uint16_t>(at);
    at += __popcll(word(w));
  }
  __syncthreads();
  if (tid == 0) a.nu[i] = base + all;
  const int64_t out = static_cast<int64_t>(i) * words;
  for (int w = tid; w < words; w += kThreads) {
    a.bits[out + w] = word(w);
    a.before[out + w] = first[w];
  }
  for (int j = tid; j < a.k; j += kThreads) {
    const int c = col[j];
    if (c < 0) continue;
    bool again = false;
    float sum = weight[j];
    if (all < named) {  // some id is named twice
      sum = 0.0f;
      for (int l = 0; l < a.k; ++l) {
        if (col[l] != c) continue;
        again |= l < j;
        sum += weight[l];
      }
    }
    if (!again)
      a.qu[static_cast<int64_t>(i) * a.k + first[c >> 6] +
           __popcll(word(c >> 6) & ((1ull << (c & 63)) - 1))] = sum;
  }
}

// --------------------------------------------------------------- products --
//
// One device function computes the three products in tiles of 256 x 256 (8
// waves of 128 x 64, one block per CU) or, where those would not fill the 256
// CUs, 128 x 128 (4 waves of 64 x 64, two blocks per CU), with 16x16x32 matrix
// instructions:
//   logits   M = vocabulary rows (E), N = packed rows (Xp), K = d
//   dX       M = columns (E), N = packed rows (D), K = the vocabulary piece
//   dE       M = columns (Xp), N = vocabulary rows (D), K = packed rows
// so that a row of logits has its maximum and sum within four lanes, and a
// lane holds runs of four columns of D, dX and dE. An operand whose K runs
// along its rows in memory ("rows") is copied as rows of 128 bytes, chunk c of
// row R in slot c ^ (R / 2 mod 8), and read with 16-byte LDS loads; one whose K
// runs down its columns ("k-major") as 64 rows of the tile's width, read with
// the transposing LDS load. The direct copies of A run two K steps ahead of
// their use (three stages), those of B one (two stages): 160 KiB of LDS a CU.
//
// What bounds it is the power limit: the logits of 7187 rows x 4096 against 128000
// columns take 5.4 to 6.2 ms, as the card's power and warmth allow, 1400 to 1220
// TFLOP/s (6.04 ms with the clock at 1.58 GHz and the matrix cores 78 % busy; the
// library's product of 8192 x 4096 x 65536: 1446 TFLOP/s at 1.65 GHz, 84 %).
// Hence the 16x16x32 instructions, which draw less than 32x32x16 (25.0 against 25.7
// ms for loss and gradients at 8192 x 4096 x 128000), and a K loop that keeps copies,
// fragment reads and products apart by scheduling barriers.
//
// Copies never leave their arrays: Xp, Ep and D are padded to whole tiles;
// rows and chunks of E beyond its end are clamped to the last ones, and meet
// zeros of the other operand.

// vmcnt(N) with the other counters left alone.
template <int N> __device__ __forceinline__ void wait_vm_n() {
  static_assert(N < 16, "low four bits of the count");
  __builtin_amdgcn_s_waitcnt(0x0F70 | N);
}

constexpr int kStepK = 64;
// A block's tile, and the blocks of 16 x 16 in a wave's part of it. In a
// wave's accumulator, lane l, register i of block (mb, nb) holds M = 16 mb + 4
// (l / 16) + i, N = 16 nb + l % 16.
template <int TILE, int MB, int NB>
struct Geometry {
  static constexpr int kTile = TILE, kMB = MB, kNB = NB;
  static constexpr int kWaveM = 16 * MB, kWaveN = 16 * NB;
  static constexpr int kWavesM = TILE / kWaveM, kWavesN = TILE / kWaveN;
  static constexpr int kWaves = kWavesM * kWavesN, kThreads = 64 * kWaves;
  static constexpr int kTileBytes = TILE * kStepK * 2;
  static constexpr int kCopies = kTileBytes / 1024 / kWaves;  // a wave's, per step and operand
  static constexpr int kLds = 5 * kTileBytes;
  static constexpr int kBlocks = TILE == 256 ? 1 : 2;  // resident on a CU
  struct Acc {
    f32x4 v[MB][NB];
  };
};
typedef Geometry<256, 8, 4> BigTile;
typedef Geometry<128, 4, 4> SmallTile;
// For logits alone, where there are no more small tiles than CUs: a K step is then the
// latency of its reads and products, not their rate (logits of 185 x 200 against 5003
// columns, fp32, 80 small tiles: 14 us small, 8.5 tiny; 10 x 2000 x 25000, bf16, 196:
// 22 and 20.5; 80 x 1024 x 50304, 393: 19 and 25).
typedef Geometry<64, 4, 1> TinyTile;

// Slot of 16-byte chunk c in row k of a k-major tile. Of the
// transposing read, 16 lanes take 32 bytes from each of four rows, and the
// next 16 the same eight rows further on: the slots of these eight pieces
// differ in their 64 banks.
__device__ __forceinline__ int kslot(int k, int c) { return c ^ (4 * (k & 3)) ^ (2 * ((k >> 3) & 1)); }

struct Operand {
  const bf16* base;     // first row of the tile (rows) or of K (k-major)
  int64_t ld;           // row stride, elements
  int64_t part_stride;  // elements between the bf16 parts
  int rows;             // rows: rows there are from base; k-major: rows of K
  int cols;             // rows: elements of K in a row; k-major: columns from base
};

// The direct copies of one operand: G::kCopies of 1 KiB a wave and step.
template <class G, bool KMAJOR>
struct Copier {
  static constexpr int kChunks = G::kTile / 8;        // k-major: of a row
  static constexpr int kRowsPerCopy = 64 / kChunks;  // k-major
  const char* base;       // of the part
  const char* at;         // k-major: of the K step to copy
  uint32_t kb;            // rows: byte offset of that step; k-major: its K row
  uint32_t ldb;           // row stride, bytes
  uint32_t off[G::kCopies];  // rows: row offset; k-major: K row of the lane
  uint32_t chunk;         // byte offset of the lane's 16 bytes within the row
  uint32_t last;          // rows: last chunk of a row; k-major: last K row
  int64_t part_bytes;

  __device__ __forceinline__ void init(const Operand& o, int lane, int wave) {
    // a wave's copies are 64 (32) rows or 16 K rows apart: one swizzle for all
    static_assert(G::kWaves % 2 == 0 && G::kWaves * kRowsPerCopy % 16 == 0, "copy layout");
    base = at = reinterpret_cast<const char*>(o.base);
    kb = 0;
    ldb = static_cast<uint32_t>(o.ld) * 2u;
    part_bytes = o.part_stride * 2;
#pragma unroll
    for (int q = 0; q < G::kCopies; ++q) {
      const int g = q * G::kWaves + wave;
      if constexpr (!KMAJOR) off[q] = static_cast<uint32_t>(min(g * 8 + (lane >> 3), o.rows - 1)) * ldb;
      else off[q] = static_cast<uint32_t>(g * kRowsPerCopy + lane / kChunks);
    }
    if constexpr (!KMAJOR)
      chunk = static_cast<uint32_t>((lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7)) * 16u;
    else
      chunk = static_cast<uint32_t>(
          min(kslot(kRowsPerCopy * wave + lane / kChunks, lane % kChunks), o.cols / 8 - 1)) * 16u;
    last = KMAJOR ? static_cast<uint32_t>(o.rows - 1) : static_cast<uint32_t>(o.cols) * 2u - 16u;
  }
  // copies q0 .. q1 - 1 of the current K step (kStepK columns or rows)
  __device__ __forceinline__ void issue(char* stage, int wave, int q0, int q1) const {
    const __amdgpu_buffer_rsrc_t rs = tile_rsrc(KMAJOR ? at : base);
    const uint32_t c = min(kb + chunk, last), lim = last - kb;
#pragma unroll
    for (int q = 0; q < G::kCopies; ++q)
      if (q >= q0 && q < q1)
        copy_to_lds(rs, KMAJOR ? min(off[q], lim) * ldb + chunk : off[q] + c, 0,
                    stage + (q * G::kWaves + wave) * 1024);
  }
  __device__ __forceinline__ void next_step() {
    if constexpr (KMAJOR) {
      at += static_cast<uint64_t>(ldb) * kStepK;
      kb += kStepK;
    } else {
      kb += kStepK * 2;
    }
  }
  // the first step of the part `parts` parts further on (or back)
  __device__ __forceinline__ void next_part(int parts) {
    base += parts * part_bytes;
    at = base;
    kb = 0;
  }
};

// Matrix-core operand of a 16 x 16 x 32 product: lane l receives K 32 kk + 8
// (l / 16) .. + 7 of row (k-major: column) c0 + l % 16 of the tile.
template <class G, bool KMAJOR>
__device__ __forceinline__ bf16x8 tile_frag(const char* tile, int kk, int c0, int lane) {
  const int q16 = lane & 15, kq = lane >> 4;
  if constexpr (KMAJOR) {
    // in each group of 16 lanes, lane q addresses four consecutive columns of
    // one row, and the transposing read hands it four rows of one column
    const int n = c0 + 4 * (q16 & 3);
    v4i16 h[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = 32 * kk + 8 * kq + 4 * i + (q16 >> 2);
      h[i] = lds_read_tr(tile + k * (2 * G::kTile) + kslot(k, n >> 3) * 16 + (n & 7) * 2);
    }
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
  } else {
    const int r = c0 + q16, c = 4 * kk + kq;
    return lds_read_b128(tile + r * (kStepK * 2) + (c ^ ((r >> 1) & 7)) * 16);
  }
}

// acc = A B^T over K steps [0, n_k) of every combination of parts.
template <class G, int PARTS, bool KA, bool KB>
__device__ __forceinline__ void tile_product(const Operand& oa, const Operand& ob, int n_k,
                                             char* smem, typename G::Acc& acc) {
  typedef Combos<PARTS> C;
  constexpr int KK = kStepK / 32;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % G::kWavesM, wn = wave / G::kWavesM;
  Copier<G, KA> ca;
  Copier<G, KB> cb;
  ca.init(oa, lane, wave);
  cb.init(ob, lane, wave);
  const int n_steps = n_k * C::n;
  char* const sA = smem;
  char* const sB = smem + 3 * G::kTileBytes;
  // after the last copy of a step: the next step, or with several parts the
  // next combination's first
  int ka = 0, ia = 0, kb = 0, ib = 0;
  if (PARTS > 1) ca.next_part(C::a(0)), cb.next_part(C::b(0));
  auto issue_a = [&](int stage, int q0, int q1) {
    ca.issue(sA + stage * G::kTileBytes, wave, q0, q1);
    if (q1 < G::kCopies) return;
    if (PARTS > 1 && ++ka == n_k) ka = 0, ca.next_part(C::a(ia + 1) - C::a(ia)), ++ia;
    else ca.next_step();
  };
  auto issue_b = [&](int stage, int q0, int q1) {
    cb.issue(sB + stage * G::kTileBytes, wave, q0, q1);
    if (q1 < G::kCopies) return;
    if (PARTS > 1 && ++kb == n_k) kb = 0, cb.next_part(C::b(ib + 1) - C::b(ib)), ++ib;
    else cb.next_step();
  };
  // B's fragments of this sub-step and the next; A's of this one, each
  // replaced by the next sub-step's once its products are issued
  bf16x8 fa[G::kMB], fb[2][G::kNB];
  auto read_a = [&](int m, int sta, int kk) {
    fa[m] = tile_frag<G, KA>(sA + sta * G::kTileBytes, kk, G::kWaveM * wm + 16 * m, lane);
  };
  auto read_b = [&](int n, int stb, int kk, int to) {
    fb[to][n] = tile_frag<G, KB>(sB + stb * G::kTileBytes, kk, G::kWaveN * wn + 16 * n, lane);
  };
#pragma unroll
  for (int m = 0; m < G::kMB; ++m)
#pragma unroll
    for (int n = 0; n < G::kNB; ++n) acc.v[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (n_steps <= 0) return;
  // Copies in issue order: A and B of step 0, B and A of step 1; then during
  // step s, A of step s + 2 in its first sub-step and, after the barrier in its
  // last, B of step s + 2. Before that barrier step s + 1's copies are complete
  // once at most those of A's step s + 2 are in flight: loads return in order.
  issue_a(0, 0, G::kCopies);
  issue_b(0, 0, G::kCopies);
  wait_vm_n<0>();
  lds_barrier();
  if (n_steps > 1) {
    issue_b(1, 0, G::kCopies);
    issue_a(1, 0, G::kCopies);
  }
#pragma unroll
  for (int n = 0; n < G::kNB; ++n) read_b(n, 0, 0, 0);
#pragma unroll
  for (int m = 0; m < G::kMB; ++m) read_a(m, 0, 0);
  static_assert(KK == 2 && G::kCopies <= G::kMB && G::kNB <= G::kMB, "one copy or fragment a row");
  // A's stages of steps s, s + 1 and s + 2, and B's of step s
  int sta = 0, sta1 = 1, sta2 = 2, stb = 0;
  // MORE: there is a step s + 2 (else NEXT, at run time, a step s + 1). The two
  // last steps are an instance of their own: with tests inside one loop body the
  // compiler assumed on joining paths that older fragment reads might be in
  // flight, and made the products wait for the newest.
  auto step = [&](auto more, bool next) {
    constexpr bool MORE = decltype(more)::value;
    const bool NEXT = MORE || next;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      const int cur = kk & 1, nxt = cur ^ 1;
      const bool last = kk + 1 == KK;
#pragma unroll
      for (int m = 0; m < G::kMB; ++m) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < G::kNB; ++n)
          acc.v[m][n] = mfma<PARTS>(fa[m], fb[cur][n], acc.v[m][n]);
        __builtin_amdgcn_sched_barrier(0);
        if (last && m == 0 && NEXT) {
          wait_lgkm0();  // this wave's reads of step s are complete
          wait_vm_n<MORE ? G::kCopies : 0>();
          lds_barrier();
        }
        // the next sub-step's fragments
        if (!last) {
          read_a(m, sta, kk + 1);
          if (m < G::kNB) read_b(m, stb, kk + 1, nxt);
        } else if (NEXT) {
          read_a(m, sta1, 0);
          if (m < G::kNB) read_b(m, stb ^ 1, 0, nxt);
        }
        // the refills
        if (MORE && m < G::kCopies) {
          if (kk == 0) issue_a(sta2, m, m + 1);
          if (last) issue_b(stb, m, m + 1);
        }
      }
    }
    const int t = sta;
    sta = sta1;
    sta1 = sta2;
    sta2 = t;
    stb ^= 1;
  };
  int s = 0;
  for (; s + 2 < n_steps; ++s) step(std::true_type{}, true);
#pragma unroll 1
  for (; s < n_steps; ++s) step(std::false_type{}, s + 1 < n_steps);
}

// acc = A B^T with A the table in fp32, as the caller has it, in 128 x 128 tiles.
// With few rows the table's bytes are the time, and packing it first would read
// and write them two to three times more (30 rows x 1024 against 111117 columns:
// loss 374 us packed, 137 us as it is). A K step of 64 stays in fp32 in LDS and is
// split into three bf16 parts in registers; the six products follow per K step, the
// small ones first. A K step is 32 KiB of A and 48 KiB of B's parts, and one is
// copied while the one before it is used.
// A is as Operand says, in floats: rows (M) by K, or with KMAJOR rows of K by
// columns (M), both with 16-byte aligned rows. n_rows: B's rows that count.
struct RawOperand {
  const float* base;
  int64_t ld;
  int rows, cols;
};
constexpr int kRawStage = 5 * SmallTile::kTileBytes;

template <bool KMAJOR>
__device__ __forceinline__ void raw_product(const RawOperand& oa, const Operand& ob, int n_k,
                                            int n_rows, char* smem, SmallTile::Acc& acc) {
  typedef SmallTile G;
  typedef Combos<3> C;
  const int tid = threadIdx.x, lane = tid & 63, q16 = lane & 15, kq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % G::kWavesM, wn = wave / G::kWavesM;
  // rows: two copies of 32 floats a row for a K step. The copier counts in pairs of
  // bytes, of which a float is two.
  Copier<G, false> ca, cb[3];
  ca.init({reinterpret_cast<const bf16*>(oa.base), oa.ld * 2, 0, oa.rows, oa.cols * 2}, lane, wave);
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    Operand o = ob;
    o.base += q * ob.part_stride;
    cb[q].init(o, lane, wave);
  }
  // k-major: a copy takes two rows of K of 512 bytes; 16-byte chunk c of row k lies in
  // slot c ^ 4 (k / 8 mod 4), so that the four rows that a read touches lie in
  // different banks
  const char* at = reinterpret_cast<const char*>(oa.base);
  const uint32_t ldb = static_cast<uint32_t>(oa.ld) * 4u;
  int left = oa.rows;  // rows of K from the step to copy on
  // rows of B that the waves read: whole blocks, zero past n_rows
  const int read_rows = n_rows <= 16 ? 16 : n_rows <= 32 ? 32 : (n_rows + 63) / 64 * 64;
  const uint32_t last = static_cast<uint32_t>(oa.cols) / 4u - 1u;
  auto issue = [&](char* stage) {
    if constexpr (KMAJOR) {
      const __amdgpu_buffer_rsrc_t rs = tile_rsrc(at);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int g = q * G::kWaves + wave, k = 2 * g + (lane >> 5);
        const uint32_t c = static_cast<uint32_t>((lane & 31) ^ (4 * ((k >> 3) & 3)));
        copy_to_lds(rs, static_cast<uint32_t>(min(k, left - 1)) * ldb + min(c, last) * 16u, 0,
                    stage + g * 1024);
      }
      at += static_cast<uint64_t>(ldb) * kStepK;
      left -= kStepK;
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ca.issue(stage + h * G::kTileBytes, wave, 0, G::kCopies);
        ca.next_step();
      }
    }
    // (a wave's copies of B are 32 rows apart, eight rows each)
#pragma unroll
    for (int q = 0; q < 3; ++q) {
#pragma unroll
      for (int j = 0; j < G::kCopies; ++j)
        if ((j * G::kWaves + wave) * 8 < read_rows)
          cb[q].issue(stage + (2 + q) * G::kTileBytes, wave, j, j + 1);
      cb[q].next_step();
    }
  };
  auto read_a = [&](const char* stage, int kk, int m, bf16x8 (&f)[3]) {
    float x[8];
    const int r = G::kWaveM * wm + 16 * m + q16;
    if constexpr (KMAJOR) {
      const char* p = stage + ((r >> 2) ^ (4 * kq)) * 16 + (r & 3) * 4;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = lds_read_f32(p + (32 * kk + 8 * kq + i) * 512);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 v = __builtin_bit_cast(
            f32x4, lds_read_b128(stage + kk * G::kTileBytes + r * 128 +
                                 ((2 * kq + h) ^ ((r >> 1) & 7)) * 16));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * h + i] = v[i];
      }
    }
    // the first part is truncated, so that no finite value becomes an infinity,
    // the others are rounded: exact as well, and without a test
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float h = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x[i]) & 0xFFFF0000u);
      f[0][i] = static_cast<bf16>(h);
      x[i] -= h;
      f[1][i] = static_cast<bf16>(x[i]);
      f[2][i] = static_cast<bf16>(x[i] - static_cast<float>(f[1][i]));
    }
  };
#pragma unroll
  for (int m = 0; m < G::kMB; ++m)
#pragma unroll
    for (int n = 0; n < G::kNB; ++n) acc.v[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (n_k <= 0) return;
  // NB: blocks of 16 of B's rows that count for this wave. HALF: there are at most 64
  // rows, which all waves take, those of each wn one half of the K step.
  auto run = [&](auto nb, auto half) {
    constexpr int NB = decltype(nb)::value;
    constexpr bool HALF = decltype(half)::value;
    issue(smem);
    for (int s = 0; s < n_k; ++s) {
      const char* stage = smem + (s & 1) * kRawStage;
      wait_lgkm0();  // this wave's reads of step s - 1 are complete
      wait_vm_n<0>();
      lds_barrier();
      if (s + 1 < n_k) issue(smem + ((s + 1) & 1) * kRawStage);
      if constexpr (NB > 0) {
#pragma unroll
        for (int kk0 = 0; kk0 < (HALF ? 1 : 2); ++kk0) {
          const int kk = HALF ? wn : kk0;
          bf16x8 fb[3][NB];
#pragma unroll
          for (int q = 0; q < 3; ++q)
#pragma unroll
            for (int n = 0; n < NB; ++n)
              fb[q][n] = tile_frag<G, false>(stage + (2 + q) * G::kTileBytes, kk,
                                             (HALF ? 0 : G::kWaveN * wn) + 16 * n, lane);
#pragma unroll
          for (int m = 0; m < G::kMB; ++m) {
            bf16x8 fa[3];
            read_a(stage, kk, m, fa);
#pragma unroll
            for (int c = 0; c < C::n; ++c)
#pragma unroll
              for (int n = 0; n < NB; ++n)
                acc.v[m][n] = mfma<3>(fa[C::a(c)], fb[C::b(c)][n], acc.v[m][n]);
          }
        }
      }
    }
  };
  if (n_rows > G::kWaveN) {
    if (wn == 0 || n_rows > G::kWaveN + 32) run(std::integral_constant<int, 4>{}, std::false_type{});
    else run(std::integral_constant<int, 2>{}, std::false_type{});
    return;
  }
  if (n_rows <= 16) run(std::integral_constant<int, 1>{}, std::true_type{});
  else if (n_rows <= 32) run(std::integral_constant<int, 2>{}, std::true_type{});
  else run(std::integral_constant<int, 4>{}, std::true_type{});
  // the second half's sums join the first's
  f32x4* sums = reinterpret_cast<f32x4*>(smem) + wm * (G::kMB * G::kNB * 64) + lane;
  __syncthreads();
#pragma unroll
  for (int m = 0; m < G::kMB; ++m)
#pragma unroll
    for (int n = 0; n < G::kNB; ++n)
      if (wn == 1) {
        sums[(m * G::kNB + n) * 64] = acc.v[m][n];
        acc.v[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
  __syncthreads();
  if (wn == 0) {
#pragma unroll
    for (int m = 0; m < G::kMB; ++m)
#pragma unroll
      for (int n = 0; n < G::kNB; ++n) acc.v[m][n] += sums[(m * G::kNB + n) * 64];
  }
}

// The tile (m, n) of a block among mt x nt: each XCD takes a
// contiguous run of them, in bands of eight m, so that the blocks an XCD runs
// together share eight A and four B tiles in its L2. False past the last.
__device__ __forceinline__ bool tile_of_block(int block, int mt, int nt, int& m, int& n) {
  const int total = mt * nt;
  const int per = (total + 7) >> 3;
  const int at = (block & 7) * per + (block >> 3);
  if ((block >> 3) >= per || at >= total) return false;
  const int band = at / (8 * nt), in = at - band * 8 * nt;
  const int h = min(8, mt - band * 8);
  m = band * 8 + in % h;
  n = in / h;
  return true;
}

template <class G>
__device__ __forceinline__ int row_tiles(const VocabArgs& a) {
  return (a.count[0] + G::kTile - 1) / G::kTile;
}

// E as an operand of the current piece: packed, or the caller's own.
__device__ __forceinline__ Operand table_operand(const VocabArgs& a, bool kmajor, int row0, int col0) {
  Operand o;
  if (a.Ep) {
    o.base = a.Ep;
    o.ld = a.ldx;
    o.rows = a.ldd - row0;
    o.cols = a.ldx;
  } else {
    o.base = static_cast<const bf16*>(a.E) + static_cast<int64_t>(a.v0) * a.d;
    o.ld = a.d;
    o.rows = a.vn - row0;
    o.cols = a.d;
  }
  o.base += static_cast<int64_t>(row0) * o.ld + col0;
  if (kmajor) o.cols -= col0;
  o.part_stride = static_cast<int64_t>(a.ldd) * a.ldx;
  return o;
}
__device__ __forceinline__ Operand rows_operand(const bf16* base, int64_t ld, int64_t part_stride,
                                                int rows, int cols) {
  Operand o;
  o.base = base;
  o.ld = ld;
  o.part_stride = part_stride;
  o.rows = rows;
  o.cols = cols;
  return o;
}

// The teacher's ids among the columns of a lane's accumulator for one packed
// row: the 64 columns from column c0 of the piece, of them the lane's quarter
// (4 kq .. 4 kq + 3 of every 16).
struct LaneIds {
  uint64_t word;
  __device__ __forceinline__ static int64_t index(const VocabArgs& a, int r, int c0) {
    return static_cast<int64_t>(r) * (a.ldd / 64) + c0 / 64;
  }
  __device__ __forceinline__ void load(const VocabArgs& a, int r, int rows, int c0) {
    word = r < rows ? a.bits[index(a, r, c0)] : 0;
  }
  // fn(column - 4 kq in the accumulator's order, place in qu) for each of them
  template <class F>
  __device__ __forceinline__ void each(const VocabArgs& a, int r, int c0, int kq, F fn) const {
    uint64_t mine = word & (0x000F000F000F000Full << (4 * kq));
    if (!mine) return;
    const int64_t base = static_cast<int64_t>(r) * a.k + a.before[index(a, r, c0)];
    while (mine) {
      const int b = __ffsll(static_cast<unsigned long long>(mine)) - 1;
      mine &= mine - 1;
      fn(b - 4 * kq, base + __popcll(word & ((1ull << b) - 1)));
    }
  }
};

// A tile of logits before their scale, E's rows against packed rows: with fp32
// operands the columns' scales are taken out, the rows' are left to the caller.
template <class G, int PARTS>
__device__ __forceinline__ void logits_tile(const VocabArgs& a, int c0, int r0, char* smem,
                                            typename G::Acc& acc) {
  constexpr int LP = kLogitParts<PARTS>;
  if constexpr (PARTS == kRaw) {
    const RawOperand e = {static_cast<const float*>(a.E) + (static_cast<int64_t>(a.v0) + c0) * a.d,
                          a.d, a.vn - c0, a.d};
    raw_product<false>(e, rows_operand(a.Xp + static_cast<int64_t>(r0) * a.ldx, a.ldx,
                                       static_cast<int64_t>(a.np) * a.ldx, G::kTile, a.ldx),
                       a.ldx / kStepK, a.count[0] - r0, smem, acc);
    return;
  }
  const bf16* x = LP == 2 ? reinterpret_cast<const bf16*>(a.Xh) : a.Xp;
  const Operand rows = rows_operand(x + static_cast<int64_t>(r0) * a.ldx, a.ldx,
                                    static_cast<int64_t>(a.np) * a.ldx, G::kTile, a.ldx);
  const Operand table =
      LP == 2 ? rows_operand(reinterpret_cast<const bf16*>(a.Eh) + static_cast<int64_t>(c0) * a.ldx,
                             a.ldx, static_cast<int64_t>(a.ldd) * a.ldx, G::kTile, a.ldx)
              : table_operand(a, false, c0, 0);
  tile_product<G, LP, false, false>(table, rows, a.ldx / kStepK, smem, acc);
  if constexpr (LP == 2) {
    const int lane = threadIdx.x & 63, wm = (threadIdx.x >> 6) % G::kWavesM;
    const float* se = a.se + c0 + G::kWaveM * wm + 4 * (lane >> 4);
#pragma unroll
    for (int mb = 0; mb < G::kMB; ++mb) {
      const f32x4 f = *reinterpret_cast<const f32x4*>(se + 16 * mb);
#pragma unroll
      for (int nb = 0; nb < G::kNB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc.v[mb][nb][i] *= f[i];
    }
  }
}
// The scale that logits_tile left to packed row r.
template <int PARTS>
__device__ __forceinline__ float row_scale(const VocabArgs& a, int r) {
  return PARTS == 3 ? a.sx[r] : 1.0f;
}

// LDS of a logits kernel, and its blocks on a CU.
template <class G, int PARTS> constexpr int kLdsOf = PARTS == kRaw ? 2 * kRawStage : G::kLds;
template <class G, int PARTS> constexpr int kBlocksOf = PARTS == kRaw ? 1 : G::kBlocks;

// fn(std::true_type) where a tile reaches past the piece's last column,
// fn(std::false_type) for the others, whose columns need no test.
template <class F>
__device__ __forceinline__ void with_edge(bool edge, F fn) {
  if (edge) fn(std::true_type{});
  else fn(std::false_type{});
}

// Each row's maximum and sum of exponentials over a tile's columns, and the
// logits of the targets there. Works in base 2: z log2(e). What a row needs is
// loaded before the product, so that its latency hides behind it.
template <class G, int PARTS, bool TEACHER>
__global__ __launch_bounds__(G::kThreads, (kBlocksOf<G, PARTS>)) void stats_kernel(const VocabArgs a,
                                                                               int tile0) {
  __shared__ __attribute__((aligned(1024))) char smem[kLdsOf<G, PARTS>];
  int mt, nt;
  if (!tile_of_block(blockIdx.x, (a.vn + G::kTile - 1) / G::kTile, row_tiles<G>(a), mt, nt)) return;
  const int c0 = mt * G::kTile, r0 = nt * G::kTile;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave % G::kWavesM, wn = wave / G::kWavesM, r16 = lane & 15, kq = lane >> 4;
  const int cl = c0 + G::kWaveM * wm + 4 * kq, rl = r0 + G::kWaveN * wn + r16;  // the lane's first
  LaneIds ids[G::kNB][G::kWaveM / 64];
  int at[G::kNB];
#pragma unroll
  for (int nb = 0; nb < G::kNB; ++nb) {
    if constexpr (TEACHER) {
#pragma unroll
      for (int h = 0; h < G::kWaveM / 64; ++h)
        ids[nb][h].load(a, rl + 16 * nb, a.count[0], c0 + G::kWaveM * wm + 64 * h);
    } else {
      at[nb] = a.target[rl + 16 * nb];
    }
  }
  typename G::Acc acc;
  logits_tile<G, PARTS>(a, c0, r0, smem, acc);
  const int left = a.vn - cl;
  float zrow[G::kNB], m[G::kNB], s[G::kNB];
#pragma unroll
  for (int nb = 0; nb < G::kNB; ++nb) zrow[nb] = a.zscale * row_scale<PARTS>(a, rl + 16 * nb);
#pragma unroll
  for (int nb = 0; nb < G::kNB; ++nb) {
    auto logit = [&](int at, float* to) {  // (written where the lane holds it)
      float z = 0.0f;
#pragma unroll
      for (int mb = 0; mb < G::kMB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i) z = at == 16 * mb + i ? acc.v[mb][nb][i] : z;
      if ((at & 15) < 4) *to = z * zrow[nb];
    };
    const int r = rl + 16 * nb;
    if constexpr (TEACHER) {
#pragma unroll
      for (int h = 0; h < G::kWaveM / 64; ++h)
        ids[nb][h].each(a, r, c0 + G::kWaveM * wm + 64 * h, kq, [&](int at, int64_t place) { logit(64 * h + at, a.zt + place); });
    } else {
      const int c = at[nb] - a.v0 - cl;
      if (at[nb] >= 0 && c >= 0 && c < G::kWaveM) logit(c, a.zt + r);
    }
  }
  if (a.zscale < 0.0f) {
#pragma unroll
    for (int mb = 0; mb < G::kMB; ++mb)
#pragma unroll
      for (int nb = 0; nb < G::kNB; ++nb)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc.v[mb][nb][i] = -acc.v[mb][nb][i];
  }
  with_edge(c0 + G::kTile > a.vn, [&](auto edge) {
    constexpr bool E = decltype(edge)::value;
#pragma unroll
    for (int nb = 0; nb < G::kNB; ++nb) {
      float x = -INFINITY;
#pragma unroll
      for (int mb = 0; mb < G::kMB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!E || 16 * mb + i < left) x = fmaxf(x, acc.v[mb][nb][i]);
      x = fmaxf(x, __shfl_xor(x, 16, 64));
      x = fmaxf(x, __shfl_xor(x, 32, 64));
      const float z2 = fabsf(zrow[nb]) * kLog2e;
      // (a wave whose columns all lie past the end has no maximum)
      const float ref = x == -INFINITY ? 0.0f : x * z2;
      float t = 0.0f;
#pragma unroll
      for (int mb = 0; mb < G::kMB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!E || 16 * mb + i < left) t += exp2_(fmaf(acc.v[mb][nb][i], z2, -ref));
      t += __shfl_xor(t, 16, 64);
      t += __shfl_xor(t, 32, 64);
      m[nb] = x == -INFINITY ? x : ref;
      s[nb] = t;
    }
  });
  // the waves that share a row
  float2* red = reinterpret_cast<float2*>(smem);
  __syncthreads();
  if (kq == 0)
#pragma unroll
    for (int nb = 0; nb < G::kNB; ++nb)
      red[wm * G::kTile + G::kWaveN * wn + 16 * nb + r16] = make_float2(m[nb], s[nb]);
  __syncthreads();
  if (tid < G::kTile) {
    float2 p[G::kWavesM];
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < G::kWavesM; ++w) {
      p[w] = red[w * G::kTile + tid];
      mm = fmaxf(mm, p[w].x);
    }
    const float ref = mm == -INFINITY ? 0.0f : mm;
    float ss = 0.0f;
#pragma unroll
    for (int w = 0; w < G::kWavesM; ++w) ss = fmaf(p[w].y, exp2_(p[w].x - ref), ss);
    a.part[static_cast<int64_t>(tile0 + mt) * a.np + r0 + tid] = make_float2(mm, ss);
  }
}

// A tile of bf16 values, staged in LDS and written in whole rows: an accumulator
// value's N is its row, its M its column. Rows >= n_rows and columns >= n_cols are
// not written. 16-byte chunk c of row R sits in slot c ^ (R mod the chunks of a row).
template <class G, class F>
__device__ __forceinline__ void write_tile(char* smem, bf16* dst, int64_t ld, int n_rows, int n_cols,
                                           F value) {
  constexpr int kRow = 2 * G::kTile, kChunks = kRow / 16, kPer = 64 / kChunks;  // rows a wave writes
  static_assert(G::kTile * kRow <= G::kLds, "the staged tile fits");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave % G::kWavesM, wn = wave / G::kWavesM, r16 = lane & 15, kq = lane >> 4;
  __syncthreads();
#pragma unroll
  for (int nb = 0; nb < G::kNB; ++nb) {
    const int r = G::kWaveN * wn + 16 * nb + r16;
#pragma unroll
    for (int mb = 0; mb < G::kMB; ++mb) {
      Vec4<bf16>::type v;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = value(nb, mb, q);
      const int c = G::kWaveM / 8 * wm + 2 * mb + (kq >> 1);
      *reinterpret_cast<Vec4<bf16>::type*>(smem + r * kRow + (c ^ (r % kChunks)) * 16 + (kq & 1) * 8) = v;
    }
  }
  __syncthreads();
#pragma unroll
  for (int it = 0; it < G::kTile / (kPer * G::kWaves); ++it) {
    const int r = (it * G::kWaves + wave) * kPer + lane / kChunks, c = lane % kChunks;
    const bf16x8 v = lds_read_b128(smem + r * kRow + (c ^ (r % kChunks)) * 16);
    if (r < n_rows && c * 8 < n_cols)
      store_row(dst + static_cast<int64_t>(r) * ld + c * 8, n_cols - c * 8, v);
  }
}

// One tile of D for the piece: g_n (exp(z - lse_n) - q), zero beyond the piece and
// the packed rows. One rounding to bf16, after the target's weight is subtracted: D
// enters two products whose other operand is bf16; with fp32 D is kept in three
// parts.
template <class G, int PARTS, bool TEACHER>
__global__ __launch_bounds__(G::kThreads, (kBlocksOf<G, PARTS>)) void grad_logits_kernel(
    const VocabArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[kLdsOf<G, PARTS>];
  int mt, nt;
  if (!tile_of_block(blockIdx.x, (a.vn + G::kTile - 1) / G::kTile, row_tiles<G>(a), mt, nt)) return;
  const int c0 = mt * G::kTile, r0 = nt * G::kTile;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave % G::kWavesM, wn = wave / G::kWavesM, r16 = lane & 15, kq = lane >> 4;
  const int cl = c0 + G::kWaveM * wm + 4 * kq, rl = r0 + G::kWaveN * wn + r16;  // the lane's first
  LaneIds ids[G::kNB][G::kWaveM / 64];
  int at[G::kNB];
  float g[G::kNB], lse2[G::kNB];
#pragma unroll
  for (int nb = 0; nb < G::kNB; ++nb) {
    if constexpr (TEACHER) {
#pragma unroll
      for (int h = 0; h < G::kWaveM / 64; ++h)
        ids[nb][h].load(a, rl + 16 * nb, a.count[0], c0 + G::kWaveM * wm + 64 * h);
    } else {
      at[nb] = a.target[rl + 16 * nb];
    }
  }
  auto load_rows = [&] {
#pragma unroll
    for (int nb = 0; nb < G::kNB; ++nb) {
      g[nb] = a.g[rl + 16 * nb];
      lse2[nb] = a.lse2[rl + 16 * nb];
    }
  };
  // (with the teacher's bits or two parts of each operand the registers are full)
  constexpr bool kEarly = !TEACHER && PARTS == 1;
  if (kEarly) load_rows();
  typename G::Acc acc;
  logits_tile<G, PARTS>(a, c0, r0, smem, acc);
  if (!kEarly) load_rows();
  const int left = a.vn - cl;
  float z2[G::kNB];
#pragma unroll
  for (int nb = 0; nb < G::kNB; ++nb) z2[nb] = a.zscale * kLog2e * row_scale<PARTS>(a, rl + 16 * nb);
  with_edge(c0 + G::kTile > a.vn, [&](auto edge) {
    constexpr bool E = decltype(edge)::value;
#pragma unroll
    for (int nb = 0; nb < G::kNB; ++nb)
#pragma unroll
      for (int mb = 0; mb < G::kMB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = g[nb] * exp2_(fmaf(acc.v[mb][nb][i], z2[nb], -lse2[nb]));
          acc.v[mb][nb][i] = !E || 16 * mb + i < left ? x : 0.0f;
        }
  });
#pragma unroll
  for (int nb = 0; nb < G::kNB; ++nb) {
    auto subtract = [&](int at, float q) {
#pragma unroll
      for (int mb = 0; mb < G::kMB; ++mb)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc.v[mb][nb][i] -= at == 16 * mb + i ? q : 0.0f;
    };
    if constexpr (TEACHER) {
#pragma unroll
      for (int h = 0; h < G::kWaveM / 64; ++h)
        ids[nb][h].each(a, rl + 16 * nb, c0 + G::kWaveM * wm + 64 * h, kq,
                        [&](int at, int64_t place) { subtract(64 * h + at, g[nb] * a.qu[place]); });
    } else {
      const int c = at[nb] - a.v0 - cl;
      if (at[nb] >= 0 && c >= 0 && c < G::kWaveM) subtract(c, g[nb]);
    }
  }
  bf16* dst = a.D + static_cast<int64_t>(r0) * a.ldd + c0;
  if constexpr (PARTS == 1) {
    write_tile<G>(smem, dst, a.ldd, G::kTile, G::kTile,
               [&](int nb, int mb, int i) { return from_float<bf16>(acc.v[mb][nb][i]); });
  } else {
#pragma unroll
    for (int q = 0; q < 3; ++q)
      write_tile<G>(smem, dst + static_cast<int64_t>(q) * a.np * a.ldd, a.ldd, G::kTile, G::kTile,
                 [&](int nb, int mb, int i) { return take_part(acc.v[mb][nb], i); });
  }
}

// Writes a tile to rows of ld floats, or adds it to them: an accumulator value's N
// is its row, its M its column. Columns >= n_cols (a multiple of 16) stay.
template <class G>
__device__ __forceinline__ void add_tile(float* dst, int64_t ld, int n_cols, bool add,
                                         const typename G::Acc& acc) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave % G::kWavesM, wn = wave / G::kWavesM, r16 = lane & 15, kq = lane >> 4;
#pragma unroll
  for (int mb = 0; mb < G::kMB; ++mb) {
    const int c = G::kWaveM * wm + 16 * mb;
    if (c >= n_cols) continue;
#pragma unroll
    for (int nb = 0; nb < G::kNB; ++nb) {
      f32x4* p = reinterpret_cast<f32x4*>(
          dst + static_cast<int64_t>(G::kWaveN * wn + 16 * nb + r16) * ld + c + 4 * kq);
      f32x4 x = acc.v[mb][nb];
      if (add) {
        const f32x4 y = *p;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] += y[i];
      }
      *p = x;
    }
  }
}

// dXacc[split] (+)= D E over the split's part of the piece.
template <class G, int PARTS>
__device__ __forceinline__ void dx_tile(const VocabArgs& a, int block, char* smem) {
  int mt, nt;
  const int ct = (a.ldx + G::kTile - 1) / G::kTile;
  if (!tile_of_block(block, row_tiles<G>(a), ct * a.splits, mt, nt)) return;
  const int split = nt / ct;
  const int c0 = (nt - split * ct) * G::kTile, r0 = mt * G::kTile;
  const int steps = (a.vn + kStepK - 1) / kStepK, per = (steps + a.splits - 1) / a.splits;
  const int k0 = min(steps, split * per), k1 = min(steps, k0 + per);
  typename G::Acc acc;
  const Operand d = rows_operand(a.D + static_cast<int64_t>(r0) * a.ldd + k0 * kStepK, a.ldd,
                                 static_cast<int64_t>(a.np) * a.ldd, G::kTile, a.ldd - k0 * kStepK);
  if constexpr (PARTS == kRaw) {
    const int64_t row = static_cast<int64_t>(a.v0) + k0 * kStepK;
    const RawOperand e = {static_cast<const float*>(a.E) + row * a.d + c0, a.d, a.vn - k0 * kStepK,
                          a.d - c0};
    raw_product<true>(e, d, k1 - k0, a.count[0] - r0, smem, acc);
  } else {
    tile_product<G, PARTS, true, false>(table_operand(a, true, k0 * kStepK, c0), d, k1 - k0, smem, acc);
  }
  add_tile<G>(a.dXacc + (static_cast<int64_t>(split) * a.np + r0) * a.ldx + c0, a.ldx, a.ldx - c0,
              a.v0 != 0, acc);
}

// The piece's rows of dE = D^T X, rounded once; with several splits of the packed
// rows, each split's sums.
template <class G, typename T>
__device__ __forceinline__ void de_tile(const VocabArgs& a, T* dE, int block, char* smem) {
  constexpr int PARTS = kParts<T>;
  int mt, nt;
  const int ct = (a.ldx + G::kTile - 1) / G::kTile;
  // (bands of eight run over the vocabulary, the longer side)
  if (!tile_of_block(block, (a.vn + G::kTile - 1) / G::kTile, ct * a.splits_e, nt, mt)) return;
  const int split = mt / ct;
  const int c0 = (mt - split * ct) * G::kTile, w0 = nt * G::kTile;
  const int steps = (a.count[0] + kStepK - 1) / kStepK, per = (steps + a.splits_e - 1) / a.splits_e;
  const int k0 = min(steps, split * per), k1 = min(steps, k0 + per);
  const int64_t row = static_cast<int64_t>(k0) * kStepK;
  typename G::Acc acc;
  tile_product<G, PARTS, true, true>(
      rows_operand((PARTS == 1 ? a.Xg : a.Xp) + row * a.ldx + c0, a.ldx,
                   static_cast<int64_t>(a.np) * a.ldx, a.np - k0 * kStepK, a.ldx - c0),
      rows_operand(a.D + row * a.ldd + w0, a.ldd, static_cast<int64_t>(a.np) * a.ldd,
                   a.np - k0 * kStepK, G::kTile),
      k1 - k0, smem, acc);
  if (a.splits_e > 1) {
    add_tile<G>(a.dEacc + (static_cast<int64_t>(split) * a.ldd + w0) * a.ldx + c0, a.ldx, a.ldx - c0,
                false, acc);
    return;
  }
  T* dst = dE + (static_cast<int64_t>(a.v0) + w0) * a.d + c0;
  const int n_rows = a.vn - w0, n_cols = a.d - c0;
  if constexpr (PARTS == 1) {
    write_tile<G>(smem, dst, a.d, n_rows, n_cols,
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
        store_row(dst + static_cast<int64_t>(r) * a.d + c, n_cols - c, acc.v[mb][nb]);
      }
    }
  }
}

// lse and loss of every row from its tile partials: one wave per row. Bound by the
// partials' latency (12 us for 8192 rows of 197 tiles, 4 us for 4 rows of 393).
__global__ __launch_bounds__(kThreads) void lse_kernel(const VocabArgs a, int tiles) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (n >= a.N) return;
  const int lane = threadIdx.x & 63;
  const int i = a.inv[n];
  if (i < 0) {
    if (lane == 0) a.loss[n] = 0.0f, a.lse[n] = 0.0f;
    return;
  }
  // eight tiles of a lane in flight: with few rows their latency is the time
  float m = -INFINITY, s = 0.0f;
  for (int t0 = lane; t0 < tiles; t0 += 8 * 64) {
    float2 p[8];
    float mm = m;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      p[u] = a.part[static_cast<int64_t>(min(t0 + u * 64, tiles - 1)) * a.np + i];
      if (t0 + u * 64 >= tiles) p[u] = make_float2(-INFINITY, 0.0f);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) mm = fmaxf(mm, p[u].x);
    const float ref = mm == -INFINITY ? 0.0f : mm;
    s *= exp2_(m - ref);
#pragma unroll
    for (int u = 0; u < 8; ++u) s = fmaf(p[u].y, exp2_(p[u].x - ref), s);
    m = mm;
  }
  const float lane_m = m;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  s *= exp2_(lane_m - (m == -INFINITY ? 0.0f : m));
  s = wave_sum(s);
  const float lse = kLn2 * m + logf(s);
  float qz = 0.0f;
  if (a.t) {
    const int64_t at = static_cast<int64_t>(i) * a.k;
    for (int j = lane; j < a.nu[i]; j += 64) qz = fmaf(a.qu[at + j], a.zt[at + j] - lse, qz);
    qz = wave_sum(qz);
  }
  if (lane == 0) {
    a.lse[n] = lse;
    a.loss[n] = a.t ? a.tau * a.tau * (a.ent[n] - qz) : lse - a.zt[i];
  }
}

// The gradients' products of one piece: dX's tiles in blocks [0, dx_blocks), dE's
// in the rest. Small problems run both in one launch; large ones run faster one
// after the other, in kernels of their own (8192 x 4096 x 32768: 3.12 ms
// against 3.23, the two read different arrays, and each compiles better alone).
template <class G, typename T, bool DX, bool DE>
__global__ __launch_bounds__(G::kThreads, G::kBlocks) void products_kernel(const VocabArgs a,
                                                                           int dx_blocks, T* dE) {
  __shared__ __attribute__((aligned(1024))) char smem[G::kLds];
  const int block = blockIdx.x;
  if (DX && (!DE || block < dx_blocks)) dx_tile<G, kParts<T>>(a, block, smem);
  else if (DE) de_tile<G, T>(a, dE, block - dx_blocks, smem);
}

// dX's tiles with the table as the caller has it.
__global__ __launch_bounds__(SmallTile::kThreads, 1) void raw_dx_kernel(const VocabArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[2 * kRawStage];
  dx_tile<SmallTile, kRaw>(a, blockIdx.x, smem);
}

// Row n of a gradient: its sums in `splits` arrays (stride floats apart) of rows
// of a.ldx, added in order and rounded once. With inv, row inv[n] of them, times its
// factor where there are any, and zero where that is negative (a row without
// target). lanes = 2^lane_bits
// threads a row, each four columns at a time, so that narrow rows share a block.
template <typename T>
__global__ __launch_bounds__(kThreads) void out_kernel(const VocabArgs a, const float* sums,
                                                       int64_t stride, int splits, const int32_t* inv,
                                                       const float* factor, int64_t rows,
                                                       int lane_bits, T* out) {
  const int64_t n = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> lane_bits;
  if (n >= rows) return;
  const int64_t i = inv ? inv[n] : n;
  const bool vec = a.d % 4 == 0 && is_aligned(out, 4 * sizeof(T));
  const float* src = sums + (i < 0 ? 0 : i) * a.ldx;
  const float f = factor && i >= 0 ? factor[i] : 1.0f;
  const int lanes = 1 << lane_bits;
  for (int c = (threadIdx.x & (lanes - 1)) * 4; c < a.d; c += lanes * 4) {
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    if (i >= 0)
      for (int s0 = 0; s0 < splits; s0 += 8) {  // (eight loads in flight)
        f32x4 y[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          y[u] = *reinterpret_cast<const f32x4*>(src + min(s0 + u, splits - 1) * stride + c);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (s0 + u < splits) {
#pragma unroll
            for (int q = 0; q < 4; ++q) x[q] += y[u][q];
          }
      }
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] *= f;
    T* p = out + n * a.d + c;
    if (vec) {
      store4<T>(p, x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (c + q < a.d) p[q] = from_float<T>(x[q]);
    }
  }
}

// ------------------------------------------------------------------- host --

int fail(int code, const std::string& msg) { return record_error(code, msg.c_str()); }

int check_launch(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(DPG_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
  return DPG_OK;
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

// What a call was given.
struct VocabCall {
  const void *X, *E;
  const int64_t* ids;
  const float* t;  // null for cross entropy
  int64_t N, d, V;
  int32_t k, dtype;
  double scale, tau;
};

int check_call_shape(const VocabCall& c) {
  if (c.N < 1 || c.N > (1ll << 22)) return fail(DPG_ERR_INVALID_ARG, "N must be in [1, 2^22]");
  if (c.V < 1 || c.V > (1ll << 22)) return fail(DPG_ERR_INVALID_ARG, "V must be in [1, 2^22]");
  if (c.d < 1 || c.d > (1ll << 16)) return fail(DPG_ERR_INVALID_ARG, "d must be in [1, 2^16]");
  if (c.k < 1 || c.k > kMaxTop) return fail(DPG_ERR_INVALID_ARG, "k must be in [1, 1024]");
  if (c.dtype != DPG_FP32 && c.dtype != DPG_BF16) return fail(DPG_ERR_INVALID_ARG, "unknown dtype");
  return DPG_OK;
}

int check_call(const VocabCall& c, bool distill) {
  if (const int st = check_call_shape(c)) return st;
  if (!std::isfinite(c.scale)) return fail(DPG_ERR_INVALID_ARG, "scale must be finite");
  if (!(c.tau > 0.0) || !std::isfinite(c.tau))
    return fail(DPG_ERR_INVALID_ARG, "temperature must be positive and finite");
  if (!c.X || !c.E || !c.ids || (distill && !c.t)) return fail(DPG_ERR_INVALID_ARG, "NULL data pointer");
  return DPG_OK;
}

// Whether a launch of `tiles` big tiles takes them. Fewer than three for every
// four CUs leave too much of the chip idle, and a K step of a big tile takes 64
// KiB through a CU's LDS where a small one takes 32 (128 rows x 64 against 1000
// columns, fp32: 18 us big, 12 us small; 252 big tiles of a product of six at 999 x
// 768 x 32003: 311 us big, 424 us small). With at most 128 rows half of a big
// tile would be padding (4 rows x 2048 against 50304 columns: 53 us big, 40 us
// small).
bool big_tiles(int64_t tiles, int64_t rows) { return tiles >= 192 && rows > SmallTile::kTile; }

// The logits' tiles for a piece of vn columns, of a table that is packed or not (raw).
enum Tile { kBig, kSmall, kTiny };
Tile logits_tiles(int64_t vn, int64_t N, bool raw) {
  if (big_tiles(ceil_div(vn, BigTile::kTile) * ceil_div(N, BigTile::kTile), N)) return kBig;
  return raw || ceil_div(vn, SmallTile::kTile) * ceil_div(N, SmallTile::kTile) > 256 ? kSmall : kTiny;
}
template <class F>
void with_tile(Tile t, F fn) {
  if (t == kBig) fn(BigTile());
  else if (t == kSmall) fn(SmallTile());
  else fn(TinyTile());
}

// Bytes of D, and of the packed table, kept at a time; of a packed table that
// is needed only where the caller's is not 16-byte aligned. (A last piece of few
// tiles leaves CUs idle: 288 x 1024 x 108627, fp32, loss and dX: 1460 us with a table
// of 512 MiB at a time, 1360 with 1 GiB.)
constexpr int64_t kPieceBytes = 512ll << 20, kTableBytes = 1024ll << 20, kRarePieceBytes = 64ll << 20;

// Tiles and splits of K for an output of m x n values over `steps` K steps of
// `combos` products. Modelled on measurements: a K step takes 1.7 us in a big
// tile, 1.3 in a small one with two on each CU, 0.7 with one, and a block 4 us
// around its steps; the splits' sums are written and read at 4 TB/s. What counts
// is that the last round of blocks leaves few CUs idle.
// dE at 6633 x 576 x 2325, fp32 (30 big tiles of 624 steps): 692 us without
// splits, 145 us with 8 and their sum.
struct Split {
  bool big;
  int32_t splits;
};
Split choose_split(int64_t m, int64_t n, int64_t steps, int combos, bool sums_anyway) {
  Split best{true, 1};
  double best_us = 1e30;
  for (const bool big : {true, false}) {
    const int64_t tile = big ? BigTile::kTile : SmallTile::kTile, slots = big ? 256 : 512;
    const int64_t tiles = ceil_div(m, tile) * ceil_div(n, tile);
    const int64_t most = std::max<int64_t>(1, std::min(slots / tiles, steps / 2));
    // (every count up to 16, then steps of an eighth, and the most)
    for (int64_t k = 1; k <= most; k = k < most ? std::min(k + std::max<int64_t>(1, k / 8), most) : k + 1) {
      const int64_t blocks = tiles * k;
      const double step = big ? 1.7 : blocks > 256 ? 1.3 : 0.7;
      double us = static_cast<double>(ceil_div(blocks, slots)) *
                  (static_cast<double>(ceil_div(steps, k) * combos) * step + 4.0);
      if (k > 1 || sums_anyway)
        us += (sums_anyway ? 0.0 : 5.0) + static_cast<double>(k * m * n) * 8 / 4e6;
      if (us < best_us) best_us = us, best = {big, static_cast<int32_t>(k)};
    }
  }
  return best;
}

// Least table (elements) that few fp32 rows read as it is: packing a smaller one
// costs less than splitting it in every block (loss and gradients of 128 rows x 64
// against 1000 columns: 49 us packed, 58 as it is; 98 x 1024 x 9349: 181 and 189;
// loss of 24 x 1024 x 9019: 52 and 37).
constexpr int64_t kRawElements = 8ll << 20;

struct VocabPlan {
  int64_t ldx = 0, np = 0, piece = 0, packed_piece = 0;
  int32_t splits = 1, splits_e = 1;
  bool big_x = false, big_e = false;  // dX's and dE's tiles
  bool packed = false;  // the table is packed whatever its alignment
  bool raw = false;     // fp32, and the table is read as it is where it is aligned
  size_t off_flag, off_count, off_row, off_inv, off_target, off_g, off_gx, off_lse2, off_q, off_ent, off_zt, off_qu, off_nu, off_bits,
      off_before, off_Xp, off_Xg, off_Ep, off_Xh, off_Eh, off_sx, off_se, off_part, off_D, off_dX, off_dE, total;
};

int64_t whole_pads(int64_t x) { return std::max<int64_t>(kPad, x / kPad * kPad); }

VocabPlan plan_vocab(int64_t N, int64_t d, int64_t V, int32_t k, int32_t dtype, bool distill, bool grad) {
  VocabPlan p;
  const int64_t parts = dtype == DPG_BF16 ? 1 : 3;
  p.ldx = round_up(d, kStepK);
  p.np = round_up(N, kPad);
  p.raw = parts > 1 && N <= SmallTile::kTile && d % 4 == 0 && V * d >= kRawElements;
  p.packed = parts > 1 ? !p.raw : d % 8 != 0;
  // one piece of the vocabulary: its D, its teacher ids' bits, and its packed
  // table
  const int64_t row_bytes = p.ldx * 2 * parts;
  // (at most 2^23 small tiles a launch, whose threads stay under 2^32)
  p.piece = std::min(round_up(V, kPad), whole_pads((int64_t{1} << 37) / p.np));
  if (grad) p.piece = std::min(p.piece, whole_pads(kPieceBytes / (p.np * 2 * parts)));
  if (distill)
    p.piece = std::min({p.piece, whole_pads(kPieceBytes / (N * 10) * 64), int64_t{64 * kMaxWords}});
  if (p.packed) p.piece = std::min(p.piece, whole_pads(kTableBytes / row_bytes));
  p.packed_piece = p.packed ? p.piece : std::min(p.piece, whole_pads(kRarePieceBytes / row_bytes));
  if (grad) {
    const int combos = parts == 1 ? 1 : Combos<3>::n;
    const int64_t piece_rows = std::min(V, p.piece);
    const Split x = choose_split(N, p.ldx, ceil_div(piece_rows, kStepK), combos, true);
    const Split e = choose_split(piece_rows, p.ldx, ceil_div(N, kStepK), combos, false);
    p.big_x = x.big, p.splits = x.splits;
    if (p.raw) {  // memory bound: one block a CU, each with at least two K steps
      const int64_t tiles = ceil_div(d, SmallTile::kTile);
      p.big_x = false;
      p.splits = static_cast<int32_t>(std::max<int64_t>(
          1, std::min(256 / tiles, ceil_div(piece_rows, kStepK) / 2)));
    }
    p.big_e = e.big, p.splits_e = e.splits;
  }
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align_up(bytes);
    return at;
  };
  p.off_flag = take(distill ? N * 4 : 0);
  p.off_count = take(4);
  p.off_row = take(N * 4);
  p.off_inv = take(N * 4);
  p.off_target = take(p.np * 4);
  p.off_g = take(grad ? p.np * 4 : 0);
  p.off_gx = take(grad && parts == 1 ? p.np * 4 : 0);
  p.off_lse2 = take(grad ? p.np * 4 : 0);
  p.off_q = take(distill ? N * k * 4 : 0);
  p.off_ent = take(distill ? N * 4 : 0);
  p.off_zt = take(grad ? 0 : N * k * 4);
  p.off_qu = take(distill ? N * k * 4 : 0);
  p.off_nu = take(distill ? N * 4 : 0);
  p.off_bits = take(distill ? N * (p.piece / 64) * 8 : 0);
  p.off_before = take(distill ? N * (p.piece / 64) * 2 : 0);
  // (the loss of fp32 operands needs only their fp16 parts)
  const bool half = parts > 1, whole = !half || grad || p.raw;
  p.off_Xp = take(whole ? parts * p.np * p.ldx * 2 : 0);
  p.off_Xg = take(grad && parts == 1 ? p.np * p.ldx * 2 : 0);
  p.off_Ep = take(whole ? parts * p.packed_piece * p.ldx * 2 : 0);
  p.off_Xh = take(half ? 2 * p.np * p.ldx * 2 : 0);
  p.off_Eh = take(half ? 2 * p.packed_piece * p.ldx * 2 : 0);
  p.off_sx = take(half ? p.np * 4 : 0);
  p.off_se = take(half ? p.packed_piece * 4 : 0);
  // (an unaligned table has smaller pieces, and perhaps smaller tiles)
  const Tile t = logits_tiles(std::min(p.packed_piece, V), N, false);
  const int64_t tile = t == kBig ? BigTile::kTile : t == kSmall ? SmallTile::kTile : TinyTile::kTile;
  p.off_part = take(grad ? 0 : ceil_div(V, tile) * p.np * 8);
  p.off_D = take(grad ? parts * p.np * p.piece * 2 : 0);
  p.off_dX = take(grad ? p.splits * p.np * p.ldx * 4 : 0);
  p.off_dE = take(p.splits_e > 1 ? p.splits_e * p.piece * p.ldx * 4 : 0);
  p.total = off;
  return p;
}

// rows, table: the gradient needs X's, E's bf16 parts (for dE, for dX).
VocabArgs make_args(const VocabCall& c, VocabPlan& p, char* ws, bool rows, bool table) {
  VocabArgs a{};
  a.X = c.X;
  a.E = c.E;
  a.ids = c.ids;
  a.t = c.t;
  a.N = c.N;
  a.V = static_cast<int32_t>(c.V);
  a.d = static_cast<int32_t>(c.d);
  a.k = c.k;
  a.ldx = static_cast<int32_t>(p.ldx);
  a.np = static_cast<int32_t>(p.np);
  a.zscale = static_cast<float>(c.scale / c.tau);
  a.dscale = static_cast<float>(c.scale * c.tau);
  a.tau = static_cast<float>(c.tau);
  a.flag = reinterpret_cast<int32_t*>(ws + p.off_flag);
  a.count = reinterpret_cast<int32_t*>(ws + p.off_count);
  a.row = reinterpret_cast<int32_t*>(ws + p.off_row);
  a.inv = reinterpret_cast<int32_t*>(ws + p.off_inv);
  a.target = reinterpret_cast<int32_t*>(ws + p.off_target);
  a.g = reinterpret_cast<float*>(ws + p.off_g);
  a.gx = reinterpret_cast<float*>(ws + p.off_gx);
  a.lse2 = reinterpret_cast<float*>(ws + p.off_lse2);
  a.q = reinterpret_cast<float*>(ws + p.off_q);
  a.ent = reinterpret_cast<float*>(ws + p.off_ent);
  a.zt = reinterpret_cast<float*>(ws + p.off_zt);
  a.qu = reinterpret_cast<float*>(ws + p.off_qu);
  a.nu = reinterpret_cast<int32_t*>(ws + p.off_nu);
  a.bits = reinterpret_cast<uint64_t*>(ws + p.off_bits);
  a.before = reinterpret_cast<uint16_t*>(ws + p.off_before);
  const bool fp32 = c.dtype == DPG_FP32, pack = p.packed || !aligned(c.E, 16);
  p.raw = p.raw && aligned(c.E, 16);
  const bool half = fp32 && !p.raw;
  a.Xp = !half || rows ? reinterpret_cast<bf16*>(ws + p.off_Xp) : nullptr;
  a.Xg = !fp32 && rows ? reinterpret_cast<bf16*>(ws + p.off_Xg) : nullptr;
  a.Ep = pack && (!half || table) ? reinterpret_cast<bf16*>(ws + p.off_Ep) : nullptr;
  if (half) {
    a.Xh = reinterpret_cast<_Float16*>(ws + p.off_Xh);
    a.Eh = reinterpret_cast<_Float16*>(ws + p.off_Eh);
    a.sx = reinterpret_cast<float*>(ws + p.off_sx);
    a.se = reinterpret_cast<float*>(ws + p.off_se);
  }
  a.part = reinterpret_cast<float2*>(ws + p.off_part);
  a.D = reinterpret_cast<bf16*>(ws + p.off_D);
  a.dXacc = reinterpret_cast<float*>(ws + p.off_dX);
  a.ldd = static_cast<int32_t>(pack ? p.packed_piece : p.piece);
  a.splits = p.splits;
  a.splits_e = p.splits_e;
  a.dEacc = reinterpret_cast<float*>(ws + p.off_dE);
  return a;
}

unsigned blocks_of(int64_t n, int64_t per) { return static_cast<unsigned>(ceil_div(n, per)); }
// grid of tile_of_block for mt x nt tiles
dim3 tile_grid(int64_t mt, int64_t nt) { return dim3(static_cast<unsigned>(round_up(mt * nt, 8))); }

// Target weights, then the packed rows; a launch of pack_kernel for rows and
// the first piece of the table together, for the table alone afterwards.
template <typename T>
void launch_pack(const VocabArgs& a, bool rows, hipStream_t s) {
  const unsigned rb = rows ? blocks_of(a.N, kPackRows) + kPadBlocks : 0;
  const unsigned tb = a.Ep || a.Eh ? blocks_of(round_up(a.vn, kPad), 4) : 0;
  if (rb + tb)
    hipLaunchKernelGGL(pack_kernel<T>, dim3(rb + tb), dim3(kThreads), 0, s, a, static_cast<int>(rb));
}

// fn for every piece of the vocabulary, after its rows are packed and its
// teacher ids found.
template <typename T, class F>
void for_pieces(VocabArgs& a, hipStream_t s, F fn) {
  if (a.t) hipLaunchKernelGGL(teacher_kernel, dim3(blocks_of(a.N, 4)), dim3(kThreads), 0, s, a);
  for (int64_t v0 = 0; v0 < a.V; v0 += a.ldd) {
    a.v0 = static_cast<int32_t>(v0);
    a.vn = static_cast<int32_t>(std::min<int64_t>(a.ldd, a.V - v0));
    launch_pack<T>(a, v0 == 0, s);
    if (a.t)
      hipLaunchKernelGGL(teacher_ids_kernel, dim3(static_cast<unsigned>(a.N)), dim3(kThreads), 0, s, a);
    fn();
  }
}

// fn with the parts of the logits kernels' operands, kRaw where the table is read as
// it is (with small tiles).
template <typename T, class G, class F>
void with_raw(bool raw, F fn) {
  if constexpr (kParts<T> == 3 && G::kTile == SmallTile::kTile) {
    if (raw) return fn(std::integral_constant<int, kRaw>{});
  }
  fn(std::integral_constant<int, kParts<T>>{});
}

template <typename T>
int run_loss(VocabArgs a, const VocabPlan& p, hipStream_t s) {
  with_tile(logits_tiles(std::min(a.ldd, a.V), a.N, p.raw), [&](auto g) {
    typedef decltype(g) G;
    for_pieces<T>(a, s, [&] {
      const dim3 grid = tile_grid(ceil_div(a.vn, G::kTile), a.np / G::kTile), b(G::kThreads);
      const int tile0 = a.v0 / G::kTile;
      with_raw<T, G>(p.raw, [&](auto parts) {
        constexpr int P = decltype(parts)::value;
        if (a.t) hipLaunchKernelGGL((stats_kernel<G, P, true>), grid, b, 0, s, a, tile0);
        else hipLaunchKernelGGL((stats_kernel<G, P, false>), grid, b, 0, s, a, tile0);
      });
    });
    hipLaunchKernelGGL(lse_kernel, dim3(blocks_of(a.N, 4)), dim3(kThreads), 0, s, a,
                       static_cast<int>(ceil_div(a.V, G::kTile)));
  });
  return check_launch("vocab loss");
}

// Each row's sums over the splits, rounded.
template <typename T>
void launch_out(const VocabArgs& a, const float* sums, int64_t stride, int splits, const int32_t* inv,
                const float* factor, int64_t rows, T* out, hipStream_t s) {
  int bits = 0;
  while (bits < 8 && 4 << bits < a.d) ++bits;
  hipLaunchKernelGGL(out_kernel<T>, dim3(blocks_of(rows, kThreads >> bits)), dim3(kThreads), 0, s, a,
                     sums, stride, splits, inv, factor, rows, bits, out);
}

template <typename T>
int run_grad(VocabArgs a, const VocabPlan& p, void* dX, void* dE, hipStream_t s) {
  for_pieces<T>(a, s, [&] {
    with_tile(logits_tiles(a.vn, a.N, p.raw), [&](auto g) {
      typedef decltype(g) G;
      const dim3 grid = tile_grid(ceil_div(a.vn, G::kTile), a.np / G::kTile), b(G::kThreads);
      with_raw<T, G>(p.raw, [&](auto parts) {
        constexpr int P = decltype(parts)::value;
        if (a.t) hipLaunchKernelGGL((grad_logits_kernel<G, P, true>), grid, b, 0, s, a);
        else hipLaunchKernelGGL((grad_logits_kernel<G, P, false>), grid, b, 0, s, a);
      });
    });
    T* de = static_cast<T*>(dE);
    auto blocks_x = [&](int64_t tile) {
      return tile_grid(a.np / tile, ceil_div(a.ldx, tile) * a.splits).x;
    };
    auto blocks_e = [&](int64_t tile) {
      return tile_grid(ceil_div(a.vn, tile), ceil_div(a.ldx, tile) * a.splits_e).x;
    };
    if (dX && dE && !p.raw && !p.big_x && !p.big_e) {
      const unsigned nx = blocks_x(SmallTile::kTile), ne = blocks_e(SmallTile::kTile);
      hipLaunchKernelGGL((products_kernel<SmallTile, T, true, true>), dim3(nx + ne),
                         dim3(SmallTile::kThreads), 0, s, a, static_cast<int>(nx), de);
    } else {
      if (dX && p.raw)
        hipLaunchKernelGGL(raw_dx_kernel, dim3(blocks_x(SmallTile::kTile)),
                           dim3(SmallTile::kThreads), 0, s, a);
      else if (dX)
        with_tile(p.big_x ? kBig : kSmall, [&](auto g) {
          typedef decltype(g) G;
          if constexpr (!std::is_same<G, TinyTile>::value)
            hipLaunchKernelGGL((products_kernel<G, T, true, false>), dim3(blocks_x(G::kTile)),
                               dim3(G::kThreads), 0, s, a, 0, de);
        });
      if (dE)
        with_tile(p.big_e ? kBig : kSmall, [&](auto g) {
          typedef decltype(g) G;
          if constexpr (!std::is_same<G, TinyTile>::value)
            hipLaunchKernelGGL((products_kernel<G, T, false, true>), dim3(blocks_e(G::kTile)),
                               dim3(G::kThreads), 0, s, a, 0, de);
        });
    }
    if (dE && a.splits_e > 1)
      launch_out<T>(a, a.dEacc, static_cast<int64_t>(a.ldd) * a.ldx, a.splits_e, nullptr, nullptr, a.vn,
                    de + static_cast<int64_t>(a.v0) * a.d, s);
  });
  if (dX)
    launch_out<T>(a, a.dXacc, static_cast<int64_t>(a.np) * a.ldx, a.splits, a.inv,
                  kParts<T> == 1 ? a.gx : nullptr, a.N, static_cast<T*>(dX), s);
  return check_launch("vocab gradient");
}

int check_ws(const void* ws, size_t have, size_t need) {
  if (!ws) return fail(DPG_ERR_WORKSPACE, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(DPG_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (have < need)
    return fail(DPG_ERR_WORKSPACE, "workspace of " + std::to_string(have) + " bytes, " +
                                       std::to_string(need) + " needed");
  return DPG_OK;
}

int loss_impl(const VocabCall& c, bool distill, float* loss, float* lse, void* workspace,
              size_t workspace_bytes, void* stream) {
  record_error(DPG_OK, "");
  if (const int st = check_call(c, distill)) return st;
  if (!loss || !lse) return fail(DPG_ERR_INVALID_ARG, "loss and lse must not be NULL");
  VocabPlan p = plan_vocab(c.N, c.d, c.V, c.k, c.dtype, distill, false);
  if (const int st = check_ws(workspace, workspace_bytes, p.total)) return st;
  VocabArgs a = make_args(c, p, static_cast<char*>(workspace), false, false);
  a.loss = loss;
  a.lse = lse;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return c.dtype == DPG_BF16 ? run_loss<bf16>(a, p, s) : run_loss<float>(a, p, s);
}

int grad_impl(const VocabCall& c, bool distill, const float* lse, const float* dloss, void* dX,
              void* dE, void* workspace, size_t workspace_bytes, void* stream) {
  record_error(DPG_OK, "");
  if (const int st = check_call(c, distill)) return st;
  if (!lse || !dloss) return fail(DPG_ERR_INVALID_ARG, "lse and dloss must not be NULL");
  if (!dX && !dE) return fail(DPG_ERR_INVALID_ARG, "dX and dE are both NULL");
  VocabPlan p = plan_vocab(c.N, c.d, c.V, c.k, c.dtype, distill, true);
  if (const int st = check_ws(workspace, workspace_bytes, p.total)) return st;
  VocabArgs a = make_args(c, p, static_cast<char*>(workspace), dE != nullptr, dX != nullptr);
  a.lse = const_cast<float*>(lse);
  a.dloss = dloss;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return c.dtype == DPG_BF16 ? run_grad<bf16>(a, p, dX, dE, s) : run_grad<float>(a, p, dX, dE, s);
}

int size_impl(int64_t N, int64_t d, int64_t V, int32_t k, int32_t dtype, int32_t grad, bool distill,
              size_t* bytes) {
  record_error(DPG_OK, "");
  if (!bytes) return fail(DPG_ERR_INVALID_ARG, "bytes is NULL");
  VocabCall c{};
  c.N = N, c.d = d, c.V = V, c.k = k, c.dtype = dtype;
  if (const int st = check_call_shape(c)) return st;
  *bytes = plan_vocab(N, d, V, k, dtype, distill, grad != 0).total;
  return DPG_OK;
}

}  // namespace
}  // namespace dpg

using namespace dpg;

extern "C" {

int dpg_vocab_loss_workspace_size(int64_t N, int64_t d, int64_t V, int32_t dtype, int32_t grad,
                                  size_t* bytes) {
  return size_impl(N, d, V, 1, dtype, grad, false, bytes);
}

int dpg_vocab_loss(const void* X, const void* E, const int64_t* targets, int64_t N, int64_t d,
                   int64_t V, int32_t dtype, double scale, float* loss, float* lse,
                   void* workspace, size_t workspace_bytes, void* stream) {
  return loss_impl({X, E, targets, nullptr, N, d, V, 1, dtype, scale, 1.0}, false, loss, lse,
                   workspace, workspace_bytes, stream);
}

int dpg_vocab_loss_grad(const void* X, const void* E, const int64_t* targets, const float* lse,
                        const float* dloss, int64_t N, int64_t d, int64_t V, int32_t dtype,
                        double scale, void* dX, void* dE, void* workspace, size_t workspace_bytes,
                        void* stream) {
  return grad_impl({X, E, targets, nullptr, N, d, V, 1, dtype, scale, 1.0}, false, lse, dloss, dX,
                   dE, workspace, workspace_bytes, stream);
}

int dpg_distill_loss_workspace_size(int64_t N, int64_t d, int64_t V, int32_t k, int32_t dtype,
                                    int32_t grad, size_t* bytes) {
  return size_impl(N, d, V, k, dtype, grad, true, bytes);
}

int dpg_distill_loss(const void* X, const void* E, const int64_t* top_ids, const float* top_logits,
                     int64_t N, int64_t d, int64_t V, int32_t k, int32_t dtype, double scale,
                     double temperature, float* loss, float* lse, void* workspace,
                     size_t workspace_bytes, void* stream) {
  return loss_impl({X, E, top_ids, top_logits, N, d, V, k, dtype, scale, temperature}, true, loss,
                   lse, workspace, workspace_bytes, stream);
}

int dpg_distill_loss_grad(const void* X, const void* E, const int64_t* top_ids,
                          const float* top_logits, const float* lse, const float* dloss, int64_t N,
                          int64_t d, int64_t V, int32_t k, int32_t dtype, double scale,
                          double temperature, void* dX, void* dE, void* workspace,
                          size_t workspace_bytes, void* stream) {
  return grad_impl({X, E, top_ids, top_logits, N, d, V, k, dtype, scale, temperature}, true, lse,
                   dloss, dX, dE, workspace, workspace_bytes, stream);
}

}  // extern "C"
