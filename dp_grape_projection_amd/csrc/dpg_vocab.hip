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

constexpr int kRowThreads = 1024;
constexpr int kRun = 256;  // terms of one run of an fp32 product's sum

template <typename T> struct VocabStep { static constexpr int v = sizeof(T) == 2 ? kStepBf16 : kStepF32; };
template <typename T> using VocabTile = Tile<T, kTileM, kTileN, VocabStep<T>::v, 4, 1>;

// Per-call tables in the workspace. Row i of the packed arrays is the i-th
// row that has a target.
struct VocabArgs {
  const void* X;        // [N][d]
  const void* E;        // [V][d]
  const int64_t* ids;   // [N][k] targets
  const float* t;       // [N][k] teacher logits, or null (cross entropy)
  const float* dloss;   // [N]
  int64_t N;
  int32_t V, d, k, ldx; // ldx: row stride of Xp
  float zscale;         // c / tau
  float dscale;         // c tau
  float tau;
  float* loss;          // [N]
  float* lse;           // [N]: written by the loss, read by the gradient
  // workspace
  int32_t* flag;        // [N] row has a target
  int32_t* count;       // [1] packed rows
  int32_t* row;         // [N] packed -> row
  int32_t* inv;         // [N] row -> packed, -1
  float* q;             // [N][k] target weights (distillation)
  float* ent;           // [N] sum q ln q (distillation)
  float* zt;            // [N][k] packed: target logits
  void* Xp;             // [N][ldx] packed rows of X
  float2* part;         // [col tiles][N] packed: tile maximum and sum
  void* D;              // [N][ldd] packed: one piece of D
  float* dXacc;         // [N][d] packed
  int32_t ldd;
  int32_t v0, vn;       // the piece: columns v0 .. v0 + vn - 1
};

// ------------------------------------------------------------------- rows --

// Cross entropy: a row has a target when its id lies in [0, V).
__global__ __launch_bounds__(kThreads) void ce_flag_kernel(const VocabArgs a) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (n < a.N) a.flag[n] = a.ids[n] >= 0 && a.ids[n] < a.V;
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
  for (int j = lane; j < a.k; j += 64) {
    float w = 0.0f;
    if (on && id[j] >= 0 && id[j] < a.V) {
      const float x = (t[j] - m) * inv_tau;
      w = expf(x);
      if (w != 0.0f) e = fmaf(w, x, e);
    }
    q[j] = w;
    s += w;
  }
  s = wave_sum(s);
  e = wave_sum(e);
  for (int j = lane; j < a.k; j += 64) q[j] = on ? q[j] / s : 0.0f;
  if (lane == 0) {
    a.flag[n] = on;
    a.ent[n] = on ? e / s - logf(s) : 0.0f;  // sum q ln q, ln q = x - ln s
  }
}

// Packed index of every row, in order; one block.
__global__ __launch_bounds__(kRowThreads) void rows_kernel(const VocabArgs a) {
  __shared__ int wave_cnt[kRowThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int base = 0;
  for (int64_t n0 = 0; n0 < a.N; n0 += kRowThreads) {
    const int64_t n = n0 + tid;
    const bool on = n < a.N && a.flag[n];
    const uint64_t b = __ballot(on);
    if (lane == 0) wave_cnt[wave] = __popcll(b);
    __syncthreads();
    int before = base, all = 0;
    for (int w = 0; w < kRowThreads / 64; ++w) {
      const int c = wave_cnt[w];
      if (w < wave) before += c;
      all += c;
    }
    const int at = before + __popcll(b & ((1ull << lane) - 1));
    if (on) a.row[at] = static_cast<int32_t>(n);
    if (n < a.N) a.inv[n] = on ? at : -1;
    base += all;
    __syncthreads();
  }
  if (tid == 0) a.count[0] = base;
}

// Xp[i] = X[row[i]], zero beyond d; one block per packed row.
template <typename T>
__global__ __launch_bounds__(kThreads) void pack_kernel(const VocabArgs a) {
  const int i = blockIdx.x;
  if (i >= a.count[0]) return;
  const T* src = static_cast<const T*>(a.X) + static_cast<int64_t>(a.row[i]) * a.d;
  T* dst = static_cast<T*>(a.Xp) + static_cast<int64_t>(i) * a.ldx;
  for (int c = threadIdx.x; c < a.ldx; c += kThreads) dst[c] = c < a.d ? src[c] : zero_val<T>();
}

// All of a tile's steps. fp32: the products of every kRun columns are added
// by themselves first, so that a long sum rounds like a short one (at d =
// 4096 one chain leaves D off by 1.3e-5 of its value, runs of 256 by 4e-6).
template <typename T, class Tl, class LA, class LB, class LoadStep>
__device__ __forceinline__ void run_tile(LA& la, LB& lb, T* smem, Acc<Tl::MB, Tl::NB>& acc, int K,
                                         int tid, LoadStep load_step) {
  const int n_steps = (K + Tl::BK - 1) / Tl::BK;
  acc.zero();
  if constexpr (sizeof(T) == 4) {
    Acc<Tl::MB, Tl::NB> part;
    part.zero();
    run_steps<T, Tl>(la, lb, smem, part, n_steps, tid, load_step, [&](int s) {
      if ((s + 1) % (kRun / Tl::BK) == 0 || s + 1 == n_steps) {
        acc.add(part);
        part.zero();
      }
    });
  } else {
    run_steps<T, Tl>(la, lb, smem, acc, n_steps, tid, load_step, [](int) {});
  }
}

// ----------------------------------------------------------------- logits --

// One 128 x 128 tile of z (rows of Xp, columns of the vocabulary piece), on
// the matrix cores. GRAD = false: the tile's maximum and sum of exponentials
// of each row, and cross entropy's target logit. GRAD = true: the tile of D.
template <typename T, bool VEC, bool GRAD>
__global__ __launch_bounds__(kThreads, 2) void logits_kernel(const VocabArgs a) {
  typedef VocabTile<T> Tl;
  __shared__ __attribute__((aligned(16))) T smem[Tl::kLdsElems];
  const int rows = a.count[0];
  const int m0 = blockIdx.y * Tl::BM, c0 = blockIdx.x * Tl::BN;
  if (m0 >= rows) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  RowsLoader<T, Tl::BM, Tl::BK, true, IdentityRows> la;
  la.ld = a.ldx;
  la.nrows = rows - m0;
  la.K = a.ldx;
  RowsLoader<T, Tl::BN, Tl::BK, VEC, BOperandRows<Tl>> lb;
  lb.ld = a.d;
  lb.nrows = a.vn - c0;
  lb.K = a.d;
  const T* pa = static_cast<const T*>(a.Xp) + static_cast<int64_t>(m0) * a.ldx;
  const T* pb = static_cast<const T*>(a.E) + (static_cast<int64_t>(a.v0) + c0) * a.d;
  Acc<Tl::MB, Tl::NB> acc;
  run_tile<T, Tl>(la, lb, smem, acc, a.d, tid, [&](int s) {
    la.load(pa, s * Tl::BK, tid, false);
    lb.load(pb, s * Tl::BK, tid, false);
  });
  const int wm = Tl::wave_m(wave), wn = Tl::wave_n(wave);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = m0 + Tl::acc_row(wm, 0, i, lane);
    const bool in = r < rows;
    const int n = in ? a.row[r] : 0;
    const int64_t target = in && !a.t ? a.ids[n] : -1;
    if constexpr (!GRAD) {
      float m = -INFINITY;
#pragma unroll
      for (int nb = 0; nb < Tl::NB; ++nb) {
        const int c = c0 + Tl::acc_col(wn, nb, lane);
        const float z = acc.v[0][nb][i] * a.zscale;
        if (c < a.vn) m = fmaxf(m, z);
        if (c < a.vn && in && target == a.v0 + c) a.zt[r] = z;
      }
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
      float s = 0.0f;
#pragma unroll
      for (int nb = 0; nb < Tl::NB; ++nb) {
        const int c = c0 + Tl::acc_col(wn, nb, lane);
        const float z = acc.v[0][nb][i] * a.zscale;
        if (c < a.vn) s += expf(z - m);
      }
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
      if (in && (lane & 31) == 0)
        a.part[static_cast<int64_t>(blockIdx.x) * a.N + r] = make_float2(m, s);
    } else if (in) {
      const float g = a.dloss[n] * a.dscale, lse = a.lse[n];
      T* dst = static_cast<T*>(a.D) + static_cast<int64_t>(r) * a.ldd;
#pragma unroll
      for (int nb = 0; nb < Tl::NB; ++nb) {
        const int c = c0 + Tl::acc_col(wn, nb, lane);
        const float z = acc.v[0][nb][i] * a.zscale;
        float p = expf(z - lse);
        if (target == a.v0 + c) p -= 1.0f;
        if (c < a.ldd) dst[c] = c < a.vn ? from_float<T>(g * p) : zero_val<T>();
      }
    }
  }
}

// Distillation: logits of the teacher's entries, one wave per packed row.
template <typename T>
__global__ __launch_bounds__(kThreads) void target_logits_kernel(const VocabArgs a) {
  const int i = blockIdx.x;
  if (i >= a.count[0]) return;
  const int lane = threadIdx.x & 63;
  const int64_t n = a.row[i];
  const T* x = static_cast<const T*>(a.Xp) + static_cast<int64_t>(i) * a.ldx;
  for (int j = threadIdx.x >> 6; j < a.k; j += 4) {
    const int64_t id = a.ids[n * a.k + j];
    if (id < 0 || id >= a.V) continue;
    const T* e = static_cast<const T*>(a.E) + id * a.d;
    float z = 0.0f;
    for (int c = lane; c < a.d; c += 64) z = fmaf(to_float(x[c]), to_float(e[c]), z);
    z = wave_sum(z);
    if (lane == 0) a.zt[static_cast<int64_t>(i) * a.k + j] = z * a.zscale;
  }
}

// lse and loss of every row from its tile partials: one wave per row.
__global__ __launch_bounds__(kThreads) void lse_kernel(const VocabArgs a, int tiles) {
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (n >= a.N) return;
  const int lane = threadIdx.x & 63;
  const int i = a.inv[n];
  if (i < 0) {
    if (lane == 0) a.loss[n] = 0.0f, a.lse[n] = 0.0f;
    return;
  }
  float m = -INFINITY;
  for (int t = lane; t < tiles; t += 64) m = fmaxf(m, a.part[static_cast<int64_t>(t) * a.N + i].x);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  float s = 0.0f;
  for (int t = lane; t < tiles; t += 64) {
    const float2 p = a.part[static_cast<int64_t>(t) * a.N + i];
    s = fmaf(p.y, expf(p.x - m), s);
  }
  s = wave_sum(s);
  const float lse = m + logf(s);
  float qz = 0.0f;
  if (a.t) {
    for (int j = lane; j < a.k; j += 64) {
      const float q = a.q[n * a.k + j];
      const int64_t id = a.ids[n * a.k + j];
      if (id >= 0 && id < a.V && q != 0.0f) qz = fmaf(q, a.zt[static_cast<int64_t>(i) * a.k + j] - lse, qz);
    }
    qz = wave_sum(qz);
  }
  if (lane == 0) {
    a.lse[n] = lse;
    a.loss[n] = a.t ? a.tau * a.tau * (a.ent[n] - qz) : lse - a.zt[i];
  }
}

// Distillation: the entries of D in the teacher's columns, from their logits
// in fp32: g (p - sum of q over the row's entries with this id). Entries that
// name the same id write the same value.
template <typename T>
__global__ __launch_bounds__(kThreads) void teacher_entries_kernel(const VocabArgs a) {
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t i = at / a.k;
  if (i >= a.count[0]) return;
  const int64_t n = a.row[i];
  const int64_t* ids = a.ids + n * a.k;
  const int64_t id = ids[at - i * a.k];
  if (id < a.v0 || id >= a.v0 + a.vn) return;
  float q = 0.0f;
  for (int j = 0; j < a.k; ++j)
    if (ids[j] == id) q += a.q[n * a.k + j];
  const float p = expf(a.zt[at] - a.lse[n]);
  static_cast<T*>(a.D)[i * a.ldd + (id - a.v0)] = from_float<T>(a.dloss[n] * a.dscale * (p - q));
}

// --------------------------------------------------------------- products --

// dXacc (+)= D E over one piece: 128 x 128 tiles over (packed rows, d).
template <typename T, bool PAIR>
__global__ __launch_bounds__(kThreads, 2) void dx_kernel(const VocabArgs a) {
  typedef VocabTile<T> Tl;
  __shared__ __attribute__((aligned(16))) T smem[Tl::kLdsElems];
  const int rows = a.count[0];
  const int m0 = blockIdx.y * Tl::BM, c0 = blockIdx.x * Tl::BN;
  if (m0 >= rows) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  RowsLoader<T, Tl::BM, Tl::BK, true, IdentityRows> la;
  la.ld = a.ldd;
  la.nrows = rows - m0;
  la.K = a.vn;
  ColsLoader<T, Tl::BN, Tl::BK, PAIR, BOperandRows<Tl>> lb;
  lb.ld = a.d;
  lb.ncols = a.d - c0;
  lb.K = a.vn;
  const T* pa = static_cast<const T*>(a.D) + static_cast<int64_t>(m0) * a.ldd;
  const T* pb = static_cast<const T*>(a.E) + static_cast<int64_t>(a.v0) * a.d + c0;
  Acc<Tl::MB, Tl::NB> acc;
  run_tile<T, Tl>(la, lb, smem, acc, a.vn, tid, [&](int s) {
    la.load(pa, s * Tl::BK, tid, false);
    lb.load(pb, s * Tl::BK, tid, false);
  });
  const int wm = Tl::wave_m(wave), wn = Tl::wave_n(wave);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = m0 + Tl::acc_row(wm, 0, i, lane);
    if (r >= rows) continue;
    float* dst = a.dXacc + static_cast<int64_t>(r) * a.d;
#pragma unroll
    for (int nb = 0; nb < Tl::NB; ++nb) {
      const int c = c0 + Tl::acc_col(wn, nb, lane);
      if (c < a.d) dst[c] = a.v0 == 0 ? acc.v[0][nb][i] : dst[c] + acc.v[0][nb][i];
    }
  }
}

// dX[n] = the row's accumulated gradient rounded once; zero without target.
template <typename T>
__global__ __launch_bounds__(kThreads) void dx_out_kernel(const VocabArgs a, T* dX) {
  const int64_t n = blockIdx.x;
  const int i = a.inv[n];
  for (int c = threadIdx.x; c < a.d; c += kThreads)
    dX[n * a.d + c] = i < 0 ? zero_val<T>() : from_float<T>(a.dXacc[static_cast<int64_t>(i) * a.d + c]);
}

// dE rows of one piece = D^T Xp: 128 x 128 tiles over (piece, d).
template <typename T>
__global__ __launch_bounds__(kThreads, 2) void de_kernel(const VocabArgs a, T* dE) {
  typedef VocabTile<T> Tl;
  __shared__ __attribute__((aligned(16))) T smem[Tl::kLdsElems];
  const int rows = a.count[0];
  const int m0 = blockIdx.y * Tl::BM, c0 = blockIdx.x * Tl::BN;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  ColsLoader<T, Tl::BM, Tl::BK, true, IdentityRows> la;
  la.ld = a.ldd;
  la.ncols = a.vn - m0;
  la.K = rows;
  ColsLoader<T, Tl::BN, Tl::BK, true, BOperandRows<Tl>> lb;
  lb.ld = a.ldx;
  lb.ncols = a.ldx - c0;
  lb.K = rows;
  const T* pa = static_cast<const T*>(a.D) + m0;
  const T* pb = static_cast<const T*>(a.Xp) + c0;
  Acc<Tl::MB, Tl::NB> acc;
  run_tile<T, Tl>(la, lb, smem, acc, rows, tid, [&](int s) {
    la.load(pa, s * Tl::BK, tid, false);
    lb.load(pb, s * Tl::BK, tid, false);
  });
  const int wm = Tl::wave_m(wave), wn = Tl::wave_n(wave);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = m0 + Tl::acc_row(wm, 0, i, lane);
    if (r >= a.vn) continue;
    T* dst = dE + (static_cast<int64_t>(a.v0) + r) * a.d;
#pragma unroll
    for (int nb = 0; nb < Tl::NB; ++nb) {
      const int c = c0 + Tl::acc_col(wn, nb, lane);
      if (c < a.d) dst[c] = from_float<T>(acc.v[0][nb][i]);
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
  if (c.k < 1 || c.k > 1024) return fail(DPG_ERR_INVALID_ARG, "k must be in [1, 1024]");
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

// Bytes of D kept at a time.
constexpr int64_t kPieceBytes = 512ll << 20;

struct VocabPlan {
  int64_t ldx = 0, piece = 0;
  size_t off_flag, off_count, off_row, off_inv, off_q, off_ent, off_zt, off_Xp, off_part, off_D,
      off_dX, total;
};

VocabPlan plan_vocab(int64_t N, int64_t d, int64_t V, int32_t k, int32_t dtype, bool distill, bool grad) {
  VocabPlan p;
  const int64_t es = dtype == DPG_BF16 ? 2 : 4;
  p.ldx = round_up(d, 64);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align_up(bytes);
    return at;
  };
  p.off_flag = take(N * 4);
  p.off_count = take(4);
  p.off_row = take(N * 4);
  p.off_inv = take(N * 4);
  p.off_q = take(distill ? N * k * 4 : 0);
  p.off_ent = take(distill ? N * 4 : 0);
  p.off_zt = take(N * k * 4);
  p.off_Xp = take(N * p.ldx * es);
  p.off_part = take(grad ? 0 : ceil_div(V, kTileN) * N * 8);
  p.piece = std::min(round_up(V, 256), std::max<int64_t>(256, kPieceBytes / (N * es) / 256 * 256));
  p.off_D = take(grad ? N * p.piece * es : 0);
  p.off_dX = take(grad ? N * d * 4 : 0);
  p.total = off;
  return p;
}

VocabArgs make_args(const VocabCall& c, const VocabPlan& p, char* ws) {
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
  a.zscale = static_cast<float>(c.scale / c.tau);
  a.dscale = static_cast<float>(c.scale * c.tau);
  a.tau = static_cast<float>(c.tau);
  a.flag = reinterpret_cast<int32_t*>(ws + p.off_flag);
  a.count = reinterpret_cast<int32_t*>(ws + p.off_count);
  a.row = reinterpret_cast<int32_t*>(ws + p.off_row);
  a.inv = reinterpret_cast<int32_t*>(ws + p.off_inv);
  a.q = reinterpret_cast<float*>(ws + p.off_q);
  a.ent = reinterpret_cast<float*>(ws + p.off_ent);
  a.zt = reinterpret_cast<float*>(ws + p.off_zt);
  a.Xp = ws + p.off_Xp;
  a.part = reinterpret_cast<float2*>(ws + p.off_part);
  a.D = ws + p.off_D;
  a.dXacc = reinterpret_cast<float*>(ws + p.off_dX);
  a.ldd = static_cast<int32_t>(p.piece);
  a.v0 = 0;
  a.vn = a.V;
  return a;
}

unsigned blocks_of(int64_t n, int64_t per) { return static_cast<unsigned>(ceil_div(n, per)); }

// Target weights, the packed rows and their X; with distillation also the
// logits of the teacher's entries.
template <typename T>
int prepare_rows(const VocabArgs& a, hipStream_t s) {
  const dim3 b(kThreads);
  if (a.t) hipLaunchKernelGGL(teacher_kernel, dim3(blocks_of(a.N, 4)), b, 0, s, a);
  else hipLaunchKernelGGL(ce_flag_kernel, dim3(blocks_of(a.N, kThreads)), b, 0, s, a);
  hipLaunchKernelGGL(rows_kernel, dim3(1), dim3(kRowThreads), 0, s, a);
  hipLaunchKernelGGL(pack_kernel<T>, dim3(static_cast<unsigned>(a.N)), b, 0, s, a);
  if (a.t) hipLaunchKernelGGL(target_logits_kernel<T>, dim3(static_cast<unsigned>(a.N)), b, 0, s, a);
  return check_launch("vocab rows");
}

template <typename T, bool GRAD>
void launch_logits(const VocabArgs& a, hipStream_t s) {
  const dim3 g(blocks_of(GRAD ? a.ldd : a.vn, kTileN), blocks_of(a.N, kTileM)), b(kThreads);
  const bool vec = a.d % (16 / sizeof(T)) == 0 && aligned(a.E, 16);
  if (vec) hipLaunchKernelGGL((logits_kernel<T, true, GRAD>), g, b, 0, s, a);
  else hipLaunchKernelGGL((logits_kernel<T, false, GRAD>), g, b, 0, s, a);
}

template <typename T>
int run_loss(const VocabArgs& a, hipStream_t s) {
  if (const int st = prepare_rows<T>(a, s)) return st;
  launch_logits<T, false>(a, s);
  hipLaunchKernelGGL(lse_kernel, dim3(blocks_of(a.N, 4)), dim3(kThreads), 0, s, a,
                     static_cast<int>(blocks_of(a.vn, kTileN)));
  return check_launch("vocab loss");
}

template <typename T>
int run_grad(VocabArgs a, void* dX, void* dE, hipStream_t s) {
  if (const int st = prepare_rows<T>(a, s)) return st;
  const dim3 b(kThreads);
  const unsigned dt = blocks_of(a.d, kTileN);
  for (int64_t v0 = 0; v0 < a.V; v0 += a.ldd) {
    a.v0 = static_cast<int32_t>(v0);
    a.vn = static_cast<int32_t>(std::min<int64_t>(a.ldd, a.V - v0));
    launch_logits<T, true>(a, s);
    if (a.t)
      hipLaunchKernelGGL(teacher_entries_kernel<T>, dim3(blocks_of(a.N * a.k, kThreads)), b, 0, s, a);
    if (dX) {
      const dim3 g(dt, blocks_of(a.N, kTileM));
      if (a.d % 2 == 0 && aligned(a.E, 4)) hipLaunchKernelGGL((dx_kernel<T, true>), g, b, 0, s, a);
      else hipLaunchKernelGGL((dx_kernel<T, false>), g, b, 0, s, a);
    }
    if (dE)
      hipLaunchKernelGGL(de_kernel<T>, dim3(dt, blocks_of(a.vn, kTileM)), b, 0, s, a, static_cast<T*>(dE));
  }
  if (dX)
    hipLaunchKernelGGL(dx_out_kernel<T>, dim3(static_cast<unsigned>(a.N)), b, 0, s, a, static_cast<T*>(dX));
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
  const VocabPlan p = plan_vocab(c.N, c.d, c.V, c.k, c.dtype, distill, false);
  if (const int st = check_ws(workspace, workspace_bytes, p.total)) return st;
  VocabArgs a = make_args(c, p, static_cast<char*>(workspace));
  a.loss = loss;
  a.lse = lse;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return c.dtype == DPG_BF16 ? run_loss<bf16>(a, s) : run_loss<float>(a, s);
}

int grad_impl(const VocabCall& c, bool distill, const float* lse, const float* dloss, void* dX,
              void* dE, void* workspace, size_t workspace_bytes, void* stream) {
  record_error(DPG_OK, "");
  if (const int st = check_call(c, distill)) return st;
  if (!lse || !dloss) return fail(DPG_ERR_INVALID_ARG, "lse and dloss must not be NULL");
  if (!dX && !dE) return fail(DPG_ERR_INVALID_ARG, "dX and dE are both NULL");
  const VocabPlan p = plan_vocab(c.N, c.d, c.V, c.k, c.dtype, distill, true);
  if (const int st = check_ws(workspace, workspace_bytes, p.total)) return st;
  VocabArgs a = make_args(c, p, static_cast<char*>(workspace));
  a.lse = const_cast<float*>(lse);
  a.dloss = dloss;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return c.dtype == DPG_BF16 ? run_grad<bf16>(a, dX, dE, s) : run_grad<float>(a, dX, dE, s);
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
