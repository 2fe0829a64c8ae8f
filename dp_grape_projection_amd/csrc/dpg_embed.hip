// Token embedding beside the private update step: the lookup with scaling,
// every sample's squared gradient norm of the table, and the table's gradient
// with per-sample clip factors.
//
//   Y[n]       = c E[id_n]
//   norm_sq[i] += sum_v || c sum_{n in sample i, id_n = v} dY[n] ||^2
//   dE[v]      = c sum_{n: id_n = v} s_{n / T} dY[n]
//
// A position whose id lies outside [0, V) takes no part: its Y row is zero
// and its dY row is not read. The sums run over tokens in sorted order, each
// token's positions ascending, without atomics on values, so results do not
// depend on the order blocks run in. Sums are held in fp32 and rounded once.
#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include "dpg.h"
#include "dpg_device.hpp"
#include "dpg_internal.hpp"

namespace dpg {
namespace {

constexpr int kSortThreads = 1024;
// Tokens a sorting block counts in LDS; more blocks than CUs only for
// vocabularies above 256 times this.
constexpr int kSortBins = 8192;

// Eight values starting at p (VEC: two or one 16-byte accesses; otherwise
// element by element, n of them valid).
template <bool VEC>
__device__ __forceinline__ void load8(const float* p, int n, float (&v)[8]) {
  if constexpr (VEC) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = a[q], v[4 + q] = b[q];
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = q < n ? p[q] : 0.0f;
  }
}
template <bool VEC>
__device__ __forceinline__ void load8(const bf16* p, int n, float (&v)[8]) {
  if constexpr (VEC) {
    const bf16x8 a = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = to_float(a[q]);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = q < n ? to_float(p[q]) : 0.0f;
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(float* p, int n, const float (&v)[8]) {
  if constexpr (VEC) {
    f32x4 a, b;
#pragma unroll
    for (int q = 0; q < 4; ++q) a[q] = v[q], b[q] = v[4 + q];
    *reinterpret_cast<f32x4*>(p) = a;
    *reinterpret_cast<f32x4*>(p + 4) = b;
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) p[q] = v[q];
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(bf16* p, int n, const float (&v)[8]) {
  if constexpr (VEC) {
    bf16x8 a;
#pragma unroll
    for (int q = 0; q < 8; ++q) a[q] = from_float<bf16>(v[q]);
    *reinterpret_cast<bf16x8*>(p) = a;
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) p[q] = from_float<bf16>(v[q]);
  }
}

// ----------------------------------------------------------------- lookup --

// 1 << tpr_log2 threads per row, each taking units of eight columns.
template <typename TE, typename TY, bool VEC>
__global__ __launch_bounds__(kThreads) void embed_kernel(const int64_t* ids, int64_t n,
                                                         const TE* E, int64_t V, int d,
                                                         float scale, int tpr_log2, TY* Y) {
  const int tpr = 1 << tpr_log2;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads >> tpr_log2) +
                      (threadIdx.x >> tpr_log2);
  if (row >= n) return;
  const int64_t id = ids[row];
  const bool ok = id >= 0 && id < V;
  const TE* src = E + (ok ? id : 0) * d;
  TY* dst = Y + row * d;
  for (int u = threadIdx.x & (tpr - 1); u * 8 < d; u += tpr) {
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (ok) {
      load8<VEC>(src + u * 8, d - u * 8, v);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] *= scale;
    }
    store8<VEC>(dst + u * 8, d - u * 8, v);
  }
}

// ------------------------------------------------------------------- sort --

// Stable counting sort of the positions by token, in one launch. Token v
// belongs to block v % G (G a power of two), where it is bin v / G: frequent
// tokens, which often have neighbouring ids, spread over the blocks. Every
// block reads all ids, counts its own tokens in LDS and the tokens of lower
// blocks (its offset in `order`), writes its bins' starts, then reads the ids
// again in order and places its positions. start[g * (bins + 1) + b] is the
// first entry in `order` of bin b of block g, and entry [bins] its end.
//
// Reading all ids in each block costs N * 8 bytes of L2 reads per block, 64
// KiB at N = 8192, and saves the four to six dependent launches of a radix
// sort.
__global__ __launch_bounds__(kSortThreads) void token_sort_kernel(const int64_t* ids, int n,
                                                                  int64_t V, int g_log2, int bins,
                                                                  int* start, int* order) {
  __shared__ int hist[kSortBins];
  __shared__ int list_bin[kSortThreads], list_pos[kSortThreads];
  __shared__ int wave_cnt[kSortThreads / 64 + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = blockIdx.x, mask = (1 << g_log2) - 1;
  for (int b = tid; b < bins; b += kSortThreads) hist[b] = 0;
  __syncthreads();
  int less = 0;
  for (int i = tid; i < n; i += kSortThreads) {
    const int64_t id = ids[i];
    if (id < 0 || id >= V) continue;
    const int o = static_cast<int>(id) & mask;
    if (o < g) ++less;
    else if (o == g) atomicAdd(&hist[static_cast<int>(id) >> g_log2], 1);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) less += __shfl_xor(less, off, 64);
  if (lane == 0) wave_cnt[wave] = less;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < kSortThreads / 64; ++w) base += wave_cnt[w];
  __syncthreads();
  // exclusive scan of the bins, kSortThreads at a time; hist becomes each
  // bin's next free entry
  int* st = start + static_cast<int64_t>(g) * (bins + 1);
  for (int b0 = 0; b0 < bins; b0 += kSortThreads) {
    const int c = b0 + tid < bins ? hist[b0 + tid] : 0;
    int x = c;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int y = __shfl_up(x, off, 64);
      if (lane >= off) x += y;
    }
    if (lane == 63) wave_cnt[wave] = x;
    __syncthreads();
    int before = base, all = 0;
    for (int w = 0; w < kSortThreads / 64; ++w) {
      const int t = wave_cnt[w];
      if (w < wave) before += t;
      all += t;
    }
    if (b0 + tid < bins) {
      st[b0 + tid] = before + x - c;
      hist[b0 + tid] = before + x - c;
    }
    base += all;
    __syncthreads();
  }
  if (tid == 0) st[bins] = base;
  // placement, kSortThreads positions at a time and in order
  for (int i0 = 0; i0 < n; i0 += kSortThreads) {
    const int i = i0 + tid;
    int64_t id = i < n ? ids[i] : -1;
    const bool mine = id >= 0 && id < V && (static_cast<int>(id) & mask) == g;
    const uint64_t b = __ballot(mine);
    if (lane == 0) wave_cnt[wave] = __popcll(b);
    __syncthreads();
    int before = 0, m = 0;
    for (int w = 0; w < kSortThreads / 64; ++w) {
      const int t = wave_cnt[w];
      if (w < wave) before += t;
      m += t;
    }
    if (mine) {
      const int at = before + __popcll(b & ((1ull << lane) - 1));
      list_bin[at] = static_cast<int>(id) >> g_log2;
      list_pos[at] = i;
    }
    __syncthreads();
    if (tid < m) {
      const int bin = list_bin[tid];
      int rank = 0;
      for (int j = 0; j < tid; ++j) rank += list_bin[j] == bin;
      order[hist[bin] + rank] = list_pos[tid];
    }
    __syncthreads();
    if (tid < m) atomicAdd(&hist[list_bin[tid]], 1);
    __syncthreads();
  }
}

// --------------------------------------------------------------- gradient --

// 1 << tpr_log2 threads per vocabulary row: its positions are added in order.
template <typename TY, typename TE, bool VEC>
__global__ __launch_bounds__(kThreads) void embed_grad_kernel(
    const TY* dY, int64_t V, int d, int T, float scale, const float* sample_scales, int g_log2,
    int bins, const int* start, const int* order, int tpr_log2, int accumulate, TE* dE) {
  const int tpr = 1 << tpr_log2;
  const int64_t v = static_cast<int64_t>(blockIdx.x) * (kThreads >> tpr_log2) +
                    (threadIdx.x >> tpr_log2);
  if (v >= V) return;
  const int* st = start + (v & ((1 << g_log2) - 1)) * (bins + 1) + (v >> g_log2);
  const int j0 = st[0], j1 = st[1];
  if (accumulate && j0 == j1) return;
  TE* dst = dE + v * d;
  for (int u = threadIdx.x & (tpr - 1); u * 8 < d; u += tpr) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j = j0; j < j1; ++j) {
      const int pos = order[j];
      const float w = sample_scales ? scale * sample_scales[pos / T] : scale;
      float x[8];
      load8<VEC>(dY + static_cast<int64_t>(pos) * d + u * 8, d - u * 8, x);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] = fmaf(w, x[q], acc[q]);
    }
    if (accumulate) {
      float x[8];
      load8<VEC>(dst + u * 8, d - u * 8, x);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] += x[q];
    }
    store8<VEC>(dst + u * 8, d - u * 8, acc);
  }
}

// ------------------------------------------------------------------ norms --

// One block per entry of `order`: the first entry of a (token, sample) run
// adds the run's rows and writes the squared norm of the sum at its position,
// the others write zero.
template <typename TY, bool VEC>
__global__ __launch_bounds__(kThreads) void embed_run_norm_kernel(const int64_t* ids, const TY* dY,
                                                                  int d, int T, float scale,
                                                                  int g_log2, int bins,
                                                                  const int* start,
                                                                  const int* order, float* run_sq) {
  __shared__ float red[4];
  const int j = blockIdx.x, G = 1 << g_log2;
  const int total = start[static_cast<int64_t>(G) * (bins + 1) - 1];
  if (j >= total) return;
  const int pos = order[j];
  const int64_t id = ids[pos];
  const int sample = pos / T;
  if (j > 0) {
    const int prev = order[j - 1];
    if (ids[prev] == id && prev / T == sample) {
      if (threadIdx.x == 0) run_sq[pos] = 0.0f;
      return;
    }
  }
  const int end = start[(id & (G - 1)) * (bins + 1) + (id >> g_log2) + 1];
  float sq = 0.0f;
  for (int u = threadIdx.x; u * 8 < d; u += kThreads) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int i = j; i < end; ++i) {
      const int p = order[i];
      if (p / T != sample) break;
      float x[8];
      load8<VEC>(dY + static_cast<int64_t>(p) * d + u * 8, d - u * 8, x);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] += x[q];
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) sq = fmaf(scale * acc[q], scale * acc[q], sq);
  }
  sq = wave_sum(sq);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sq;
  __syncthreads();
  if (threadIdx.x == 0) run_sq[pos] = ((red[0] + red[1]) + red[2]) + red[3];
}

// norm_sq[i] += the run norms at sample i's positions, in a fixed order.
__global__ __launch_bounds__(kThreads) void embed_norm_sum_kernel(const int64_t* ids, int64_t V,
                                                                  int T, const float* run_sq,
                                                                  float* norm_sq) {
  __shared__ float red[4];
  const int64_t base = static_cast<int64_t>(blockIdx.x) * T;
  float t = 0.0f;
  for (int k = threadIdx.x; k < T; k += kThreads) {
    const int64_t id = ids[base + k];
    if (id >= 0 && id < V) t += run_sq[base + k];
  }
  t = wave_sum(t);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = t;
  __syncthreads();
  if (threadIdx.x == 0) norm_sq[blockIdx.x] += ((red[0] + red[1]) + red[2]) + red[3];
}

// ------------------------------------------------------------------- host --

int fail(int code, const std::string& msg) { return record_error(code, msg.c_str()); }

int check_launch(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(DPG_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
  return DPG_OK;
}

bool valid_dtype(int32_t t) { return t == DPG_FP32 || t == DPG_BF16; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

// log2 of the threads that share a row of d columns: one per unit of eight
// columns, at most a block.
int row_threads_log2(int64_t d) {
  int l = 0;
  while (l < 8 && (8ll << l) < d) ++l;
  return l;
}

// One block may stand for each token and each vocabulary row, and a launch
// has fewer than 2^32 threads.
constexpr int64_t kMaxTokens = 1ll << 23;

int check_embed_shape(int64_t n, int64_t V, int64_t d) {
  if (n < 1 || n > kMaxTokens)
    return fail(DPG_ERR_INVALID_ARG, "the number of tokens must be in [1, 2^23]");
  if (V < 1 || V > kMaxTokens) return fail(DPG_ERR_INVALID_ARG, "V must be in [1, 2^23]");
  if (d < 1 || d > (1ll << 20)) return fail(DPG_ERR_INVALID_ARG, "d must be in [1, 2^20]");
  return DPG_OK;
}

int check_batch(int64_t B, int64_t T) {
  if (B < 1 || T < 1 || B > kMaxTokens || T > kMaxTokens || B * T > kMaxTokens)
    return fail(DPG_ERR_INVALID_ARG, "B and T must be >= 1 and B*T <= 2^23");
  return DPG_OK;
}

int check_ws(const void* ws, size_t have, size_t need) {
  if (!ws) return fail(DPG_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) % 256 != 0)
    return fail(DPG_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (have < need)
    return fail(DPG_ERR_WORKSPACE, "workspace of " + std::to_string(have) + " bytes, " +
                                       std::to_string(need) + " needed");
  return DPG_OK;
}

struct SortPlan {
  int g_log2 = 0, bins = 0;
  size_t off_order = 0, off_run = 0, total = 0;
};

// 256 sorting blocks (one per CU), fewer for vocabularies under 1024, more
// where a block's share of the tokens would exceed its LDS bins.
SortPlan plan_sort(int64_t n, int64_t V) {
  SortPlan p;
  while (p.g_log2 < 8 && (4ll << p.g_log2) <= V) ++p.g_log2;
  while (((V - 1) >> p.g_log2) + 1 > kSortBins) ++p.g_log2;
  p.bins = static_cast<int>(((V - 1) >> p.g_log2) + 1);
  p.off_order = align_up((static_cast<size_t>(1) << p.g_log2) * (p.bins + 1) * 4);
  p.off_run = p.off_order + align_up(static_cast<size_t>(n) * 4);
  p.total = p.off_run + align_up(static_cast<size_t>(n) * 4);
  return p;
}

int sort_tokens(const SortPlan& p, const int64_t* ids, int64_t n, int64_t V, char* ws,
                hipStream_t s) {
  hipLaunchKernelGGL(token_sort_kernel, dim3(1u << p.g_log2), dim3(kSortThreads), 0, s, ids,
                     static_cast<int>(n), V, p.g_log2, p.bins, reinterpret_cast<int*>(ws),
                     reinterpret_cast<int*>(ws + p.off_order));
  return check_launch("token_sort");
}

template <typename TE, typename TY>
void launch_embed(const int64_t* ids, int64_t n, const void* E, int64_t V, int64_t d, double scale,
                  void* Y, hipStream_t s) {
  const int l = row_threads_log2(d);
  const dim3 g(static_cast<unsigned>(ceil_div(n, kThreads >> l))), b(kThreads);
  const TE* e = static_cast<const TE*>(E);
  TY* y = static_cast<TY*>(Y);
  if (d % 8 == 0 && aligned16(E) && aligned16(Y))
    hipLaunchKernelGGL((embed_kernel<TE, TY, true>), g, b, 0, s, ids, n, e, V,
                       static_cast<int>(d), static_cast<float>(scale), l, y);
  else
    hipLaunchKernelGGL((embed_kernel<TE, TY, false>), g, b, 0, s, ids, n, e, V,
                       static_cast<int>(d), static_cast<float>(scale), l, y);
}

template <typename TY, typename TE>
void launch_embed_grad(const SortPlan& p, const void* dY, int64_t V, int64_t d, int64_t T,
                       double scale, const float* sample_scales, int accumulate, void* dE,
                       const char* ws, hipStream_t s) {
  const int l = row_threads_log2(d);
  const dim3 g(static_cast<unsigned>(ceil_div(V, kThreads >> l))), b(kThreads);
  const int* start = reinterpret_cast<const int*>(ws);
  const int* order = reinterpret_cast<const int*>(ws + p.off_order);
  auto go = [&](auto vec) {
    hipLaunchKernelGGL((embed_grad_kernel<TY, TE, decltype(vec)::value>), g, b, 0, s,
                       static_cast<const TY*>(dY), V, static_cast<int>(d), static_cast<int>(T),
                       static_cast<float>(scale), sample_scales, p.g_log2, p.bins, start, order, l,
                       accumulate, static_cast<TE*>(dE));
  };
  if (d % 8 == 0 && aligned16(dY) && aligned16(dE)) go(std::true_type{});
  else go(std::false_type{});
}

}  // namespace
}  // namespace dpg

using namespace dpg;

extern "C" {

int dpg_embed(const int64_t* ids, int64_t n, const void* E, int64_t V, int64_t d,
              int32_t table_dtype, double scale, int32_t dtype, void* Y, void* stream) {
  record_error(DPG_OK, "");
  if (const int st = check_embed_shape(n, V, d)) return st;
  if (!valid_dtype(table_dtype) || !valid_dtype(dtype))
    return fail(DPG_ERR_INVALID_ARG, "unknown dtype");
  if (table_dtype == DPG_BF16 && dtype == DPG_FP32)
    return fail(DPG_ERR_INVALID_ARG, "a bf16 table is looked up in bf16");
  if (!std::isfinite(scale)) return fail(DPG_ERR_INVALID_ARG, "scale must be finite");
  if (!ids || !E || !Y) return fail(DPG_ERR_INVALID_ARG, "NULL data pointer");
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (table_dtype == DPG_BF16) launch_embed<bf16, bf16>(ids, n, E, V, d, scale, Y, s);
  else if (dtype == DPG_BF16) launch_embed<float, bf16>(ids, n, E, V, d, scale, Y, s);
  else launch_embed<float, float>(ids, n, E, V, d, scale, Y, s);
  return check_launch("embed");
}

int dpg_embed_workspace_size(int64_t B, int64_t T, int64_t V, int64_t d, size_t* bytes) {
  record_error(DPG_OK, "");
  if (!bytes) return fail(DPG_ERR_INVALID_ARG, "bytes is NULL");
  if (const int st = check_batch(B, T)) return st;
  if (const int st = check_embed_shape(B * T, V, d)) return st;
  *bytes = plan_sort(B * T, V).total;
  return DPG_OK;
}

int dpg_embed_norms(const int64_t* ids, const void* dY, int64_t B, int64_t T, int64_t V, int64_t d,
                    int32_t dtype, double scale, float* norm_sq, void* workspace,
                    size_t workspace_bytes, void* stream) {
  record_error(DPG_OK, "");
  if (const int st = check_batch(B, T)) return st;
  if (const int st = check_embed_shape(B * T, V, d)) return st;
  if (!valid_dtype(dtype)) return fail(DPG_ERR_INVALID_ARG, "unknown dtype");
  if (!std::isfinite(scale)) return fail(DPG_ERR_INVALID_ARG, "scale must be finite");
  if (!ids || !dY || !norm_sq) return fail(DPG_ERR_INVALID_ARG, "NULL data pointer");
  const SortPlan p = plan_sort(B * T, V);
  if (const int st = check_ws(workspace, workspace_bytes, p.total)) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  if (const int st = sort_tokens(p, ids, B * T, V, ws, s)) return st;
  const int* start = reinterpret_cast<const int*>(ws);
  const int* order = reinterpret_cast<const int*>(ws + p.off_order);
  float* run_sq = reinterpret_cast<float*>(ws + p.off_run);
  auto go = [&](auto zero, auto vec) {
    typedef decltype(zero) TY;
    hipLaunchKernelGGL((embed_run_norm_kernel<TY, decltype(vec)::value>),
                       dim3(static_cast<unsigned>(B * T)), dim3(kThreads), 0, s, ids,
                       static_cast<const TY*>(dY), static_cast<int>(d), static_cast<int>(T),
                       static_cast<float>(scale), p.g_log2, p.bins, start, order, run_sq);
  };
  const bool vec = d % 8 == 0 && aligned16(dY);
  if (dtype == DPG_BF16) vec ? go(bf16(), std::true_type{}) : go(bf16(), std::false_type{});
  else vec ? go(0.0f, std::true_type{}) : go(0.0f, std::false_type{});
  if (const int st = check_launch("embed_run_norm")) return st;
  hipLaunchKernelGGL(embed_norm_sum_kernel, dim3(static_cast<unsigned>(B)), dim3(kThreads), 0, s,
                     ids, V, static_cast<int>(T), run_sq, norm_sq);
  return check_launch("embed_norm_sum");
}

int dpg_embed_grad(const int64_t* ids, const void* dY, int64_t B, int64_t T, int64_t V, int64_t d,
                   int32_t dtype, double scale, const float* sample_scales, int32_t table_dtype,
                   int32_t accumulate, void* dE, void* workspace, size_t workspace_bytes,
                   void* stream) {
  record_error(DPG_OK, "");
  if (const int st = check_batch(B, T)) return st;
  if (const int st = check_embed_shape(B * T, V, d)) return st;
  if (!valid_dtype(table_dtype) || !valid_dtype(dtype))
    return fail(DPG_ERR_INVALID_ARG, "unknown dtype");
  if (table_dtype == DPG_BF16 && dtype == DPG_FP32)
    return fail(DPG_ERR_INVALID_ARG, "a bf16 table is looked up in bf16");
  if (!std::isfinite(scale)) return fail(DPG_ERR_INVALID_ARG, "scale must be finite");
  if (!ids || !dY || !dE) return fail(DPG_ERR_INVALID_ARG, "NULL data pointer");
  const SortPlan p = plan_sort(B * T, V);
  if (const int st = check_ws(workspace, workspace_bytes, p.total)) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  if (const int st = sort_tokens(p, ids, B * T, V, ws, s)) return st;
  if (table_dtype == DPG_BF16)
    launch_embed_grad<bf16, bf16>(p, dY, V, d, T, scale, sample_scales, accumulate, dE, ws, s);
  else if (dtype == DPG_BF16)
    launch_embed_grad<bf16, float>(p, dY, V, d, T, scale, sample_scales, accumulate, dE, ws, s);
  else
    launch_embed_grad<float, float>(p, dY, V, d, T, scale, sample_scales, accumulate, dE, ws, s);
  return check_launch("embed_grad");
}

}  // extern "C"
