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
constexpr int kSortItems = 8;                            // ids a thread holds at a time
constexpr int kSortBatch = kSortThreads * kSortItems;
// Tokens a sorting block counts in LDS; more blocks than CUs only for
// vocabularies above 256 times this.
constexpr int kSortBins = 8192;

// A thread takes eight columns of a row at a time, in two halves of four, in
// vectors at any element's address (the global loads and stores take them). WIDE:
// the halves lie side by side. SPLIT: they lie tpr * 4 columns apart, so that the
// threads of a row write neighbouring 16-byte vectors of floats (the gradient of
// a 50304 x 2048 fp32 table: 80 us side by side, 70 us apart). Where a half would
// reach past the row's end, it takes the last columns of the row, of which the
// first `skip` are another thread's too: both compute the same values for them.
// NARROW: a row has fewer than eight columns; one thread takes it element by
// element.
enum Kind { WIDE, SPLIT, NARROW };
template <Kind K>
struct Cols {
  int at[2], skip[2], n;
  // column c of a row of d; past the end, all columns are skipped, and loads stay
  // inside
  __device__ __forceinline__ Cols(int c, int apart, int d) : n(K == NARROW ? d : 8) {
    if (K == SPLIT) {
      at[0] = min(c, d - 4), at[1] = min(c + apart, d - 4);
      skip[0] = min(c - at[0], 4), skip[1] = min(c + apart - at[1], 4);
    } else if (K == WIDE) {
      at[0] = min(c, d - 8), at[1] = at[0] + 4;
      skip[0] = min(c - at[0], 4), skip[1] = max(min(c - at[0] - 4, 4), 0);
    } else {
      at[0] = 0, at[1] = 4, skip[0] = skip[1] = c;
    }
  }
  __device__ __forceinline__ bool mine(int q) const { return (q & 3) >= skip[q >> 2] && q < n; }
  // whether every column is to be written as part of a vector
  __device__ __forceinline__ bool vector(bool own) const {
    return K != NARROW && !(own && (skip[0] || skip[1]));
  }
  // thread t's first column in a group of tpr * 8
  __device__ __forceinline__ static int first(int t) { return t * (K == SPLIT ? 4 : 8); }
};
typedef f32x4 any_f32x4 __attribute__((aligned(4)));
typedef u32x4 any_u32x4 __attribute__((aligned(2)));
typedef uint32_t two_words __attribute__((ext_vector_type(2)));
typedef two_words any_two_words __attribute__((aligned(2)));

// Eight columns as loaded; expanded where they are used, so that loads do not wait
// for one another.
template <typename T> struct Raw8;
template <> struct Raw8<float> {
  f32x4 v[2];
  template <Kind K>
  __device__ __forceinline__ void load(const float* p, const Cols<K>& k) {
    if constexpr (K == NARROW) {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q >> 2][q & 3] = q < k.n ? p[q] : 0.0f;
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) v[h] = *reinterpret_cast<const any_f32x4*>(p + k.at[h]);
    }
  }
  __device__ __forceinline__ float operator[](int q) const { return v[q >> 2][q & 3]; }
};
template <> struct Raw8<bf16> {
  u32x4 a;
  template <Kind K>
  __device__ __forceinline__ void load(const bf16* p, const Cols<K>& k) {
    if constexpr (K == NARROW) {
      bf16x8 v;
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = q < k.n ? p[q] : zero_val<bf16>();
      a = __builtin_bit_cast(u32x4, v);
    } else if constexpr (K == SPLIT) {
      const two_words x = *reinterpret_cast<const any_two_words*>(p + k.at[0]);
      const two_words y = *reinterpret_cast<const any_two_words*>(p + k.at[1]);
      a = u32x4{x[0], x[1], y[0], y[1]};
    } else {
      a = *reinterpret_cast<const any_u32x4*>(p + k.at[0]);
    }
  }
  __device__ __forceinline__ float operator[](int q) const {
    const uint32_t w = a[q >> 1];
    return __builtin_bit_cast(float, q & 1 ? w & 0xFFFF0000u : w << 16);
  }
};
// own: only the columns that are no other thread's.
template <Kind K>
__device__ __forceinline__ void store8(float* p, const Cols<K>& k, const float (&v)[8], bool own) {
  if (k.vector(own)) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<any_f32x4*>(p + k.at[h]) =
          f32x4{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (k.mine(q)) p[k.at[q >> 2] + (q & 3)] = v[q];
  }
}
template <Kind K>
__device__ __forceinline__ void store8(bf16* p, const Cols<K>& k, const float (&v)[8], bool own) {
  static_assert(K != SPLIT, "eight bf16 columns are one vector");
  bf16x8 a;
#pragma unroll
  for (int q = 0; q < 8; ++q) a[q] = from_float<bf16>(v[q]);
  if (k.vector(own)) {
    *reinterpret_cast<any_u32x4*>(p + k.at[0]) = __builtin_bit_cast(u32x4, a);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (k.mine(q)) p[k.at[q >> 2] + (q & 3)] = a[q];
  }
}

// ----------------------------------------------------------------- lookup --

// 1 << tpr_log2 threads per row. Bound by memory (8192 rows of 2048, fp32 to bf16: 17
// us, 5.9 TB/s with every row from HBM) and, for few rows, by the launch.
template <typename TE, typename TY, Kind K>
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
  for (int c = Cols<K>::first(threadIdx.x & (tpr - 1)); c < d; c += tpr * 8) {
    const Cols<K> k(c, 0, d);
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (ok) {
      Raw8<TE> x;
      x.load(src, k);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = scale * x[q];
    }
    store8(dst, k, v, false);
  }
}

// ------------------------------------------------------------------- sort --

// Stable counting sort of the positions by token, in one launch. Token v
// belongs to block v % G (G a power of two), where it is bin v / G: frequent
// tokens, which often have neighbouring ids, spread over the blocks. Every
// block reads all ids, counts its own tokens in LDS and the tokens of lower
// blocks (its offset in `order`), writes its bins' starts, and places its
// positions in order. start[g * (bins + 1) + b] is the first entry in `order`
// of bin b of block g, and entry [bins] its end.
//
// Reading all ids in each block costs N * 8 bytes of L2 reads per block, 64
// KiB at N = 8192 (twice that beyond), and saves the four to six dependent launches
// of a radix sort (8192 ids: 10 us, of which most are the dependent phases).
// Placement takes a batch of ids at a time: each wave finds, among 64 of the block's
// own entries, those that share a bin (one step per distinct bin), and one wave then
// runs through the groups of 64 in order with one LDS read and write each. Both grow
// with N on every block: 2^17 ids take 135 us, 2^20 1.0 ms, and 3.7 ms where all are
// one token, which one block places.
__global__ __launch_bounds__(kSortThreads) void token_sort_kernel(const int64_t* ids, int n,
                                                                  int64_t V, int g_log2, int bins,
                                                                  int* start, int* order) {
  __shared__ int hist[kSortBins];
  __shared__ int list_bin[kSortBatch], list_pos[kSortBatch];
  __shared__ unsigned char list_rank[kSortBatch], list_cnt[kSortBatch];
  __shared__ int wave_cnt[kSortItems * (kSortThreads / 64)];
  constexpr int W = kSortThreads / 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = blockIdx.x, mask = (1 << g_log2) - 1;
  for (int b = tid; b < bins; b += kSortThreads) hist[b] = 0;
  __syncthreads();
  int tok[kSortItems];  // the batch's ids, -1 where they take no part
  auto load = [&](int i0) {
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
      const int i = i0 + j * kSortThreads + tid;
      const int64_t id = i < n ? ids[i] : -1;
      tok[j] = id >= 0 && id < V ? static_cast<int>(id) : -1;
    }
  };
  int less = 0;
  for (int i0 = 0; i0 < n; i0 += kSortBatch) {
    load(i0);
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
      const int o = tok[j] & mask;
      if (tok[j] >= 0 && o < g) ++less;
      if (tok[j] >= 0 && o == g) atomicAdd(&hist[tok[j] >> g_log2], 1);
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) less += __shfl_xor(less, off, 64);
  if (lane == 0) wave_cnt[wave] = less;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < W; ++w) base += wave_cnt[w];
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
    for (int w = 0; w < W; ++w) {
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
  for (int i0 = 0; i0 < n; i0 += kSortBatch) {
    if (n > kSortBatch) load(i0);  // (else they are still held)
    // the block's own entries, in order
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
      const uint64_t b = __ballot(tok[j] >= 0 && (tok[j] & mask) == g);
      if (lane == 0) wave_cnt[j * W + wave] = __popcll(b);
    }
    __syncthreads();
    int m = 0, before[kSortItems];
    static_assert(kSortItems * W == 128, "two counts a lane");
    {
      const int c0 = wave_cnt[2 * lane], c1 = wave_cnt[2 * lane + 1];
      int x = c0 + c1;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int y = __shfl_up(x, off, 64);
        if (lane >= off) x += y;
      }
      m = __shfl(x, 63, 64);
#pragma unroll
      for (int j = 0; j < kSortItems; ++j) {
        const int at = j * W + wave;  // this wave's counter of item j
        const int end = __shfl(x, at >> 1, 64), last = __shfl(c1, at >> 1, 64),
                  first = __shfl(c0, at >> 1, 64);
        before[j] = at & 1 ? end - last : end - last - first;
      }
    }
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
      const bool mine = tok[j] >= 0 && (tok[j] & mask) == g;
      const uint64_t b = __ballot(mine);
      if (mine) {
        const int at = before[j] + __popcll(b & ((1ull << lane) - 1));
        list_bin[at] = tok[j] >> g_log2;
        list_pos[at] = i0 + j * kSortThreads + tid;
      }
    }
    __syncthreads();
    // rank of an entry among those of its bin in its group of 64; the first
    // of them also holds their number
    for (int e0 = wave * 64; e0 < m; e0 += kSortThreads) {
      const int e = e0 + lane;
      const int bin = e < m ? list_bin[e] : -1;
      uint64_t left = __ballot(e < m);
      while (left) {
        const int first = __ffsll(static_cast<unsigned long long>(left)) - 1;
        const uint64_t same = __ballot(bin == __shfl(bin, first, 64)) & left;
        if ((same >> lane) & 1) {
          list_rank[e] = static_cast<unsigned char>(__popcll(same & ((1ull << lane) - 1)));
          list_cnt[e] = static_cast<unsigned char>(__popcll(same));
        }
        left &= ~same;
      }
    }
    __syncthreads();
    if (wave == 0) {
      for (int e = lane; e - lane < m; e += 64) {
        if (e < m) {
          const int bin = list_bin[e], rank = list_rank[e], at = hist[bin];
          order[at + rank] = list_pos[e];
          if (rank == 0) hist[bin] = at + list_cnt[e];
        }
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------ sorted sums --

// acc += sum over j in [j0, j1) of w(order[j]) dY[order[j]], in order, eight
// rows in flight: a row's latency, some 2 us under load, is what long sums are made
// of (chunks of 16 rows at 8192 x 2048: 13 us with loads that wait for one another,
// 8 so).
template <typename TY, Kind K, class F>
__device__ __forceinline__ void add_rows(const TY* dY, const int* order, int j0, int j1,
                                         int d, const Cols<K>& k, F weight, float (&acc)[8]) {
  constexpr int U = 8;
  for (int j = j0; j < j1; j += U) {
    int pos[U];
    float w[U];
    Raw8<TY> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) pos[u] = order[min(j + u, j1 - 1)];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = weight(pos[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) x[u].load(dY + static_cast<int64_t>(pos[u]) * d, k);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (j + u < j1) {
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] = fmaf(w[u], x[u][q], acc[q]);
      }
  }
}

struct SortedIds {
  const int64_t* ids;
  const int* start;
  const int* order;
  int g_log2, bins;
  int chunk;  // entries of `order` a long token's sum is cut into
  __device__ __forceinline__ const int* range(int64_t v) const {
    return start + (v & ((1 << g_log2) - 1)) * (bins + 1) + (v >> g_log2);
  }
  __device__ __forceinline__ int total() const {
    return start[(static_cast<int64_t>(bins) + 1) * (1 << g_log2) - 1];
  }
};

struct SampleWeight {
  const float* s;  // [B] or null
  float scale;
  int T;
  __device__ __forceinline__ float operator()(int pos) const {
    return s ? scale * s[pos / T] : scale;
  }
};

// A token that occurs more than `chunk` times is summed in aligned chunks of
// `order` first, one block per chunk and slot: slot 0 of a chunk holds the sum of its
// first entry's token, slot 1 that of its last entry's token where that one
// begins inside the chunk. (No long token lies wholly inside a chunk.) Without
// this the most frequent token's sum, 459 rows of 7168 in a 1 / rank
// distribution over 50304 tokens, outlasts all others: 490 us against 90.
template <typename TY, Kind K>
__global__ __launch_bounds__(kThreads) void embed_chunk_kernel(const TY* dY, int d, SortedIds o,
                                                               SampleWeight weight, int tpr_log2,
                                                               float* part) {
  const int tpr = 1 << tpr_log2;
  const int total = o.total(), rows = kThreads >> tpr_log2;
  const int chunk = blockIdx.x * rows + (threadIdx.x >> tpr_log2);
  const int j0 = chunk * o.chunk, j1 = min(total, j0 + o.chunk);
  if (j0 >= j1) return;
  const int* first = o.range(o.ids[o.order[j0]]);
  const int* last = o.range(o.ids[o.order[j1 - 1]]);
  const int fb = first[0], fe = first[1], lb = last[0], le = last[1];
  const int slot = blockIdx.y;
  const int b = slot == 0 ? j0 : lb, e = slot == 0 ? min(fe, j1) : j1;
  if (slot == 0 ? fe - fb <= o.chunk : (lb <= j0 || le - lb <= o.chunk)) return;
  for (int c = Cols<K>::first(threadIdx.x & (tpr - 1)); c < d; c += tpr * 8) {
    const Cols<K> k(c, 0, d);
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    add_rows(dY, o.order, b, e, d, k, weight, acc);
    store8(part + (static_cast<int64_t>(chunk) * 2 + slot) * d, k, acc, false);
  }
}

// 1 << tpr_log2 threads per vocabulary row: its positions are added in order
// (its chunks' sums, for a long token). Bound by writing the table (50304 x 2048, fp32:
// 70 us, 5.9 TB/s; a fill reaches 6.7).
template <typename TY, typename TE, Kind K>
__global__ __launch_bounds__(kThreads) void embed_grad_kernel(const TY* dY, int64_t V, int d,
                                                              SortedIds o, SampleWeight weight,
                                                              const float* part, int tpr_log2,
                                                              int accumulate, TE* dE) {
  const int tpr = 1 << tpr_log2;
  const int64_t v = static_cast<int64_t>(blockIdx.x) * (kThreads >> tpr_log2) +
                    (threadIdx.x >> tpr_log2);
  if (v >= V) return;
  const int* st = o.range(v);
  const int j0 = st[0], j1 = st[1];
  if (accumulate && j0 == j1) return;
  TE* dst = dE + v * d;
  for (int c = Cols<K>::first(threadIdx.x & (tpr - 1)); c < d; c += tpr * 8) {
    const Cols<K> k(c, tpr * 4, d);
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (j1 - j0 <= o.chunk) {
      add_rows(dY, o.order, j0, j1, d, k, weight, acc);
    } else {
      const int h0 = j0 / o.chunk, h1 = (j1 - 1) / o.chunk;
      for (int h = h0; h <= h1; h += 8) {
        Raw8<float> x[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int at = min(h + u, h1);
          x[u].load(part + (static_cast<int64_t>(at) * 2 + (at == h0 && j0 % o.chunk != 0)) * d, k);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (h + u <= h1) {
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] += x[u][q];
          }
      }
    }
    if (accumulate) {
      Raw8<TE> x;
      x.load(dst, k);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] += x[q];
    }
    store8(dst, k, acc, accumulate != 0);
  }
}

// ------------------------------------------------------------------ norms --

// ||scale sum over j in [j0, j1) of dY[list[j]]||^2, by one block; the same value
// in thread 0 only. 1 << tpr_log2 threads share a row; where that leaves threads
// over (d up to 1024), each group of so many adds a part of a long run, and the parts
// are added in order; wider rows' runs are one chain (a sample of one token 8192 times:
// all of the operator 0.33 ms at d 512, 0.57 at 1024, 1.0 at 2048, 2.0 at 4096). A wave reads 64 entries of the
// list at once, so that the rows' loads do not wait for their positions. (2 x 3957
// positions over 632 tokens, d 576: 122 us in one chain of batches, 30 us so; 16 x 512
// over 50304, d 2048: 19 us.) Rows are added in fp32 64 at a time and those sums in
// 64 bits: in one fp32 chain the terms of a long run of like sign fall below the sum's
// last bits (2^20 equal rows of 5 columns: off by 2.1e-3, and a sample whose norm is
// too small is clipped too little).
template <typename TY, Kind K>
__device__ __forceinline__ float run_norm(const TY* dY, int d, const int* list, int j0, int j1,
                                          int tpr_log2, float scale) {
  constexpr int U = 8;
  __shared__ float parts[kThreads * 8];
  __shared__ float red[4];
  const int tid = threadIdx.x, lane = tid & 63;
  // (a group is one or more whole waves)
  const int tpr = max(64, 1 << tpr_log2), groups = j1 - j0 > U ? kThreads / tpr : 1;
  const int group = __builtin_amdgcn_readfirstlane(tid / tpr), t = tid % tpr;
  const int per = (j1 - j0 + groups - 1) / groups;
  const int b = j0 + group * per, e = group < groups ? min(j1, b + per) : b;
  float sq = 0.0f;
  for (int c0 = 0; c0 < d; c0 += tpr * 8) {
    const int c = c0 + t * 8;
    const Cols<K> k(c, 0, d);
    float acc[8];
    double sum[8] = {0., 0., 0., 0., 0., 0., 0., 0.};
    for (int j = b; j < e; j += 64) {
      const int mine = list[min(j + lane, e - 1)], m = min(64, e - j);
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[q] = 0.0f;
      for (int u0 = 0; u0 < m; u0 += U) {
        Raw8<TY> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int pos = __builtin_amdgcn_readlane(mine, u0 + u);
          x[u].load(dY + static_cast<int64_t>(pos) * d, k);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u0 + u < m) {
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] += x[u][q];
          }
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) sum[q] += acc[q];
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = static_cast<float>(sum[q]);
    if (groups > 1) {  // (then this loop's only pass)
#pragma unroll
      for (int q = 0; q < 8; ++q) parts[tid * 8 + q] = acc[q];
      __syncthreads();
      if (group == 0)
        for (int g = 1; g < groups; ++g) {
#pragma unroll
          for (int q = 0; q < 8; ++q) acc[q] += parts[(g * tpr + t) * 8 + q];
        }
    }
    if (group == 0) {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (k.mine(q)) sq = fmaf(scale * acc[q], scale * acc[q], sq);
    }
  }
  sq = wave_sum(sq);
  if (lane == 0) red[tid >> 6] = sq;
  __syncthreads();
  return ((red[0] + red[1]) + red[2]) + red[3];
}

// One block per entry of `order`: the first entry of a (token,
// sample) run adds the run's rows and writes the squared norm of the sum at
// its position, the others write zero.
template <typename TY, Kind K>
__global__ __launch_bounds__(kThreads) void embed_run_norm_kernel(const TY* dY, int d, SortedIds o,
                                                                  int T, float scale,
                                                                  int tpr_log2, float* run_sq) {
  const int j = blockIdx.x;
  if (j >= o.total()) return;
  const int pos = o.order[j];
  const int64_t id = o.ids[pos];
  const int sample = pos / T;
  if (j > 0) {
    const int prev = o.order[j - 1];
    if (o.ids[prev] == id && prev / T == sample) {
      if (threadIdx.x == 0) run_sq[pos] = 0.0f;
      return;
    }
  }
  // the run ends before the first later entry of another sample; each wave
  // looks at 64 entries at a time
  const int end = o.range(id)[1];
  int e = j + 1;
  for (;;) {
    const int at = e + static_cast<int>(threadIdx.x & 63);
    const uint64_t out = __ballot(at >= end || o.order[min(at, end - 1)] / T != sample);
    if (out) {
      e += __ffsll(static_cast<unsigned long long>(out)) - 1;
      break;
    }
    e += 64;
  }
  const float sq = run_norm<TY, K>(dY, d, o.order, j, e, tpr_log2, scale);
  if (threadIdx.x == 0) run_sq[pos] = sq;
}

// The same for short samples, without sorting: one block per position compares
// its id with its sample's other ids (T * 8 bytes of L2 reads a block); the
// first position of a run lists the others in LDS, in order.
constexpr int kShortSample = 1024;
template <typename TY, Kind K>
__global__ __launch_bounds__(kThreads) void embed_short_norm_kernel(const int64_t* ids,
                                                                    const TY* dY, int64_t V, int d,
                                                                    int T, float scale,
                                                                    int tpr_log2, float* run_sq) {
  __shared__ int list[kShortSample];
  __shared__ int wave_cnt[kShortSample / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int pos = blockIdx.x, first = pos / T * T;
  const int64_t id = ids[pos];
  if (id < 0 || id >= V) return;
  constexpr int kPer = kShortSample / kThreads;
  uint64_t same[kPer];
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int at = q * kThreads + tid;
    same[q] = __ballot(at < T && ids[first + min(at, T - 1)] == id);
    if (lane == 0) wave_cnt[q * 4 + wave] = __popcll(same[q]);
  }
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    for (int w = 0; w < 4; ++w) {
      if (w == wave && (same[q] >> lane) & 1)
        list[all + __popcll(same[q] & ((1ull << lane) - 1))] = first + q * kThreads + tid;
      all += wave_cnt[q * 4 + w];
    }
  }
  __syncthreads();
  if (list[0] != pos) {  // the run's first position
    if (tid == 0) run_sq[pos] = 0.0f;
    return;
  }
  const float sq = run_norm<TY, K>(dY, d, list, 0, all, tpr_log2, scale);
  if (tid == 0) run_sq[pos] = sq;
}

// norm_sq[i] += the run norms at sample i's positions, in a fixed order. Summed in 64
// bits: a thread adds up to 2^15 terms of like sign (2^22 tokens of equal size, in
// fp32: off by 1.4e-4).
__global__ __launch_bounds__(kThreads) void embed_norm_sum_kernel(const int64_t* ids, int64_t V,
                                                                  int T, const float* run_sq,
                                                                  float* norm_sq) {
  __shared__ double red[4];
  const int64_t base = static_cast<int64_t>(blockIdx.x) * T;
  double t = 0.0;
  for (int k0 = threadIdx.x; k0 < T; k0 += 4 * kThreads) {  // (four loads in flight)
    int64_t id[4];
    float x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t at = base + min(k0 + u * kThreads, T - 1);
      id[u] = ids[at], x[u] = run_sq[at];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (k0 + u * kThreads < T && id[u] >= 0 && id[u] < V) t += x[u];
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) t += __shfl_xor(t, off, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = t;
  __syncthreads();
  if (threadIdx.x == 0) norm_sq[blockIdx.x] += static_cast<float>(((red[0] + red[1]) + red[2]) + red[3]);
}

// ------------------------------------------------------------------- host --

int fail(int code, const std::string& msg) { return record_error(code, msg.c_str()); }

int check_launch(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(DPG_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
  return DPG_OK;
}

bool valid_dtype(int32_t t) { return t == DPG_FP32 || t == DPG_BF16; }
size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

// fn with how a thread takes a row of d columns.
template <class F>
void with_kind(int64_t d, F fn) {
  if (d < 8) fn(std::integral_constant<Kind, NARROW>{});
  else fn(std::integral_constant<Kind, WIDE>{});
}

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
  int g_log2 = 0, bins = 0, chunk = 16, chunks = 0;
  size_t off_order = 0, off_run = 0, off_part = 0, total = 0;
  SortedIds sorted(const int64_t* ids, const char* ws) const {
    return {ids, reinterpret_cast<const int*>(ws), reinterpret_cast<const int*>(ws + off_order),
            g_log2, bins, chunk};
  }
};

// 256 sorting blocks (one per CU), fewer for vocabularies under 1024, more
// where a block's share of the tokens would exceed its LDS bins. At most 512
// chunks: a sum over one token takes chunk rows and then up to n / chunk.
SortPlan plan_sort(int64_t n, int64_t V, int64_t d) {
  SortPlan p;
  while (p.g_log2 < 8 && (4ll << p.g_log2) <= V) ++p.g_log2;
  while (((V - 1) >> p.g_log2) + 1 > kSortBins) ++p.g_log2;
  p.bins = static_cast<int>(((V - 1) >> p.g_log2) + 1);
  p.off_order = align_up((static_cast<size_t>(1) << p.g_log2) * (p.bins + 1) * 4);
  p.off_run = p.off_order + align_up(static_cast<size_t>(n) * 4);
  // (up to 128 tokens, a launch for the chunks costs more than the longest sum)
  if (n <= 128) p.chunk = 128;
  while (n > 512ll * p.chunk) p.chunk *= 2;
  p.chunks = static_cast<int>(ceil_div(n, p.chunk));
  // (the norms' runs and the gradient's chunks are never needed together)
  p.off_part = p.off_run;
  p.total = p.off_run + align_up(std::max<size_t>(n * 4, n > p.chunk ? p.chunks * 2 * d * 4 : 0));
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
  with_kind(d, [&](auto k) {
    hipLaunchKernelGGL((embed_kernel<TE, TY, decltype(k)::value>),
                       dim3(static_cast<unsigned>(ceil_div(n, kThreads >> l))), dim3(kThreads), 0, s,
                       ids, n, static_cast<const TE*>(E), V, static_cast<int>(d),
                       static_cast<float>(scale), l, static_cast<TY*>(Y));
  });
}

template <typename TY, typename TE>
void launch_embed_grad(const SortPlan& p, const int64_t* ids, const void* dY, int64_t n, int64_t T,
                       int64_t V, int64_t d, double scale, const float* sample_scales,
                       int accumulate, void* dE, char* ws, hipStream_t s) {
  const int l = row_threads_log2(d);
  const dim3 b(kThreads);
  const SortedIds o = p.sorted(ids, ws);
  const SampleWeight weight{sample_scales, static_cast<float>(scale), static_cast<int>(T)};
  float* part = reinterpret_cast<float*>(ws + p.off_part);
  const TY* dy = static_cast<const TY*>(dY);
  with_kind(d, [&](auto k) {
    constexpr Kind K = decltype(k)::value;
    if (n > p.chunk)
      hipLaunchKernelGGL((embed_chunk_kernel<TY, K>),
                         dim3(static_cast<unsigned>(ceil_div(p.chunks, kThreads >> l)), 2), b, 0, s,
                         dy, static_cast<int>(d), o, weight, l, part);
    hipLaunchKernelGGL((embed_grad_kernel<TY, TE, K == WIDE && sizeof(TE) == 4 ? SPLIT : K>),
                       dim3(static_cast<unsigned>(ceil_div(V, kThreads >> l))), b, 0, s, dy, V,
                       static_cast<int>(d), o, weight, part, l, accumulate, static_cast<TE*>(dE));
  });
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
  *bytes = plan_sort(B * T, V, d).total;
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
  const SortPlan p = plan_sort(B * T, V, d);
  if (const int st = check_ws(workspace, workspace_bytes, p.total)) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  // few positions of short samples are compared with each other, others sorted:
  // at 128 positions 5 us against 8 + 3, at 2331 (T = 333) 13 against 9 + 11, at
  // 8192 (T = 512) 34 against 10 + 24, and comparing grows with T
  const bool sorted = T > kShortSample || B * T > 4096;
  if (sorted)
    if (const int st = sort_tokens(p, ids, B * T, V, ws, s)) return st;
  float* run_sq = reinterpret_cast<float*>(ws + p.off_run);
  const int l = row_threads_log2(d);
  auto go = [&](auto zero) {
    typedef decltype(zero) TY;
    with_kind(d, [&](auto k) {
      constexpr Kind K = decltype(k)::value;
      const dim3 grid(static_cast<unsigned>(B * T)), b(kThreads);
      if (sorted)
        hipLaunchKernelGGL((embed_run_norm_kernel<TY, K>), grid, b, 0, s,
                           static_cast<const TY*>(dY), static_cast<int>(d), p.sorted(ids, ws),
                           static_cast<int>(T), static_cast<float>(scale), l, run_sq);
      else
        hipLaunchKernelGGL((embed_short_norm_kernel<TY, K>), grid, b, 0, s, ids,
                           static_cast<const TY*>(dY), V, static_cast<int>(d), static_cast<int>(T),
                           static_cast<float>(scale), l, run_sq);
    });
  };
  if (dtype == DPG_BF16) go(bf16());
  else go(0.0f);
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
  const SortPlan p = plan_sort(B * T, V, d);
  if (const int st = check_ws(workspace, workspace_bytes, p.total)) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  if (const int st = sort_tokens(p, ids, B * T, V, ws, s)) return st;
  if (table_dtype == DPG_BF16)
    launch_embed_grad<bf16, bf16>(p, ids, dY, B * T, T, V, d, scale, sample_scales,
                                  accumulate, dE, ws, s);
  else if (dtype == DPG_BF16)
    launch_embed_grad<bf16, float>(p, ids, dY, B * T, T, V, d, scale, sample_scales,
                                  accumulate, dE, ws, s);
  else
    launch_embed_grad<float, float>(p, ids, dY, B * T, T, V, d, scale, sample_scales,
                                  accumulate, dE, ws, s);
  return check_launch("embed_grad");
}

}  // extern "C"
