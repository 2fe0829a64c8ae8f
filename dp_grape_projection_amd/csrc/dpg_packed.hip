// A layer's projection from its input in 8 bits, for fp32 operands:
// Xt[b][j][t] = sum_k P[j][k] A[b][t][k], and where the step's own kernels would leave
// most CUs idle over a long T, G_hat[b][j][n] = sum_t Xt[b][j][t] dY[b][t][n] as well.
//
// What a code stands for is a bf16 number, so that A is exact as it is on the 16-bit matrix
// instructions, which are 16 times as fast as the fp32 ones; P, in fp32, is split exactly
// into three bf16 parts, and three products are all there are, the small ones first. One
// launch reads the codes back and generates P, the second is the product; where few tiles
// share a long d_in, that is split and the sums added by another. (4096 tokens
// x 768, r 128: 18 us in all, 30 with A read back to fp32 and the fp32 instructions.)
#include <algorithm>
#include <type_traits>

#include "dpg_act8.hpp"
#include "dpg_device.hpp"
#include "dpg_internal.hpp"
#include "dpg_tile.hpp"

namespace dpg {
namespace {

struct PackedPrepArgs {
  Act8Args a;
  int32_t a_blocks, p_blocks;
  bf16* P;          // [3][r][ld]
  int32_t d_in, ld, r;
  uint32_t n_ctr;   // counters of four normals
  float scale;
  uint32_t layer_id;
  StreamKey key;
};

__global__ __launch_bounds__(kThreads) void packed_prep_kernel(const PackedPrepArgs a) {
  const int block = blockIdx.x;
  if (block < a.a_blocks) {
    unpack8_block<bf16>(a.a, block);
    return;
  }
  const uint32_t t = static_cast<uint32_t>(block - a.a_blocks) * kThreads + threadIdx.x;
  const int64_t part = static_cast<int64_t>(a.r) * a.ld;
  if (block < a.a_blocks + a.p_blocks) {
    if (t >= a.n_ctr) return;
    float z[4];
    normals_at(a.key, a.layer_id, t, z);
    uint32_t j = 4 * t / static_cast<uint32_t>(a.d_in), k = 4 * t - j * static_cast<uint32_t>(a.d_in);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (j < static_cast<uint32_t>(a.r)) {
        bf16 p[3];
        split3(z[q] * a.scale, p);
#pragma unroll
        for (int i = 0; i < 3; ++i) a.P[i * part + static_cast<int64_t>(j) * a.ld + k] = p[i];
      }
      if (++k == static_cast<uint32_t>(a.d_in)) k = 0, ++j;
    }
    return;
  }
  // zero from d_in on
  const uint32_t pad = static_cast<uint32_t>(a.ld - a.d_in), at = t - static_cast<uint32_t>(a.p_blocks) * kThreads;
  const uint32_t j = at / pad;
  if (j >= static_cast<uint32_t>(a.r)) return;
#pragma unroll
  for (int i = 0; i < 3; ++i)
    a.P[i * part + static_cast<int64_t>(j) * a.ld + a.d_in + (at - j * pad)] = zero_val<bf16>();
}

struct PackedProductArgs {
  const bf16 *A, *P;
  float* Xt;      // [B][r][ldt], or, with splits,
  float* part;    // [splits][r][B T]
  int32_t B, T, r, ld, ldt, splits;
};

// A tile of tokens (M) by rows of P (N): a lane holds four consecutive tokens of one row.
template <class G>
__global__ __launch_bounds__(G::kThreads, G::kBlocks) void packed_product_kernel(const PackedProductArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[G::kLds];
  const int BT = a.B * a.T, nts = (a.r + G::kTile - 1) / G::kTile;
  int mt, nt;
  if (!tile_of_block(blockIdx.x, (BT + G::kTile - 1) / G::kTile, nts * a.splits, mt, nt)) return;
  const int split = nt / nts, m0 = mt * G::kTile, n0 = (nt - split * nts) * G::kTile;
  const int steps = a.ld / kStepK, per = (steps + a.splits - 1) / a.splits;
  const int k0 = min(steps, split * per), k1 = min(steps, k0 + per), kk = k0 * kStepK;
  typename G::Acc acc;
  tile_product<G, kThree, false, false>(
      rows_operand(a.A + static_cast<int64_t>(m0) * a.ld + kk, a.ld, 0, BT - m0, a.ld - kk),
      rows_operand(a.P + static_cast<int64_t>(n0) * a.ld + kk, a.ld, static_cast<int64_t>(a.r) * a.ld,
                   a.r - n0, a.ld - kk),
      k1 - k0, smem, acc);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave % G::kWavesM, wn = wave / G::kWavesM, r16 = lane & 15, kq = lane >> 4;
#pragma unroll
  for (int nb = 0; nb < G::kNB; ++nb) {
    const int j = n0 + G::kWaveN * wn + 16 * nb + r16;
    if (j >= a.r) continue;
#pragma unroll
    for (int mb = 0; mb < G::kMB; ++mb) {
      const int n = m0 + G::kWaveM * wm + 16 * mb + 4 * kq;
      if (n >= BT) continue;
      const f32x4 x = acc.v[mb][nb];
      const int b = n / a.T, t = n - b * a.T;
      float* dst = a.splits > 1 ? a.part + (static_cast<int64_t>(split) * a.r + j) * BT + n
                                : a.Xt + (static_cast<int64_t>(b) * a.r + j) * a.ldt + t;
      if ((a.T & 3) == 0) {
        *reinterpret_cast<f32x4*>(dst) = x;
      } else if (a.splits > 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < BT) dst[i] = x[i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (n + i >= BT) continue;
          const int bi = (n + i) / a.T;
          a.Xt[(static_cast<int64_t>(bi) * a.r + j) * a.ldt + (n + i - bi * a.T)] = x[i];
        }
      }
    }
  }
}

struct PackedHatArgs {
  const float *Xt, *dY;
  float* hat;       // [B][parts][r][d_out]
  int64_t ldt, d_out;
  int32_t B, T, r, parts, per, off32;
  int32_t m_tiles, n_tiles;
};

// One part of T of a tile of one sample's product, both operands in fp32.
typedef Tile<float, kTileM, kTileN, kStepF32, 4, 1> HatTile;
__global__ __launch_bounds__(kThreads, 2) void packed_hat_kernel(const PackedHatArgs a) {
  typedef HatTile Tl;
  __shared__ __attribute__((aligned(16))) float smem[Tl::kLdsElems];
  const int block = xcd_logical_block(), tiles = a.m_tiles * a.n_tiles;
  const int run = block / tiles, at = block - run * tiles;  // a sample's part
  if (run >= a.B * a.parts) return;
  const int i = run / a.parts, t0 = (run - i * a.parts) * a.per;
  const int j0 = at % a.m_tiles * Tl::BM, n0 = at / a.m_tiles * Tl::BN;
  const int K = min(a.per, a.T - t0);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  RowsLoader<float, Tl::BM, Tl::BK, true, IdentityRows> la{a.ldt, a.r - j0, K, {}};
  ColsLoader<float, Tl::BN, Tl::BK, true, BOperandRows<Tl>> lb{a.d_out, static_cast<int>(a.d_out) - n0, K, {}};
  const float* const Xt = a.Xt + (static_cast<int64_t>(i) * a.r + j0) * a.ldt + t0;
  const float* const dY = a.dY + (static_cast<int64_t>(i) * a.T + t0) * a.d_out + n0;
  Acc<Tl::MB, Tl::NB> acc;
  acc.zero();
  run_steps<float, Tl>(
      la, lb, smem, acc, (K + Tl::BK - 1) / Tl::BK, tid,
      [&](int s) {
        la.load(Xt, s * Tl::BK, tid, a.off32);
        lb.load(dY, s * Tl::BK, tid, a.off32);
      },
      [](int) {});
  store_tile<Tl>(a.hat + static_cast<int64_t>(run) * a.r * a.d_out, acc, a.r, static_cast<int>(a.d_out), j0, n0,
                 wave, lane);
}

// G_hat from its parts, added in their order, and the squared norm of each block's share.
__global__ __launch_bounds__(kThreads) void packed_join_kernel(const float* hat, float* ghat, float* norm_part,
                                                               int32_t parts, int64_t size, int32_t chunk,
                                                               int32_t slots) {
  __shared__ float sums[kThreads / 64];
  const int i = blockIdx.x / slots, slot = blockIdx.x - i * slots;
  const int64_t first = static_cast<int64_t>(slot) * chunk, end = min(size, first + chunk);
  hat += static_cast<int64_t>(i) * parts * size;
  float sq = 0.0f;
  for (int64_t e = first + threadIdx.x; e < end; e += kThreads) {
    float g = 0.0f;
    int p = 0;
    auto add = [&](auto n) {  // (n loads in flight)
      float x[decltype(n)::value];
#pragma unroll
      for (int u = 0; u < decltype(n)::value; ++u) x[u] = hat[(p + u) * size + e];
#pragma unroll
      for (int u = 0; u < decltype(n)::value; ++u) g += x[u];
      p += decltype(n)::value;
    };
    while (p + 8 <= parts) add(std::integral_constant<int, 8>{});
    if (parts & 4) add(std::integral_constant<int, 4>{});
    if (parts & 2) add(std::integral_constant<int, 2>{});
    if (parts & 1) add(std::integral_constant<int, 1>{});
    ghat[static_cast<int64_t>(i) * size + e] = g;
    sq = fmaf(g, g, sq);
  }
  sq = wave_sum(sq);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sq;
  __syncthreads();
  if (threadIdx.x == 0) norm_part[blockIdx.x] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}
static_assert(kThreads == 256, "the join adds four waves' sums");

}  // namespace

// Parts of T. Modelled on measurements: a step of a block alone on its CU takes 3.2 us, of
// two together 5.8 (the fp32 matrix instructions bound both), a launch 4.5, the join 2.5,
// 0.12 for every part of an element and its bytes. fp32 sums over T one after the other
// also lose bits: at most kMostT tokens, as long as all parts take 512 MiB at most (1 x 5906
// x 1600 x 384, r 8: error 1.4e-6 in one part, 2.5e-7 so). A whole call of
// dpg_project_layer, which keeps a sample's T in one block, and of this one: 1 x 5906 x 1600 x
// 384, r 8: 657 and 49 us; 1 x 8192 x 2048 x 2048, r 256: 863 and 171; 8 x 1000 x 768 x 768,
// r 128: 136 and 59. Parts where one fills the CUs: 32 x 256 x 768 x 768, r 128: 65 us in
// two, 54 in one.
constexpr int64_t kMostT = 2048;
int64_t parts_of(int64_t B, int64_t T, int64_t d_out, int64_t r) {
  const int64_t blocks = B * ceil_div(r, kTileM) * ceil_div(d_out, kTileN), all = ceil_div(T, kStepF32);
  const double elems = static_cast<double>(B * r) * static_cast<double>(d_out) / 1e6;
  int64_t best = 1;
  double best_us = 1e30;
  for (int64_t k = 1; k <= std::max<int64_t>(1, std::min(512 / blocks, all)); k += std::max<int64_t>(1, k / 4)) {
    const double step = blocks * k <= 256 ? 3.2 : 5.8 * static_cast<double>(ceil_div(blocks * k, 512));
    double us = static_cast<double>(ceil_div(all, k)) * step + 4.5;
    const double n = static_cast<double>(k), each = static_cast<double>(ceil_div(r * d_out, 256 * kThreads));
    if (k > 1) us += 2.5 + 0.12 * n * each + elems * (8.0 * n + 4.0) / 5.0;
    if (us < best_us) best_us = us, best = k;
  }
  const int64_t room = (int64_t{1} << 29) / (B * r * d_out * 4);
  return std::max<int64_t>(1, std::min(room, std::max(ceil_div(T, kMostT), best)));
}

// Tiny tiles where the others would leave most CUs idle; d_in split where even those do
// and it is long.
PackedPlan plan_packed(int64_t B, int64_t T, int64_t d_in, int64_t d_out, int32_t r) {
  const int64_t BT = B * T;
  PackedPlan p;
  p.ld = round_up(d_in, kStepK);
  const int64_t tiny = ceil_div(BT, TinyTile::kTile) * ceil_div(r, TinyTile::kTile), steps = p.ld / kStepK;
  p.small = tiny > 1024;
  p.splits = p.small ? 1
                     : static_cast<int32_t>(std::max<int64_t>(1, std::min(512 / tiny, steps / 3)));
  // (no empty part)
  p.splits = static_cast<int32_t>(ceil_div(steps, ceil_div(steps, p.splits)));
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    const size_t at = off;
    off += align_up(static_cast<size_t>(bytes));
    return at;
  };
  take(BT * p.ld * 2);
  p.off_P = take(3 * static_cast<int64_t>(r) * p.ld * 2);
  p.off_part = take(p.splits > 1 ? p.splits * r * BT * 4 : 0);
  p.per = static_cast<int32_t>(ceil_div(ceil_div(T, kStepF32), parts_of(B, T, d_out, r)) * kStepF32);
  p.parts = static_cast<int32_t>(ceil_div(T, p.per));
  p.chunk = static_cast<int32_t>(ceil_div(r * d_out, 256 * kThreads) * kThreads);
  p.slots = static_cast<int32_t>(ceil_div(r * d_out, p.chunk));
  p.off_hat = take(p.parts > 1 ? B * p.parts * r * d_out * 4 : 0);
  p.off_slots = take(p.parts > 1 ? B * p.slots * 4 : 0);
  p.total = off;
  return p;
}

hipError_t launch_packed_prep(const PackedPlan& p, const int8_t* codes, const uint8_t* exps, int64_t BT,
                              int64_t d_in, int32_t r, uint32_t layer_id, uint64_t seed, uint32_t proj_step,
                              float scale, char* ws, hipStream_t s) {
  PackedPrepArgs a{};
  a.a = unpack_args(codes, exps, BT, d_in, ws, p.ld);
  a.a_blocks = static_cast<int32_t>(cover_rows(a.a));
  a.P = reinterpret_cast<bf16*>(ws + p.off_P);
  a.d_in = static_cast<int32_t>(d_in), a.ld = static_cast<int32_t>(p.ld), a.r = r;
  a.n_ctr = static_cast<uint32_t>((static_cast<uint64_t>(r) * d_in + 3) / 4);
  a.p_blocks = static_cast<int32_t>(ceil_div(a.n_ctr, kThreads));
  a.scale = scale, a.layer_id = layer_id;
  a.key = {static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32), proj_step, 0u};
  const int64_t pad_blocks = ceil_div(r * (p.ld - d_in), kThreads);
  hipLaunchKernelGGL(packed_prep_kernel, dim3(static_cast<unsigned>(a.a_blocks + a.p_blocks + pad_blocks)),
                     dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_packed_product(const PackedPlan& p, int64_t B, int64_t T, int32_t r, int64_t ldt,
                                 const char* ws, float* Xt, float* part, hipStream_t s) {
  PackedProductArgs a{};
  a.A = reinterpret_cast<const bf16*>(ws), a.P = reinterpret_cast<const bf16*>(ws + p.off_P);
  a.Xt = Xt, a.part = part;
  a.B = static_cast<int32_t>(B), a.T = static_cast<int32_t>(T), a.r = r;
  a.ld = static_cast<int32_t>(p.ld), a.ldt = static_cast<int32_t>(ldt), a.splits = p.splits;
  auto run = [&](auto g) {
    typedef decltype(g) G;
    hipLaunchKernelGGL(packed_product_kernel<G>,
                       tile_grid(ceil_div(B * T, G::kTile), ceil_div(r, G::kTile) * p.splits),
                       dim3(G::kThreads), 0, s, a);
  };
  if (p.small) run(SmallTile());
  else run(TinyTile());
  return hipGetLastError();
}

hipError_t launch_packed_hat(const PackedPlan& p, int64_t B, int64_t T, int32_t r, int64_t ldt, int64_t d_out,
                             const float* Xt, const float* dY, char* ws, float* ghat, hipStream_t s) {
  PackedHatArgs a{};
  a.Xt = Xt, a.dY = dY, a.hat = reinterpret_cast<float*>(ws + p.off_hat);
  a.ldt = ldt, a.d_out = d_out;
  a.B = static_cast<int32_t>(B), a.T = static_cast<int32_t>(T), a.r = r;
  a.parts = p.parts, a.per = p.per;
  a.off32 = kTileM * ldt * 4 < (1ll << 31) && p.per * d_out * 4 < (1ll << 31);
  a.m_tiles = static_cast<int32_t>(ceil_div(r, kTileM)), a.n_tiles = static_cast<int32_t>(ceil_div(d_out, kTileN));
  hipLaunchKernelGGL(packed_hat_kernel, dim3(static_cast<unsigned>(round_up(B * p.parts * a.m_tiles * a.n_tiles, 8))),
                     dim3(kThreads), 0, s, a);
  hipLaunchKernelGGL(packed_join_kernel, dim3(static_cast<unsigned>(B * p.slots)), dim3(kThreads), 0, s, a.hat, ghat,
                     reinterpret_cast<float*>(ws + p.off_slots), p.parts, r * d_out, p.chunk, p.slots);
  return hipGetLastError();
}

}  // namespace dpg
