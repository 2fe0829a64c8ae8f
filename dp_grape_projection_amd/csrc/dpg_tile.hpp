// Matrix-core products in tiles staged through LDS by direct copies, for operands
// whose K runs along their rows or down their columns, in bf16 or in fp32 as parts
// of 16 bits; with what the callers need around a tile: rows of any alignment,
// writing a tile, splits of K, checks of workspaces.
#pragma once

#include <algorithm>
#include <string>
#include <type_traits>

#include "dpg.h"
#include "dpg_device.hpp"
#include "dpg_internal.hpp"

namespace dpg {

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
// One operand in two bf16 parts, the other in one, with its parts 0 elements apart.
constexpr int kTwo = 4;
template <> struct Combos<kTwo> {
  static constexpr int n = 2;
  __device__ __forceinline__ static int a(int c) { return c == 0 ? 1 : 0; }
  __device__ __forceinline__ static int b(int c) { return c == 0 ? 1 : 0; }
};
// The same with three parts.
constexpr int kThree = 5;
template <> struct Combos<kThree> {
  static constexpr int n = 3;
  __device__ __forceinline__ static int a(int c) { return (0x012 >> (4 * c)) & 15; }
  __device__ __forceinline__ static int b(int c) { return (0x012 >> (4 * c)) & 15; }
};
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

// --------------------------------------------------------------- products --
//
// One device function computes products A B^T in tiles of 256 x 256 (8
// waves of 128 x 64, one block per CU) or, where those would not fill the 256
// CUs, 128 x 128 (4 waves of 64 x 64, two blocks per CU), with 16x16x32 matrix
// instructions; those of the losses, for instance:
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

// The same for any N < 64.
template <int N> __device__ __forceinline__ void wait_vm_all() {
  static_assert(N < 64, "six bits of the count");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
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

// fn(std::integral_constant<int, 0>) .. <N - 1>: unrolled whatever its size, so that the
// accumulators it indexes stay in registers.
template <class F, int... I>
__device__ __forceinline__ void each_of(F fn, std::integer_sequence<int, I...>) {
  (fn(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F fn) {
  each_of(fn, std::make_integer_sequence<int, N>{});
}

// Slot of 16-byte chunk c in row k of a k-major tile of CHUNKS chunks a row. Of the
// transposing read, 16 lanes take 32 bytes from each of four rows, and the
// next 16 the same eight rows further on: the slots of these eight pieces
// differ in their 64 banks (rows of 8 chunks fill half of them, so that two rows do).
template <int CHUNKS>
__device__ __forceinline__ int kslot(int k, int c) {
  if constexpr (CHUNKS == 8) return c ^ (2 * ((k >> 1) & 1)) ^ (4 * ((k >> 3) & 1));
  else return c ^ (4 * (k & 3)) ^ (2 * ((k >> 3) & 1));
}

struct Operand {
  const bf16* base;     // first row of the tile (rows) or of K (k-major)
  int64_t ld;           // row stride, elements
  int64_t part_stride;  // elements between the bf16 parts
  int rows;             // rows: rows there are from base; k-major: rows of K
  int cols;             // rows: elements of K in a row; k-major: columns from base
  int64_t half = 0;     // k-major: where not 0, a wave's columns are half from base
                        // on and half from base + half on (elements, a multiple of 8)
  bool apart = false;   // and the next wave's a whole wave's columns further, not half
};

// Byte offset in a row of a k-major operand of what the tile has as its chunk c of eight
// columns.
template <class G>
__device__ __forceinline__ uint32_t column_chunk(const Operand& o, int c) {
  if (!o.half) return static_cast<uint32_t>(min(c, o.cols / 8 - 1)) * 16u;
  // a wave's first chunks from one half, the others from the other
  constexpr int kSpan = G::kWaveM / 8;
  const int at = c / kSpan * (o.apart ? kSpan : kSpan / 2) + c % (kSpan / 2);
  return static_cast<uint32_t>(min(at, o.cols / 8 - 1)) * 16u +
         (c % kSpan < kSpan / 2 ? 0u : static_cast<uint32_t>(o.half) * 2u);
}

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
    if constexpr (!KMAJOR) {
      chunk = static_cast<uint32_t>((lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7)) * 16u;
    } else {
      chunk = column_chunk<G>(o, kslot<kChunks>(kRowsPerCopy * wave + lane / kChunks, lane % kChunks));
    }
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
      h[i] = lds_read_tr(tile + k * (2 * G::kTile) + kslot<G::kTile / 8>(k, n >> 3) * 16 + (n & 7) * 2);
    }
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
  } else {
    const int r = c0 + q16, c = 4 * kk + kq;
    return lds_read_b128(tile + r * (kStepK * 2) + (c ^ ((r >> 1) & 7)) * 16);
  }
}

// acc = A B^T over K steps [0, n_k) of every combination of parts. AGAIN: the kernel has
// other products or runs this one in a loop; what is computed from the thread's number is
// then computed here and not kept in registers from before.
template <class G, int PARTS, bool KA, bool KB, bool AGAIN = false>
__device__ __forceinline__ void tile_product(const Operand& oa, const Operand& ob, int n_k,
                                             char* smem, typename G::Acc& acc) {
  typedef Combos<PARTS> C;
  constexpr int KK = kStepK / 32;
  int tid = threadIdx.x;
  if constexpr (AGAIN) asm volatile("" : "+v"(tid));
  const int lane = tid & 63;
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

// The same for operands in three bf16 parts, all of a K step's parts at once: a step of 32
// is six tiles in LDS (A's parts, then B's), read once for the six products, where a pass
// over K for every product would copy and read twelve (dX of 999 x 768 x 2050: 38 us so,
// 47 in passes; the weights' gradients 80 and 108). Three stages, the
// copies two steps ahead; a step's fragments are read while the products of the one before
// it run, which takes most of the 512 registers that four waves on a CU have. An
// operand whose K runs along its rows lies in rows of 64 bytes, chunk c of row R in slot
// c ^ (R / 4 mod 4), so that the 16 rows that a read touches lie in different banks.
constexpr int kPartsK = 32;
template <class G> constexpr int kPartsTile = G::kTile * kPartsK * 2;
template <class G> constexpr int kPartsLds = 3 * 6 * kPartsTile<G>;

template <class G, bool KMAJOR>
struct PartsCopier {
  static constexpr int kPer = kPartsTile<G> / 1024 / G::kWaves;  // copies of a wave, step and part
  static constexpr int kChunks = KMAJOR ? G::kTile / 8 : 4, kRowsPerCopy = 64 / kChunks;
  const char* at;       // the step to copy, first part
  int64_t part_bytes;
  uint32_t ldb;         // row stride, bytes
  uint32_t kb;          // rows: byte offset of the step in a row; k-major: its K row
  uint32_t last;        // rows: last chunk of a row; k-major: last K row
  uint32_t row[kPer];   // rows: row offset; k-major: K row of the lane
  uint32_t chunk[kPer]; // byte offset of the lane's 16 bytes in the row

  __device__ __forceinline__ void init(const Operand& o, int lane, int wave) {
    at = reinterpret_cast<const char*>(o.base);
    part_bytes = o.part_stride * 2;
    ldb = static_cast<uint32_t>(o.ld) * 2u;
    kb = 0;
    last = KMAJOR ? static_cast<uint32_t>(o.rows - 1) : static_cast<uint32_t>(o.cols) * 2u - 16u;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int r = (q * G::kWaves + wave) * kRowsPerCopy + lane / kChunks, slot = lane % kChunks;
      if constexpr (KMAJOR) {
        row[q] = static_cast<uint32_t>(r);
        chunk[q] = column_chunk<G>(o, kslot<kChunks>(r, slot));
      } else {
        row[q] = static_cast<uint32_t>(min(r, o.rows - 1)) * ldb;
        chunk[q] = static_cast<uint32_t>(slot ^ ((r >> 2) & 3)) * 16u;
      }
    }
  }
  // copy j of the 3 kPer of a step
  __device__ __forceinline__ void issue(char* tiles, int wave, int j) const {
    const int p = j / kPer, q = j % kPer;
    copy_to_lds(tile_rsrc(at + p * part_bytes),
                KMAJOR ? min(row[q], last - kb) * ldb + chunk[q] : row[q] + min(kb + chunk[q], last), 0,
                tiles + p * kPartsTile<G> + (q * G::kWaves + wave) * 1024);
  }
  __device__ __forceinline__ void next_step() {
    if constexpr (KMAJOR) {
      // (past the last row of K, in the second half of a last step, the same again)
      if (kb + kPartsK > last) return;
      at += static_cast<uint64_t>(ldb) * kPartsK;
      kb += kPartsK;
    } else {
      kb += kPartsK * 2;
    }
  }
};

template <class G, bool KMAJOR>
__device__ __forceinline__ bf16x8 parts_frag(const char* tile, int c0, int lane) {
  if constexpr (KMAJOR) return tile_frag<G, true>(tile, 0, c0, lane);
  const int r = c0 + (lane & 15);
  return lds_read_b128(tile + r * (2 * kPartsK) + ((lane >> 4) ^ ((r >> 2) & 3)) * 16);
}

// acc = A B^T over n_k steps of kStepK.
template <class G, bool KA, bool KB>
__device__ __forceinline__ void parts_product(const Operand& oa, const Operand& ob, int n_k, char* smem,
                                              typename G::Acc& acc) {
  typedef Combos<3> C;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % G::kWavesM, wn = wave / G::kWavesM;
  PartsCopier<G, KA> ca;
  PartsCopier<G, KB> cb;
  ca.init(oa, lane, wave);
  cb.init(ob, lane, wave);
  constexpr int kCopies = 3 * (PartsCopier<G, KA>::kPer + PartsCopier<G, KB>::kPer);
  constexpr int kStage = 6 * kPartsTile<G>;
#pragma unroll
  for (int m = 0; m < G::kMB; ++m)
#pragma unroll
    for (int n = 0; n < G::kNB; ++n) acc.v[m][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int n_steps = n_k * (kStepK / kPartsK);
  if (n_steps <= 0) return;
  auto issue = [&](int s, int j) {  // copy j of step s
    char* const to = smem + s % 3 * kStage;
    constexpr int kA = 3 * PartsCopier<G, KA>::kPer;
    if (j < kA) ca.issue(to, wave, j);
    else cb.issue(to + 3 * kPartsTile<G>, wave, j - kA);
    if (j + 1 == kCopies) ca.next_step(), cb.next_step();
  };
  auto issue_all = [&](int s) {
#pragma unroll
    for (int j = 0; j < kCopies; ++j) issue(s, j);
  };
  bf16x8 fa[2][3][G::kMB], fb[2][3][G::kNB];
  constexpr int kFrags = 3 * (G::kMB + G::kNB);
  auto read = [&](int s, int to, int j) {  // fragment j of step s
    const char* const from = smem + s % 3 * kStage;
    if (j < 3 * G::kMB) {
      const int p = j / G::kMB, m = j % G::kMB;
      fa[to][p][m] = parts_frag<G, KA>(from + p * kPartsTile<G>, G::kWaveM * wm + 16 * m, lane);
    } else {
      const int p = (j - 3 * G::kMB) / G::kNB, n = (j - 3 * G::kMB) % G::kNB;
      fb[to][p][n] = parts_frag<G, KB>(from + (3 + p) * kPartsTile<G>, G::kWaveN * wn + 16 * n, lane);
    }
  };
  // Step s: the copies of s + 1 are complete once at most those of s + 2 are in flight,
  // and once every wave has read step s, s + 3 takes its place. Reads and copies go
  // between the products, a row of blocks at a time: issued at once they would leave the
  // matrix cores idle for as long as the products take. LEFT: the steps there are after
  // it, 3 for more; no test inside a step, on whose joining paths the compiler would have
  // the products wait for the newest fragments.
  issue_all(0);
  issue_all(1);
  wait_vm_all<kCopies>();
  lds_barrier();
  if (n_steps > 2) issue_all(2);  // (n_steps is even)
#pragma unroll
  for (int j = 0; j < kFrags; ++j) read(0, 0, j);
  auto step = [&](int s, auto at, auto left) {
    constexpr int cur = decltype(at)::value, LEFT = decltype(left)::value;
    constexpr int kGroups = C::n * G::kMB;
    if constexpr (LEFT >= 1) {
      wait_lgkm0();
      wait_vm_all<LEFT >= 2 ? kCopies : 0>();
      lds_barrier();
    }
    each<kGroups>([&](auto group) {
      constexpr int g = decltype(group)::value, c = g / G::kMB, m = g % G::kMB;
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int n = 0; n < G::kNB; ++n)
        acc.v[m][n] = mfma<3>(fa[cur][C::a(c)][m], fb[cur][C::b(c)][n], acc.v[m][n]);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (LEFT >= 1) {
#pragma unroll
        for (int j = g * kFrags / kGroups; j < (g + 1) * kFrags / kGroups; ++j) read(s + 1, cur ^ 1, j);
      }
      if constexpr (LEFT >= 3) {
#pragma unroll
        for (int j = g * kCopies / kGroups; j < (g + 1) * kCopies / kGroups; ++j) issue(s + 3, j);
      }
    });
  };
  constexpr std::integral_constant<int, 0> even;
  constexpr std::integral_constant<int, 1> odd;
  constexpr std::integral_constant<int, 3> more;
  if (n_steps > 2) {
#pragma unroll 1
    for (int s = 0; s < n_steps - 4; s += 2) {
      step(s, even, more);
      step(s + 1, odd, more);
    }
    step(n_steps - 4, even, more);
    step(n_steps - 3, odd, std::integral_constant<int, 2>{});
  }
  step(n_steps - 2, even, odd);
  step(n_steps - 1, odd, even);
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

// fn(std::true_type) where a tile reaches past the piece's last column,
// fn(std::false_type) for the others, whose columns need no test.
template <class F>
__device__ __forceinline__ void with_edge(bool edge, F fn) {
  if (edge) fn(std::true_type{});
  else fn(std::false_type{});
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

// Transposes the lane quarters (kq = lane / 16) of a wave against four registers: x[j]
// of quarter kq and x[kq] of quarter j change places. What an accumulator holds as runs
// of four columns then becomes 16 bytes of one row, without LDS.
__device__ __forceinline__ void swap16(uint32_t& x, uint32_t& y) {
  const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
  x = r[0], y = r[1];
}
__device__ __forceinline__ void swap32(uint32_t& x, uint32_t& y) {
  const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
  x = r[0], y = r[1];
}
__device__ __forceinline__ void transpose4(u32x4& x) {
  uint32_t r[4] = {x[0], x[1], x[2], x[3]};
  swap16(r[0], r[1]), swap16(r[2], r[3]);
  swap32(r[0], r[2]), swap32(r[1], r[3]);
  x = u32x4{r[0], r[1], r[2], r[3]};
}
// Two neighbouring blocks of 16 columns of an accumulator's row in bf16 (the lane's four
// columns of either), as the 8 columns from pair_col(kq) on of the 32.
__device__ __forceinline__ int pair_col(int kq) { return 16 * (kq & 1) + 8 * (kq >> 1); }
__device__ __forceinline__ bf16x8 pair_cols(Vec4<bf16>::type a, Vec4<bf16>::type b) {
  typedef uint32_t u2 __attribute__((ext_vector_type(2)));
  u2 x = __builtin_bit_cast(u2, a), y = __builtin_bit_cast(u2, b);
  uint32_t x0 = x[0], x1 = x[1], y0 = y[0], y1 = y[1];
  swap16(x0, y0), swap16(x1, y1);
  return __builtin_bit_cast(bf16x8, u32x4{x0, x1, y0, y1});
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

// ------------------------------------------------------------------- host --

inline int fail(int code, const std::string& msg) { return record_error(code, msg.c_str()); }

inline int check_launch(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(DPG_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
  return DPG_OK;
}

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

inline int check_ws(const void* ws, size_t have, size_t need) {
  if (need > 0 && !ws) return fail(DPG_ERR_WORKSPACE, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(DPG_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (have < need)
    return fail(DPG_ERR_WORKSPACE, "workspace of " + std::to_string(have) + " bytes, " +
                                       std::to_string(need) + " needed");
  return DPG_OK;
}

// Whether a launch of `tiles` big tiles takes them. Fewer than three for every
// four CUs leave too much of the chip idle, and a K step of a big tile takes 64
// KiB through a CU's LDS where a small one takes 32 (128 rows x 64 against 1000
// columns, fp32: 18 us big, 12 us small; 252 big tiles of a product of six at 999 x
// 768 x 32003: 311 us big, 424 us small). With at most 128 rows half of a big
// tile would be padding (4 rows x 2048 against 50304 columns: 53 us big, 40 us
// small).
inline bool big_tiles(int64_t tiles, int64_t rows) { return tiles >= 192 && rows > SmallTile::kTile; }

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
inline Split choose_split(int64_t m, int64_t n, int64_t steps, int combos, bool sums_anyway) {
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

inline unsigned blocks_of(int64_t n, int64_t per) { return static_cast<unsigned>(ceil_div(n, per)); }
// grid of tile_of_block for mt x nt tiles
inline dim3 tile_grid(int64_t mt, int64_t nt) { return dim3(static_cast<unsigned>(round_up(mt * nt, 8))); }

}  // namespace dpg
